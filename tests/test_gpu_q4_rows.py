"""The 4-bit cache's writer, and caches of every kind read back."""
import pytest

torch = pytest.importorskip("torch")
from tests.paged_ref import HALF, Problem, turn  # noqa: E402
from tests.q4_ref import GROUP, MOST_K, MOST_V, Problem4, pack, quantise, unpack  # noqa: E402
from tests.test_gpu_rows import CASES, magnitude, places, randn, slot_view  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sage():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_attention_smooth_gb300 import sage
    return sage


ALL = CASES + [([5000, 0, 1, 2999], [5100, 0, 5, 2900])]     # the last: the kernel for many tokens
SHAPES = [(128, 8, 16, "NHD", False), (80, 3, 32, "HND", True), (64, 1, 64, "NHD", True),
          (40, 5, 48, "HND", False), (104, 2, 16, "NHD", False), (8, 2, 16, "HND", False),
          (32, 4, 256, "NHD", False)]


def wanted(p, k, v):
    """Packed rows and scales of k and v, to the bit."""
    d = p.d
    inv = torch.where(p.v_scale > 0, torch.ones_like(p.v_scale) / (64 * p.v_scale), 0.0)[:, :d]
    kn, ks = quantise(k.float() - p.k_mean[:, :d], MOST_K)
    vn, vs = quantise(v.float() * inv, MOST_V)
    return pack(kn), ks, pack(vn), vs


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,hkv,page,layout,both", SHAPES)
@pytest.mark.parametrize("case", range(len(ALL)))
def test_append(sage, dt, d, hkv, page, layout, both, case):
    q_lens, kv_lens = ALL[case]
    p = Problem4(q_lens, kv_lens, hkv, hkv, d, page, layout, dt, seed=23, both=both, poison=False,
                 offset=3.0, spare_rows=2)
    k, v = randn(24, p.q.shape[0], hkv, d, dt=dt), randn(25, p.q.shape[0], hkv, d, dt=dt)
    if k.shape[0] > 4:
        k[2] = 0.0
        p.k_mean[0] = 0.0                                # keys equal to their mean: zero codes
        k[3] = 60000.0                                   # beyond the largest scale with a mean below
        p.k_mean[-1, 0] = -30000.0
        v[3, 0] = 1e-6 if dt == torch.bfloat16 else 0.0  # scales of zero
    p.v_scale[0, 1] = 0.0
    v[0, 0, 0] = 1000.0                                  # saturates
    before = [t.clone() for t in (p.k, p.v, p.k_groups, p.v_groups)]
    cache, batch = p.sage(sage)
    rows, pages, slots, pos = places(p)
    ws = sage.alloc_workspace_paged()
    sage.kv_append(cache, batch, k, v, ws=ws)
    assert sage.device_status(ws) == sage.OK, sage.last_error()
    wk, ws_, wv, wvs = wanted(p, k[rows], v[rows])
    slot_view(p, before[0])[pages, slots] = wk
    slot_view(p, before[1])[pages, slots] = wv
    for got, want in ((p.k, before[0]), (p.v, before[1])):
        assert torch.equal(got, want)
    g = -(-d // GROUP)
    for t, s, got in ((before[2], ws_, p.k_groups), (before[3], wvs, p.v_groups)):
        t[pages, :, slots, :g] = s
        t[pages, :, slots, g:] = 0                       # groups behind D
        assert torch.equal(t.view(torch.int16), got.view(torch.int16))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,hkv,page,layout,both", SHAPES[:5])
@pytest.mark.parametrize("r,interleaved", [(8, False), (8, True), (-1, False), (-1, True)])
@pytest.mark.parametrize("case", [1, 3, len(ALL) - 1])
def test_append_with_rotation(sage, dt, d, hkv, page, layout, both, r, interleaved, case):
    q_lens, kv_lens = ALL[case]
    r = d if r < 0 else r
    p = Problem4(q_lens, kv_lens, 2 * hkv, hkv, d, page, layout, dt, seed=26, both=both, poison=False,
                 offset=2.0)
    k, v = randn(27, p.q.shape[0], hkv, d, dt=dt), randn(28, p.q.shape[0], hkv, d, dt=dt)
    cache, batch = p.sage(sage)
    rows, pages, slots, pos = places(p)
    f, gain = sage.rope_freqs(r, scaling="yarn", factor=4.0)
    q = sage.kv_append(cache, batch, k, v, q=p.q, inv_freq=f, interleaved=interleaved, mscale=gain)
    qr, _ = sage.rope(p.q[rows], None, pos, f, interleaved, gain)
    assert torch.equal(q[rows], qr)
    _, _, wv, wvs = wanted(p, k[rows], v[rows])
    assert torch.equal(slot_view(p, p.v)[pages, slots], wv)
    x = turn(k[rows], pos, f, interleaved, gain) - p.k_mean[:, :d].double()
    s = p.k_groups[pages, :, slots][..., :-(-d // GROUP)].double()
    wide = s.repeat_interleave(GROUP, -1)[..., :d]
    # the rotation's fp32 error (2^-20 of the pair) and one subtraction
    err = 2.0 ** -20 * magnitude(k[rows], r, interleaved, gain) + 2.0 ** -24 * x.abs()
    top = torch.nn.functional.pad(x.abs(), (0, -d % GROUP)).unflatten(-1, (-1, GROUP)).amax(-1)
    most = torch.nn.functional.pad(err, (0, -d % GROUP)).unflatten(-1, (-1, GROUP)).amax(-1)
    # the scale: that error, two fp32 roundings, fp16's
    assert ((s - top / 7).abs() <= (most + 2.0 ** -22 * top) / 7 + 2.0 ** -11 * top / 7 * 1.01 + 2.0 ** -25).all()
    back = unpack(slot_view(p, p.k)[pages, slots])[..., :d].double() * wide
    # half a code, and the scale's rounding down at the group's largest (7 * 2^-11 of a code)
    assert ((back - x).abs() <= wide * (0.5 + 2.0 ** -8) + 2 * err + 2.0 ** -24).all()


def test_append_bad_entries(sage):
    p = Problem4([2, 2, 2], [40, 40, 40], 4, 2, 64, 16, seed=26, poison=False)
    k, v = randn(27, 6, 2, 64), randn(28, 6, 2, 64)
    p.table[1, 2] = p.k.shape[0]                        # one past the pool
    bk, bv, bs = p.k.clone(), p.v.clone(), p.k_groups.clone()
    ws = sage.alloc_workspace_paged()
    sage.kv_append(*p.sage(sage), k, v, ws=ws)
    assert sage.device_status(ws) == sage.ERR_INVALID_ARG and "block table" in sage.last_error()
    same = torch.ones(p.k.shape[0], 16, dtype=torch.bool, device="cuda")
    for i in (0, 2):
        same[p.table[i, 2].long(), 6:8] = False
    assert torch.equal(p.k[same], bk[same]) and torch.equal(p.v[same], bv[same])
    assert torch.equal(p.k_groups.transpose(1, 2)[same].view(torch.int16),
                       bs.transpose(1, 2)[same].view(torch.int16))


# ------------------------------------------------------------------ gather
def problem(kind, dt, q_lens, kv_lens, hkv, d, page, layout, both=False, seed=40):
    if kind == "q4":
        return Problem4(q_lens, kv_lens, hkv, hkv, d, page, layout, dt, seed=seed, both=both,
                        poison=False, offset=3.0, spare_rows=3)
    return Problem(q_lens, kv_lens, hkv, hkv, d, page, layout, kind, dt, seed=seed, both=both,
                   poison=False, offset=3.0, spare_rows=3)


KINDS = [("q4", torch.bfloat16), ("q4", torch.float16), ("q8", torch.bfloat16),
         ("q8", torch.float16), ("bf16", torch.bfloat16), ("f16", torch.float16)]


@pytest.mark.parametrize("kind,dt", KINDS)
@pytest.mark.parametrize("d,hkv,page,layout,both", SHAPES)
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1, 1], [1, 16, 333]), ([3, 0, 50, 9], [3, 9, 200, 4]),
                                            ([1700, 1, 2500], [1700, 50, 2600])])
def test_gather(sage, kind, dt, d, hkv, page, layout, both, q_lens, kv_lens):
    p = problem(kind, dt, q_lens, kv_lens, hkv, d, page, layout, both)
    cache, batch = p.sage(sage)
    n = sum(q_lens)
    ko, vo = (torch.full((n + 3, hkv, d), 7.0, dtype=dt, device="cuda") for _ in range(2))
    ws = sage.alloc_workspace_paged()
    k, v = sage.kv_gather(cache, batch, n + 3, dt, k_out=ko, v_out=vo, ws=ws)
    assert k is ko and v is vo and sage.device_status(ws) == sage.OK
    rows, pages, slots, pos = places(p)
    if kind == "q4":
        wk, wv = p.rows("k", pages, slots), p.rows("v", pages, slots)
    elif kind == "q8":
        wk = slot_view(p, p.k)[pages, slots].double() * p.k_scale[pages, :, slots].double()[..., None]
        wv = (slot_view(p, p.v).view(torch.uint8)[pages, slots].view(torch.float8_e4m3fn).double() *
              p.v_scale[:, :d].double())
    if kind in ("q4", "q8"):
        wk = wk + p.k_mean[:, :d].double()
        # fp32: the product (exact with 4 bits) and the sum or second product, then 16 bits
        for got, want, mag in ((k, wk, wk.abs() + 2 * p.k_mean[:, :d].double().abs()), (v, wv, wv.abs())):
            diff = (got[rows].double() - want).abs()
            assert (diff <= HALF[dt] * want.abs() + 2.0 ** -22 * mag + 2.0 ** -25).all()
    else:
        assert torch.equal(k[rows], slot_view(p, p.k)[pages, slots])
        assert torch.equal(v[rows], slot_view(p, p.v)[pages, slots])
    empty = torch.ones(n, dtype=torch.bool, device="cuda")
    empty[rows] = False                                  # negative positions
    assert (k[:n][empty] == 0).all() and (v[:n][empty] == 0).all()
    assert (k[n:] == 7.0).all() and (v[n:] == 7.0).all()


@pytest.mark.parametrize("kind,dt", KINDS)
def test_gather_views_and_bad_pages(sage, kind, dt):
    p = problem(kind, dt, [40, 40], [40, 40], 2, 72, 16, "NHD")
    cache, batch = p.sage(sage)
    k, v = sage.kv_gather(cache, batch, 80, dt)
    kv = torch.full((80, 5, 73), 7.0, dtype=dt, device="cuda")
    views = kv[:, :2, 1:], kv[:, 2:4, :72]               # rows on 2-byte boundaries
    sage.kv_gather(cache, batch, 80, k_out=views[0], v_out=views[1])
    assert torch.equal(views[0], k) and torch.equal(views[1], v)
    assert (kv[:, 4] == 7.0).all() and (kv[:, :2, 0] == 7.0).all() and (kv[:, 2:4, 72] == 7.0).all()
    p.table[1, 1] = -3
    ws = sage.alloc_workspace_paged()
    k2, v2 = sage.kv_gather(*p.sage(sage), 80, dt, ws=ws)
    assert sage.device_status(ws) == sage.ERR_INVALID_ARG
    assert (k2[56:72] == 0).all() and (v2[56:72] == 0).all()
    k[56:72] = 0
    assert torch.equal(k2, k)
    assert sage.kv_gather(cache, batch, 0, dt)[0].shape == (0, 2, 72)
    with pytest.raises(TypeError, match="does not give"):
        sage.kv_gather(cache, batch, 80, torch.float32)
    with pytest.raises(ValueError, match="k_out"):
        sage.kv_gather(cache, batch, 80, dt, k_out=k[:5])


def test_gather_of_whole_sequences_feeds_the_dense_call(sage):
    """A prompt stored in four bits, read back whole and attended densely, against the formula on
    the values that the cache stands for."""
    hkv, d, n = 2, 64, 100
    p = Problem4([n], [n], hkv, hkv, d, 16, "NHD", torch.float16, seed=50, poison=False)
    p.k_mean.normal_()
    k, v = randn(51, n, hkv, d, dt=torch.float16), randn(52, n, hkv, d, dt=torch.float16)
    cache, batch = p.sage(sage)
    sage.kv_append(cache, batch, k, v)
    k2, v2 = sage.kv_gather(cache, batch, n, torch.float16)
    # half a code of each (the scales' roundings add 2^-9 of one), unless V saturates
    unit = p.k_groups[p.table[0, :7].long()].transpose(1, 2).flatten(0, 1)[:n].double()
    assert ((k2.double() - k.double()).abs() <= unit.repeat_interleave(32, -1)[..., :d] * 0.51 + 2.0 ** -9).all()
    q = randn(53, n, hkv, d, dt=torch.float16)
    out = sage.sageattn(q[None], k2[None], v2[None], "NHD", is_causal=True)[0]
    ref = p.reference
    p.q = q
    want = ref()[0]
    # the dense call quantises K to 8 and V and P to e4m3 in its own way: 2^-4 of the values
    assert float((out.double() - want).abs().max()) <= 2.0 ** -3 * float(v2.double().abs().max())
