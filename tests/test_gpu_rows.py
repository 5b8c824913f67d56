"""Rotary positions and the paged cache's writer against 64-bit forms, and the
serving operators together."""
import pytest

torch = pytest.importorskip("torch")
from tests.paged_ref import HALF, Problem, turn  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sage():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_attention_smooth_gb300 import sage
    return sage


def randn(seed, *shape, dt=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dt)


def near(got, ref, mag):
    """One rounding to got's type, and fp32 arithmetic on magnitudes `mag`: cos
    and sin within 2^-21 (their argument's cut to fp32 and their own error),
    three roundings of 2^-24 each."""
    u = HALF[got.dtype]
    # fp16's smallest step is 2^-24, half of it 2^-25
    bound = u * ref.abs() + 2.0 ** -20 * mag + (2.0 ** -25 if got.dtype == torch.float16 else 0)
    diff = (got.double() - ref).abs()
    assert (diff <= bound).all(), float((diff / bound).max())


def magnitude(x, r, interleaved, gain=1.0):
    """|x1| + |x2| of each channel's pair."""
    a = x.double().abs()
    m = a.clone()
    i, j = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    m[..., i] = m[..., j] = (a[..., i] + a[..., j]) * gain
    return m


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,r", [(128, 128), (128, 64), (64, 16), (80, 80), (40, 20), (128, 2),
                                 (72, 36), (3, 2), (1 + 32, 30), (120, 120)])
@pytest.mark.parametrize("t", [1, 7, 700])
def test_rope(sage, dt, interleaved, d, r, t):
    q, k = randn(1, t, 5, d, dt=dt), randn(2, t, 2, d, dt=dt)
    pos = torch.randint(0, 1 << 20, (t,), device="cuda")
    f, gain = sage.rope_freqs(r, scaling="yarn", factor=4.0)
    qo, ko = sage.rope(q, k, pos, f, interleaved, gain)
    for x, y in ((q, qo), (k, ko)):
        near(y, turn(x, pos, f, interleaved, gain), magnitude(x, r, interleaved, gain))
        assert torch.equal(y[..., r:], x[..., r:])
    # int32 positions, and in place
    qi, ki = q.clone(), k.clone()
    sage.rope(qi, ki, pos.int(), f, interleaved, gain, q_out=qi, k_out=ki)
    assert torch.equal(qi, qo) and torch.equal(ki, ko)
    only, none = sage.rope(q, None, pos, f, interleaved, gain)
    assert none is None and torch.equal(only, qo)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_views(sage, interleaved):
    qkv = randn(3, 333, 12, 64, dt=torch.float16)
    q, k = qkv[:, :6], qkv[:, 6:9]
    pos = torch.arange(333, device="cuda")
    f, _ = sage.rope_freqs(64)
    want = sage.rope(q.contiguous(), k.contiguous(), pos, f, interleaved)
    got = sage.rope(q, k, pos, f, interleaved)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    v = qkv[:, 9:].clone()
    sage.rope(q, k, pos, f, interleaved, q_out=q, k_out=k)     # inside the projection
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[:, 9:], v)
    odd = randn(4, 50, 3, 65, dt=torch.float16)[..., 1:]       # rows on 2-byte boundaries
    a, _ = sage.rope(odd, None, pos[:50], f, interleaved)
    b, _ = sage.rope(odd.contiguous(), None, pos[:50], f, interleaved)
    assert torch.equal(a, b)
    sage.rope(odd, None, pos[:50], f, interleaved, q_out=odd)
    assert torch.equal(odd, b)


def test_rope_far_and_negative_positions(sage):
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, 10 ** 6 + 7, 2 ** 40 + 3],
                       device="cuda")
    f = torch.tensor([1.0, 0.37, 1e-4, 6.5, 0.0, 100.25], dtype=torch.float64, device="cuda")
    q = randn(5, 8, 2, 16, dt=torch.float16)
    got, _ = sage.rope(q, None, pos, f)
    ref = turn(q, pos, f)
    # the double product's own error at 2^40 * 100 rad is 2^-53 * 2^47 = 2^-6; below it the
    # 64-bit reference is itself exact enough
    fine = [i for i in range(8) if i != 7]
    near(got[fine], ref[fine], magnitude(q, 12, False)[fine])
    assert torch.equal(got[0], q[0])


def test_rope_inverse_is_the_gradient(sage):
    """<R x, g> = <x, R' g>: the inverse call is the transpose; and differences
    of the loss along single channels agree with it."""
    t, h, d, r = 9, 3, 32, 24
    x, g = randn(6, t, h, d, dt=torch.float16), randn(7, t, h, d, dt=torch.float16)
    pos = torch.randint(0, 5000, (t,), device="cuda")
    f, gain = sage.rope_freqs(r, scaling="yarn", factor=2.0)
    for inter in (False, True):
        grad, _ = sage.rope(g, None, pos, f, inter, gain, inverse=True)
        ref = turn(g, pos, f, inter, gain, sign=-1.0)
        near(grad, ref, magnitude(g, r, inter, gain))
        lhs = (turn(x, pos, f, inter, gain) * g.double()).sum()
        rhs = (x.double() * ref).sum()
        assert abs(float(lhs - rhs)) <= 1e-9 * float(x.double().abs().sum())
        for ch in (0, 5, 13, r - 1, r, d - 1):           # linear: a difference of any size is exact
            e = torch.zeros_like(x)
            e[4, 1, ch] = 1.0
            moved, _ = sage.rope(e, None, pos, f, inter, gain)
            slope = float((moved.double() * g.double()).sum())
            # two fp16 roundings of the moved pair (2^-11 each times |g| <= 4), one of grad
            assert abs(slope - float(grad[4, 1, ch])) <= 2.0 ** -11 * 4 * 3 * gain


def test_the_binding_refuses_what_it_would_misread(sage):
    q, pos = randn(8, 3, 2, 64), torch.arange(3, device="cuda")
    f, _ = sage.rope_freqs(64)
    for bad, match in [((q[0], None, pos, f), r"\(T, H, D\)"), ((q.float(), None, pos, f), "float16"),
                       ((q, q.half(), pos, f), "not torch.bfloat16"), ((q, q[:2], pos, f), "shape"),
                       ((q, None, pos[:2], f), "positions"), ((q, None, pos.float(), f), "positions"),
                       ((q, None, pos.cpu(), f), "positions is not on"), ((q, None, pos, f.float()), "inv_freq"),
                       ((q.transpose(1, 2), None, pos, f), "contiguous channels")]:
        with pytest.raises((ValueError, TypeError), match=match):
            sage.rope(*bad)
    with pytest.raises(ValueError, match="q_out has shape"):
        sage.rope(q, None, pos, f, q_out=q[:2])
    with pytest.raises(sage.SageError, match="even"):
        sage.rope(q, None, pos, torch.ones(33, dtype=torch.float64, device="cuda"))
    p = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    cache = sage.PagedCache(p, p.clone())
    batch = sage.PagedBatch(torch.tensor([0, 3], dtype=torch.int32, device="cuda"),
                            torch.tensor([3], dtype=torch.int32, device="cuda"),
                            torch.zeros(1, 1, dtype=torch.int32, device="cuda"), 3, 16)
    with pytest.raises(ValueError, match="do not fit"):
        sage.kv_append(cache, batch, q[:, :1], q[:, :1])
    with pytest.raises(sage.SageError, match="kind"):
        sage.kv_append(cache, batch, q.half(), q.half())
    with pytest.raises(ValueError, match="channels"):
        sage.attn_paged(cache, batch, q[..., :32])
    with pytest.raises(ValueError, match="contiguous"):
        sage.attn_paged(cache, batch, q, out=randn(9, 3, 4, 64)[:, ::2])
    with pytest.raises(ValueError, match="lse"):
        sage.attn_paged(cache, batch, q, lse=torch.zeros(3, 2, device="cuda").double())
    for bad, match in [((p, p.half()), "bfloat16"), ((p, p[:2]), "one shape"),
                       ((p.to(torch.int8), p.to(torch.float8_e4m3fn)), "k_scale"),
                       ((p, p.transpose(1, 2).contiguous().transpose(1, 2)), "strides")]:
        with pytest.raises((ValueError, TypeError), match=match):
            sage.PagedCache(*bad)
    with pytest.raises(TypeError, match="int32"):
        sage.PagedBatch(batch.cu_q.long(), batch.kv_lens, batch.block_table, 3, 16)
    with pytest.raises(ValueError, match="entries"):
        sage.PagedBatch(batch.cu_q[:1], batch.kv_lens, batch.block_table, 3, 16)


def test_rope_frequencies(sage):
    f, g = sage.rope_freqs(64, base=500.0)
    assert g == 1.0 and torch.allclose(f, 500.0 ** (-torch.arange(32, device="cuda").double() / 32),
                                       rtol=1e-15)
    lin, _ = sage.rope_freqs(64, base=500.0, scaling="linear", factor=4.0)
    assert torch.equal(lin, f / 4)
    ntk, _ = sage.rope_freqs(64, base=500.0, scaling="ntk", factor=4.0)
    assert torch.allclose(ntk[[0, -1]], torch.stack((f[0], f[-1] / 4)), rtol=1e-12)
    part, one = sage.rope_freqs(64, scaling="by_parts", factor=8.0)
    plain, _ = sage.rope_freqs(64)
    assert one == 1.0 and part[0] == plain[0] and torch.isclose(part[-1], plain[-1] / 8, rtol=1e-14)
    _, gain = sage.rope_freqs(64, scaling="yarn", factor=8.0)
    assert abs(gain - (0.1 * 2.0794415416798357 + 1)) < 1e-15


# ------------------------------------------------------------------ append
def places(p):
    """(row, page, slot, position) of every new token that has a place."""
    rows, pages, slots, pos = [], [], [], []
    a = 0
    for i, n in enumerate(p.q_lens):
        for t in range(n):
            j = p.kv_lens[i] - n + t
            if j >= 0:
                rows.append(a + t)
                pages.append(int(p.table[i, j // p.page]))
                slots.append(j % p.page)
                pos.append(j)
        a += n
    dev = p.q.device
    return [torch.tensor(x, device=dev) for x in (rows, pages, slots, pos)]


def slot_view(p, t):
    return t if p.layout == "NHD" else t.transpose(1, 2)


CASES = [([1, 1, 1], [1, 16, 333]), ([3, 0, 50, 7], [3, 9, 200, 4]), ([300, 1], [300, 77]),
         ([410, 1, 300], [410, 50, 333]), ([3000, 0, 1, 2500], [3100, 0, 5, 2400])]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,hkv,page,layout,both", [(128, 8, 16, "NHD", False), (80, 3, 32, "HND", True),
                                                    (64, 1, 64, "NHD", True), (40, 5, 48, "HND", False),
                                                    (8, 2, 16, "NHD", False)])
@pytest.mark.parametrize("r,interleaved", [(0, False), (8, False), (8, True), (-1, False), (-1, True)])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_append_16bit(sage, dt, d, hkv, page, layout, both, r, interleaved, case):
    q_lens, kv_lens = CASES[case]
    r = d if r < 0 else r
    p = Problem(q_lens, kv_lens, 2 * hkv, hkv, d, page, layout,
                "bf16" if dt == torch.bfloat16 else "f16", dt, seed=20, both=both, poison=False,
                spare_rows=2)
    k, v = randn(21, p.q.shape[0], hkv, d, dt=dt), randn(22, p.q.shape[0], hkv, d, dt=dt)
    before_k, before_v = p.k.clone(), p.v.clone()
    cache, batch = p.sage(sage)
    ws = sage.alloc_workspace_paged()
    rows, pages, slots, pos = places(p)
    q_out = torch.full_like(p.q, 7.0)
    if r:
        f, gain = sage.rope_freqs(r, scaling="yarn", factor=3.0)
        sage.kv_append(cache, batch, k, v, q=p.q, q_out=q_out, inv_freq=f, interleaved=interleaved,
                       mscale=gain, ws=ws)
        # the same numbers as the stand-alone rotation, to the bit
        kr, _ = sage.rope(k[rows], None, pos, f, interleaved, gain)
        qr, _ = sage.rope(p.q[rows], None, pos, f, interleaved, gain)
        assert torch.equal(q_out[rows], qr)
        assert (q_out[sum(q_lens):] == 7.0).all()
        near(kr, turn(k[rows], pos, f, interleaved, gain), magnitude(k[rows], r, interleaved, gain))
    else:
        assert sage.kv_append(cache, batch, k, v, ws=ws) is None
        kr = k[rows]
    assert sage.device_status(ws) == sage.OK, sage.last_error()
    slot_view(p, before_k)[pages, slots] = kr
    slot_view(p, before_v)[pages, slots] = v[rows]
    assert torch.equal(p.k, before_k) and torch.equal(p.v, before_v)     # and nothing else moved


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,hkv,page,layout,both", [(128, 8, 16, "NHD", False), (80, 3, 32, "HND", True),
                                                    (64, 1, 64, "NHD", True), (40, 5, 48, "HND", False),
                                                    (104, 2, 16, "NHD", False)])
@pytest.mark.parametrize("r", [0, 8, -1])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_append_q8(sage, dt, d, hkv, page, layout, both, r, case):
    q_lens, kv_lens = CASES[case]
    r = d if r < 0 else r
    p = Problem(q_lens, kv_lens, hkv, hkv, d, page, layout, "q8", dt, seed=23, both=both,
                poison=False, offset=3.0)
    k, v = randn(24, p.q.shape[0], hkv, d, dt=dt), randn(25, p.q.shape[0], hkv, d, dt=dt)
    if k.shape[0] > 2:
        k[2] = 0.0
        p.k_mean[0] = 0.0                                # a key equal to its mean: zero codes
    p.v_scale[0, 1] = 0.0
    v[0, 0, 0] = 1000.0                                  # saturates
    bk, bv, bs = p.k.clone(), p.v.view(torch.uint8).clone(), p.k_scale.clone()
    cache, batch = p.sage(sage)
    rows, pages, slots, pos = places(p)
    ws = sage.alloc_workspace_paged()
    f, gain = sage.rope_freqs(r) if r else (None, 1.0)
    sage.kv_append(cache, batch, k, v, inv_freq=f, mscale=gain, ws=ws)
    assert sage.device_status(ws) == sage.OK, sage.last_error()
    # values: one e4m3 rounding of one fp32 product
    inv = torch.where(p.v_scale > 0, p.v_scale.reciprocal(), 0.0)[:, :d]
    want_v = (v[rows].float() * inv).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    slot_view(p, bv)[pages, slots] = want_v
    assert torch.equal(p.v.view(torch.uint8), bv)
    mean = p.k_mean[:, :d]
    got_k, got_s = slot_view(p, p.k)[pages, slots], p.k_scale[pages, :, slots]
    if r:
        x = turn(k[rows], pos, f) - mean.double()
        top = x.abs().amax(-1)
        # the rotation's fp32 error (see near) on |k| and one subtraction
        err = (2.0 ** -20 * magnitude(k[rows], r, False) + 2.0 ** -24 * x.abs()).amax(-1)
        assert ((got_s.double() - top / 127).abs() <= (err + 2.0 ** -23 * top) / 127 + 1e-38).all()
        back = got_k.double() * got_s.double()[..., None]
        # half a code, and the error of x
        bound = (got_s.double() * 0.5 * (1 + 2.0 ** -15) + 2 * err)[..., None] + 1e-30
        assert ((back - x).abs() <= bound).all()
    else:
        x = k[rows].float() - mean
        top = x.abs().amax(-1, keepdim=True)
        most = torch.full_like(top, 127.0)               # tensor / tensor: one rounding
        code = torch.where(top > 0, torch.round(x * (most / top)), 0.0).to(torch.int8)
        assert torch.equal(got_k, code) and torch.equal(got_s, (top / most).squeeze(-1))
    slot_view(p, bk)[pages, slots] = got_k
    bs[pages, :, slots] = got_s
    assert torch.equal(p.k, bk) and torch.equal(p.k_scale, bs)           # and nothing else moved


@pytest.mark.parametrize("kind", ["bf16", "q8"])
def test_append_bad_entries(sage, kind):
    p = Problem([2, 2, 2], [40, 40, 40], 4, 2, 64, 16, "NHD", kind, seed=26, poison=False)
    k, v = randn(27, 6, 2, 64), randn(28, 6, 2, 64)
    p.table[1, 2] = p.k.shape[0]                        # one past the pool
    bk, bv = p.k.clone(), p.v.view(torch.uint8).clone()
    ws = sage.alloc_workspace_paged()
    sage.kv_append(*p.sage(sage), k, v, ws=ws)
    assert sage.device_status(ws) == sage.ERR_INVALID_ARG and "block table" in sage.last_error()
    same = torch.ones(p.k.shape[0], 16, dtype=torch.bool, device="cuda")
    for i in (0, 2):
        same[p.table[i, 2].long(), 6:8] = False
    assert torch.equal(p.k[same], bk[same])
    assert torch.equal(p.v.view(torch.uint8)[same], bv[same])
    p.lens[2] = 10 ** 6
    ws = sage.alloc_workspace_paged()
    sage.kv_append(*p.sage(sage), k, v, ws=ws)
    assert sage.device_status(ws) == sage.ERR_INVALID_ARG


def test_append_views_and_many_tokens(sage):
    """Slices of a fused projection, thousands of tokens, pages of another stride."""
    n = [1500, 700, 1, 2000]
    p = Problem(n, n, 6, 2, 128, 32, "NHD", "f16", torch.float16, seed=29, both=True, poison=False)
    qkv = randn(30, sum(n), 10, 128, dt=torch.float16)
    q, k, v = qkv[:, :6], qkv[:, 6:8], qkv[:, 8:]
    f, gain = sage.rope_freqs(128)
    qo = sage.kv_append(*p.sage(sage), k, v, q=q, inv_freq=f)
    rows, pages, slots, pos = places(p)
    kr, _ = sage.rope(k, None, pos, f)
    qr, _ = sage.rope(q, None, pos, f)
    assert torch.equal(qo, qr)
    assert torch.equal(p.k[pages, slots], kr) and torch.equal(p.v[pages, slots], v)


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("kind,dt", [("bf16", torch.bfloat16), ("f16", torch.float16),
                                     ("q8", torch.bfloat16)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 4)])
def test_a_prompt_then_decoding(sage, kind, dt, window, sinks):
    """A served sequence: the prompt in two chunks, then single tokens, against
    attention of the whole sequence in 64 bits; the quantised cache takes its
    means and scales from kv_stats_noalloc on the prompt's rotated keys."""
    hq, hkv, d, page, total = 8, 2, 64, 16, 150
    q, k, v = (randn(40 + i, total, h, d, dt=dt) for i, h in enumerate((hq, hkv, hkv)))
    k = (k.float() + 2.0).to(dt)
    f, _ = sage.rope_freqs(d)
    pos = torch.arange(total, device="cuda")
    qr, kr = turn(q, pos, f), turn(k, pos, f)
    pages = 12
    cache_dt = torch.int8 if kind == "q8" else dt
    kp = torch.zeros(pages, page, hkv, d, dtype=cache_dt, device="cuda")
    vp = torch.zeros(pages, page, hkv, d, device="cuda").to(torch.float8_e4m3fn if kind == "q8" else dt)
    extra = {}
    if kind == "q8":
        mean, scale = torch.empty(hkv * 64, device="cuda"), torch.empty(hkv * 64, device="cuda")
        sage.kv_stats_noalloc(kr[None].to(dt), v[None], "NHD", mean, scale)
        extra = dict(k_scale=torch.zeros(pages, hkv, page, device="cuda"),
                     k_mean=mean.view(hkv, 64), v_scale=scale.view(hkv, 64))
    cache = sage.PagedCache(kp, vp, "NHD", **extra)
    table = torch.randperm(pages, device="cuda").int()[None, :10].contiguous()
    ws = sage.alloc_workspace_paged()
    outs, at = [], 0
    for n in [70, 65] + [1] * 15:
        lens = torch.tensor([at + n], dtype=torch.int32, device="cuda")
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        batch = sage.PagedBatch(cu, lens, table, n, total)
        part = slice(at, at + n)
        qo = sage.kv_append(cache, batch, k[part], v[part], q=q[part], inv_freq=f, ws=ws)
        outs.append(sage.attn_paged(cache, batch, qo, window=window, sinks=sinks, ws=ws))
        at += n
    assert sage.device_status(ws) == sage.OK
    out = torch.cat(outs).double()
    see = pos[None] <= pos[:, None]
    if window:
        see &= (pos[None] > pos[:, None] - window) | (pos[None] < sinks)
    u = HALF[dt]
    for h in range(hq):
        x = (qr[:, h] @ kr[:, h // 4].T) * d ** -0.5
        w = torch.softmax(x.masked_fill(~see, float("-inf")), -1)
        vh = v[:, h // 4].double()
        ref, mean_v = w @ vh, w @ vh.abs()
        # q and k are rounded once each after the rotation, which moves a logit by at most
        # e = 2 u sum|q k| / sqrt(d) and a weight by 2 e; the 8-bit cache's keys by half a
        # code, sum|q| s / 2 (K's smoothed codes), and its values by 2^-4 of themselves, or
        # half a step of e4m3's smallest, 2^-10 of the scale
        e = 2 * u * (qr[:, h].abs() @ kr[:, h // 4].abs().T).amax(-1, keepdim=True) * d ** -0.5
        tail = 0.0
        if kind == "q8":
            top = (kr[:, h // 4] - extra["k_mean"][h // 4].double()).abs().amax(-1)
            e = e + (qr[:, h].abs().sum(-1, keepdim=True) * top[None] / 254 * d ** -0.5).amax(
                -1, keepdim=True)
            tail = 2.0 ** -4 * mean_v + 2.0 ** -10 * extra["v_scale"][h // 4].double()
        bound = u * ref.abs() + (u + 2 * e) * mean_v * (1 + 2 * e) + tail * (1 + 2 * e) + 1e-6
        assert ((out[:, h] - ref).abs() <= bound).all()


def test_append_and_attention_replay_in_a_graph(sage):
    """A captured decoding step: the lengths advance on the device."""
    p = Problem([1, 1], [100, 30], 8, 2, 64, 16, "NHD", "bf16", seed=50, poison=False, max_kv=112)
    # room for ten more tokens
    free = [x for x in range(p.k.shape[0]) if x not in set(p.table[:, :7].flatten().tolist())]
    p.table[1, 2] = free[0]
    k, v, q = (torch.empty(2, h, 64, dtype=torch.bfloat16, device="cuda") for h in (2, 2, 8))
    cache, batch = p.sage(sage)
    ws = sage.alloc_workspace_paged()
    f, _ = sage.rope_freqs(64)

    def step():
        qo = sage.kv_append(cache, batch, k, v, q=q, inv_freq=f, ws=ws)
        return sage.attn_paged(cache, batch, qo, ws=ws)

    def fill(i):
        for x, s in ((k, 60), (v, 70), (q, 80)):
            x.copy_(randn(s + i, *x.shape))

    start_k, start_v, start_l = p.k.clone(), p.v.clone(), p.lens.clone()
    fill(0)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    p.k.copy_(start_k), p.v.copy_(start_v)
    got = []
    for i in range(10):
        p.lens.copy_(start_l + i)
        fill(i)
        graph.replay()
        got.append(out.clone())
    end_k = p.k.clone()
    p.k.copy_(start_k), p.v.copy_(start_v)
    for i in range(10):
        p.lens.copy_(start_l + i)
        fill(i)
        assert torch.equal(step(), got[i])
    assert torch.equal(p.k, end_k) and sage.device_status(ws) == sage.OK
