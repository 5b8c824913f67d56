"""The 8-bit cache's writer in the forms of its rotation: both pairings, a part of the
head, q beside it, few tokens and many (two kernels)."""
import pytest

torch = pytest.importorskip("torch")
from tests.paged_ref import Problem, turn  # noqa: E402
from tests.test_gpu_rows import magnitude, places, randn, sage, slot_view  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,r", [(128, 128), (128, 32), (80, 16), (80, 80), (64, 64), (72, 32),
                                 (104, 24), (40, 16)])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 3, 0, 50], [9, 3, 0, 200]),
                                            ([1200, 1, 700], [1300, 5, 700])])
def test_append_q8_with_rotation(sage, dt, interleaved, d, r, q_lens, kv_lens):  # noqa: F811
    """q_out has the bits of the stand-alone rotation; a code is off by half a step
    and the rotation's fp32 error, as in the writer's other tests; nothing else in
    the cache moves."""
    hkv = 3
    p = Problem(q_lens, kv_lens, 2 * hkv, hkv, d, 32, "NHD", "q8", dt, seed=80, poison=False,
                offset=3.0, spare_rows=2)
    k, v = randn(81, p.q.shape[0], hkv, d, dt=dt), randn(82, p.q.shape[0], hkv, d, dt=dt)
    bk, bv, bs = p.k.clone(), p.v.view(torch.uint8).clone(), p.k_scale.clone()
    f, gain = sage.rope_freqs(r, scaling="by_parts", factor=3.0)
    gain = 1.25
    q_out = torch.full_like(p.q, 7.0)
    ws = sage.alloc_workspace_paged()
    got = sage.kv_append(*p.sage(sage), k, v, q=p.q, q_out=q_out, inv_freq=f,
                         interleaved=interleaved, mscale=gain, ws=ws)
    assert got is q_out and sage.device_status(ws) == sage.OK, sage.last_error()
    rows, pages, slots, pos = places(p)
    qr, _ = sage.rope(p.q[rows], None, pos, f, interleaved, gain)
    assert torch.equal(q_out[rows], qr) and (q_out[sum(q_lens):] == 7.0).all()
    inv = torch.where(p.v_scale > 0, p.v_scale.reciprocal(), 0.0)[:, :d]
    want_v = (v[rows].float() * inv).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    slot_view(p, bv)[pages, slots] = want_v
    assert torch.equal(p.v.view(torch.uint8), bv)
    got_k, got_s = slot_view(p, p.k)[pages, slots], p.k_scale[pages, :, slots]
    x = turn(k[rows], pos, f, interleaved, gain) - p.k_mean[:, :d].double()
    top = x.abs().amax(-1)
    err = (2.0 ** -20 * magnitude(k[rows], r, interleaved, gain) + 2.0 ** -24 * x.abs()).amax(-1)
    assert ((got_s.double() - top / 127).abs() <= (err + 2.0 ** -23 * top) / 127 + 1e-38).all()
    back = got_k.double() * got_s.double()[..., None]
    assert ((back - x).abs() <= (got_s.double() * 0.5 * (1 + 2.0 ** -15) + 2 * err)[..., None]).all()
    slot_view(p, bk)[pages, slots] = got_k
    bs[pages, :, slots] = got_s
    assert torch.equal(p.k, bk) and torch.equal(p.k_scale, bs)


@pytest.mark.parametrize("interleaved", [False, True])
def test_few_and_many_tokens_give_the_same_codes(sage, interleaved):  # noqa: F811
    """The kernels for few and for many tokens: one call of 1500 tokens, and calls of 100."""
    n, hkv, d = 1500, 2, 96
    two = [Problem([n], [n], 4, hkv, d, 16, "HND", "q8", torch.bfloat16, seed=83, poison=False)
           for _ in range(2)]
    k, v, q = (randn(84 + i, n, h, d) for i, h in enumerate((hkv, hkv, 4)))
    f, gain = sage.rope_freqs(64, scaling="linear", factor=2.0)
    turn_args = dict(inv_freq=f, interleaved=interleaved, mscale=gain)
    qa = sage.kv_append(*two[0].sage(sage), k, v, q=q, **turn_args)
    cache, _ = two[1].sage(sage)
    qb = torch.empty_like(q)
    for a in range(0, n, 100):
        batch = sage.PagedBatch(torch.tensor([0, 100], dtype=torch.int32, device="cuda"),
                                torch.tensor([a + 100], dtype=torch.int32, device="cuda"),
                                two[1].table, 100, n)
        part = slice(a, a + 100)
        sage.kv_append(cache, batch, k[part], v[part], q=q[part], q_out=qb[part], **turn_args)
    assert torch.equal(qa, qb)
    assert torch.equal(two[0].k, two[1].k) and torch.equal(two[0].k_scale, two[1].k_scale)
    assert torch.equal(two[0].v.view(torch.uint8), two[1].v.view(torch.uint8))
