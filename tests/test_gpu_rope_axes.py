"""Rotary positions of several axes, alone and in the cache append, against 64 bits."""
import pytest

torch = pytest.importorskip("torch")
from tests.paged_ref import Problem  # noqa: E402
from tests.q4_ref import Problem4  # noqa: E402
from tests.test_gpu_rows import magnitude, near, places, randn, slot_view  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sage():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_attention_smooth_gb300 import sage
    return sage


def turn(x, pos, axes, f, interleaved=False, gain=1.0, sign=1.0):
    """x (T, H, D) with pair i turned by pos[axes[i]] f[i], in 64 bits."""
    x = x.double().clone()
    r = 2 * f.numel()
    a = (pos.double()[axes.long()] * f[:, None] * sign).T[:, None]
    c, s = a.cos() * gain, a.sin() * gain
    i, j = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    x1, x2 = x[..., i].clone(), x[..., j].clone()
    x[..., i], x[..., j] = x1 * c - x2 * s, x2 * c + x1 * s
    return x


def positions(t, axes, seed=1, far=50000):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-20, far, (axes, t), generator=g, device="cuda")


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,sections,in_turn", [(128, (16, 24, 24), False), (128, (24, 20, 20), True),
                                                (64, (8, 8), False), (80, (10, 10, 10, 10), True),
                                                (40, (3, 7), False), (128, (1,), False),
                                                (72, (0, 20, 4), False), (33, (5, 5, 6), True)])
@pytest.mark.parametrize("t", [1, 7, 700])
def test_rope(sage, dt, interleaved, d, sections, in_turn, t):
    q, k = randn(1, t, 5, d, dt=dt), randn(2, t, 2, d, dt=dt)
    r = 2 * sum(sections)
    pos, axes = positions(t, len(sections)), sage.rope_axes(sections, in_turn)
    assert [int((axes == a).sum()) for a in range(len(sections))] == list(sections)
    f, gain = sage.rope_freqs(r, scaling="yarn", factor=4.0)
    qo, ko = sage.rope(q, k, pos, f, interleaved, gain, axes=axes)
    for x, y in ((q, qo), (k, ko)):
        near(y, turn(x, pos, axes, f, interleaved, gain), magnitude(x, r, interleaved, gain))
        assert torch.equal(y[..., r:], x[..., r:])
    # int32 positions out of wider rows, and in place
    wide = torch.zeros(len(sections), t + 9, dtype=torch.int32, device="cuda")
    wide[:, 4:4 + t] = pos
    qi, ki = q.clone(), k.clone()
    sage.rope(qi, ki, wide[:, 4:4 + t], f, interleaved, gain, q_out=qi, k_out=ki, axes=axes)
    assert torch.equal(qi, qo) and torch.equal(ki, ko)
    # equal positions on every axis are those of one axis, to the bit
    one = pos[:1].expand(len(sections), t).contiguous()
    a = sage.rope(q, k, one, f, interleaved, gain, axes=axes)
    b = sage.rope(q, k, pos[0].contiguous(), f, interleaved, gain)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("t", [3, 900])
def test_inverse_is_the_gradient(sage, t):
    """<R x, g> = <x, R' g>, and differences along single channels agree with it."""
    x, g = randn(6, t, 3, 32, dt=torch.float16), randn(7, t, 3, 32, dt=torch.float16)
    pos, axes = positions(t, 3), sage.rope_axes((4, 5, 3))
    f, gain = sage.rope_freqs(24, scaling="yarn", factor=2.0)
    for inter in (False, True):
        grad, _ = sage.rope(g, None, pos, f, inter, gain, inverse=True, axes=axes)
        ref = turn(g, pos, axes, f, inter, gain, sign=-1.0)
        near(grad, ref, magnitude(g, 24, inter, gain))
        lhs = (turn(x, pos, axes, f, inter, gain) * g.double()).sum()
        rhs = (x.double() * ref).sum()
        assert abs(float(lhs - rhs)) <= 1e-9 * float(x.double().abs().sum())
        for ch in (0, 5, 13, 23, 24, 31):                # linear: a difference of any size is exact
            e = torch.zeros_like(x)
            e[1, 1, ch] = 1.0
            moved, _ = sage.rope(e, None, pos, f, inter, gain, axes=axes)
            slope = float((moved.double() * g.double()).sum())
            # two fp16 roundings of the moved pair (2^-11 each times |g| <= 4), one of grad
            assert abs(slope - float(grad[1, 1, ch])) <= 2.0 ** -11 * 4 * 3 * gain


def test_frequencies_by_the_axis_and_far_positions(sage):
    axes = sage.rope_axes((4, 6, 6))
    f = torch.cat([100.0 ** (-torch.arange(n, device="cuda", dtype=torch.float64) / n) for n in (4, 6, 6)])
    q = randn(8, 6, 2, 32, dt=torch.float16)
    pos = torch.tensor([[0, 1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, 5], [9, 0, 1, 2, 3, -4],
                        [0, 0, 0, 2 ** 20, 1, 10 ** 6]], device="cuda")
    got, _ = sage.rope(q, None, pos, f, axes=axes)
    near(got, turn(q, pos, axes, f), magnitude(q, 32, False))


def test_an_axis_beyond_the_last_takes_the_last(sage):
    q, pos = randn(9, 40, 2, 64), positions(40, 2)
    f, _ = sage.rope_freqs(64)
    axes = sage.rope_axes((10, 22))
    over = torch.where(axes == 1, 200, 0).to(torch.uint8)
    assert torch.equal(sage.rope(q, None, pos, f, axes=over)[0], sage.rope(q, None, pos, f, axes=axes)[0])


@pytest.mark.parametrize("kind", ["bf16", "q8", "q4"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1, 1], [1, 16, 333]), ([3, 0, 50, 7], [3, 9, 200, 4]),
                                            ([700, 1, 300], [710, 50, 333]),
                                            ([7000, 1, 900], [7010, 50, 950])])
def test_append(sage, kind, interleaved, q_lens, kv_lens):
    """The append at given positions stores what the rotation alone gives, and turns q alike."""
    dt, hkv, d = torch.bfloat16, 2, 128
    make = (lambda: Problem4(q_lens, kv_lens, 4, hkv, d, 16, "NHD", dt, seed=30, poison=False,
                             spare_rows=2)) if kind == "q4" else (
        lambda: Problem(q_lens, kv_lens, 4, hkv, d, 16, "NHD", kind, dt, seed=30, poison=False,
                        spare_rows=2))
    p = make()
    k, v = randn(31, p.q.shape[0], hkv, d, dt=dt), randn(32, p.q.shape[0], hkv, d, dt=dt)
    pos, axes = positions(p.q.shape[0], 3), sage.rope_axes((16, 24, 24))
    f, gain = sage.rope_freqs(d)
    ws = sage.alloc_workspace_paged()
    rows, pages, slots, _ = places(p)
    q_out = torch.full_like(p.q, 7.0)
    sage.kv_append(*p.sage(sage), k, v, q=p.q, q_out=q_out, inv_freq=f, interleaved=interleaved,
                   mscale=gain, positions=pos, axes=axes, ws=ws)
    assert sage.device_status(ws) == sage.OK
    qr, kr = sage.rope(p.q, k, pos, f, interleaved, gain, axes=axes)
    assert torch.equal(q_out[rows], qr[rows]) and (q_out[sum(q_lens):] == 7.0).all()
    if kind == "bf16":
        assert torch.equal(slot_view(p, p.k)[pages, slots], kr[rows])
        assert torch.equal(slot_view(p, p.v)[pages, slots], v[rows])
        return
    back, _ = sage.kv_gather(*p.sage(sage), p.q.shape[0], dt)
    x = turn(k[rows], pos[:, rows], axes, f, interleaved, gain)
    top = (x - p.k_mean[:, :d].double()).abs().amax(-1, keepdim=True)
    # half a code of 127 or 7 to a side, and bf16's rounding of what comes back
    half = top / (254 if kind == "q8" else 14) * 1.01
    assert ((back[rows].double() - x).abs() <= half + 2.0 ** -8 * x.abs() + 2.0 ** -6).all()


def test_append_at_one_axis(sage):
    """Positions without axes: given ones in the place of the cache's."""
    p = Problem([5, 3], [5, 30], 2, 2, 64, 16, poison=False)
    k, v = randn(33, 8, 2, 64), randn(34, 8, 2, 64)
    f, _ = sage.rope_freqs(64)
    pos = positions(8, 1)[0]
    sage.kv_append(*p.sage(sage), k, v, inv_freq=f, positions=pos)
    rows, pages, slots, _ = places(p)
    assert torch.equal(p.k[pages, slots], sage.rope(k, None, pos, f)[0][rows])


def test_what_the_binding_refuses(sage):
    q, pos = randn(8, 3, 2, 64), positions(3, 2)
    f, _ = sage.rope_freqs(64)
    axes = sage.rope_axes((16, 16))
    for kw, match in [(dict(positions=pos[:, :2]), "positions"), (dict(positions=pos.float()), "positions"),
                      (dict(positions=pos.T.contiguous().T), "positions"),
                      (dict(positions=positions(3, 9)), "positions"),
                      (dict(positions=pos.cpu()), "positions is not on"),
                      (dict(axes=axes[:5]), "axes"), (dict(axes=axes.int()), "axes"),
                      (dict(axes=axes.cpu()), "axes is not on")]:
        with pytest.raises((ValueError, TypeError), match=match):
            sage.rope(q, None, **{**dict(positions=pos, inv_freq=f, axes=axes), **kw})
    p = Problem([3], [3], 2, 2, 64, 16, poison=False)
    args = p.sage(sage) + (q, q)
    for kw, match in [(dict(positions=pos), "without inv_freq"), (dict(positions=pos, inv_freq=f), "need `axes`"),
                      (dict(inv_freq=f, axes=axes), "without positions")]:
        with pytest.raises(ValueError, match=match):
            sage.kv_append(*args, **kw)
    for bad in ((), (65,), (-1, 3), (1,) * 9, (0, 0)):
        with pytest.raises(ValueError, match="sections"):
            sage.rope_axes(bad)
