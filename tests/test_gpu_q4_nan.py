"""What the 4-bit cache makes of NaN and infinities: a group that holds a NaN reads back as NaN, an
infinity saturates, and every other group keeps its codes and scale to the bit."""
import pytest

torch = pytest.importorskip("torch")
from tests.q4_ref import GROUP, Problem4, unpack  # noqa: E402
from tests.test_gpu_rows import places, randn, slot_view  # noqa: E402

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def sage():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_attention_smooth_gb300 import sage
    return sage


# the second and third: the kernel for many tokens (from 48 tokens per SM on)
@pytest.mark.parametrize("n", [40, 7901, 9000])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,hkv,page,layout", [(128, 2, 16, "NHD"), (72, 3, 32, "HND"), (64, 1, 64, "NHD")])
@pytest.mark.parametrize("turned", [None, False, True])      # no rotation, half layout, neighbours
def test_append_and_gather(sage, n, dt, d, hkv, page, layout, turned):
    p = Problem4([n], [n + 7], hkv, hkv, d, page, layout, dt, seed=n, poison=False, offset=1.0)
    p.v_scale *= 100                                         # finite values are far below saturation
    k, v = randn(1, n, hkv, d, dt=dt), randn(2, n, hkv, d, dt=dt)
    cache, batch = p.sage(sage)
    _, pages, slots, _ = places(p)
    kw = {}
    if turned is not None:
        kw = dict(inv_freq=sage.rope_freqs(d - d % 16)[0], interleaved=turned)

    def stored():
        sage.kv_append(cache, batch, k, v, **kw)
        back = sage.kv_gather(cache, batch, n, dt)
        return [(unpack(slot_view(p, x)[pages, slots]).unflatten(-1, (-1, GROUP)).clone(),
                 g[pages, :, slots][..., :p.groups].clone(), y)
                for x, g, y in ((p.k, p.k_groups, back[0]), (p.v, p.v_groups, back[1]))]

    clean = stored()
    r = d - d % 16
    spots = [(0, 0, 1, NAN), (1, hkv - 1, d - 1, INF), (n // 2, 0, r // 2, -INF), (n - 3, hkv - 1, 7, NAN),
             (n - 2, 0, r // 2 + 1, INF), (n - 1, hkv - 1, d - 1, NAN)]
    for t, h, c, x in spots:
        k[t, h, c] = v[t, h, c] = x
    got = stored()
    for which, (codes, scales, back), (codes0, scales0, back0) in zip("kv", got, clean):
        touched = torch.zeros_like(scales, dtype=torch.bool)
        for t, h, c, x in spots:
            channels = {c}
            if which == "k" and turned is not None and c < r:
                channels.add(c ^ 1 if turned else (c + r // 2) % r)
            for group in {c // GROUP for c in channels}:
                touched[t, h, group] = True
                s, n8 = scales[t, h, group], codes[t, h, group]
                mine = back[t, h, group * GROUP:(group + 1) * GROUP]
                if x != x:
                    assert torch.isnan(s) and (n8 == 0).all() and torch.isnan(mine).all()
                    continue
                assert float(s) == (9352.0 if which == "k" else 1.0)
                inside = [c % GROUP for c in channels if c // GROUP == group]
                want = torch.zeros_like(n8)
                want[inside] = 7
                assert torch.equal(n8.abs(), want) and torch.isfinite(mine).all()
                if which == "v" or turned is None:
                    assert int(n8[c % GROUP]) == (7 if x > 0 else -7)
        assert torch.equal(codes[~touched], codes0[~touched])
        assert torch.equal(scales[~touched].view(torch.int16), scales0[~touched].view(torch.int16))
        wide = touched.repeat_interleave(GROUP, -1)[..., :d]
        assert torch.equal(back[~wide], back0[~wide])
