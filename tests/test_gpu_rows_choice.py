"""Rotations and appends of many tokens at once, against the same tokens a few at a time: the kernels
for many and for few tokens write the same bits, whatever the heads and lengths that choose them."""
import pytest

torch = pytest.importorskip("torch")
from tests.paged_ref import Problem  # noqa: E402
from tests.q4_ref import Problem4  # noqa: E402
from tests.test_gpu_rows import randn  # noqa: E402

pytestmark = pytest.mark.gpu
FEW = 250


@pytest.fixture(scope="module")
def sage():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_attention_smooth_gb300 import sage
    return sage


# either side of the choice for many heads and for one
SHAPES = [(32, 8, 128, 700), (32, 8, 128, 4700), (64, 8, 128, 2300), (8, 1, 64, 13000), (8, 1, 64, 30000),
          (16, 16, 80, 5000), (2, 1, 40, 45000), (0, 1, 128, 14000), (0, 2, 80, 26000)]
TURNS = [None, False, True]                          # as it is, half layout, neighbours


def turned(sage, d, how):
    r = d if d % 16 == 0 or how else d - d % 16      # (the half layout's kernel for many wants whole vectors)
    return {} if how is None else dict(inv_freq=sage.rope_freqs(r)[0], interleaved=how)


@pytest.mark.parametrize("hq,hkv,d,t", SHAPES)
@pytest.mark.parametrize("how", TURNS[1:])
def test_rope(sage, hq, hkv, d, t, how):
    q, k = randn(1, t, max(hq, 1), d), randn(2, t, hkv, d)
    pos = torch.arange(t, device="cuda") * 7 - 100
    kw = turned(sage, d, how)
    a = sage.rope(q, k, pos, **kw)
    for i in range(0, t, FEW):
        b = sage.rope(q[i:i + FEW], k[i:i + FEW], pos[i:i + FEW], **kw)
        assert all(torch.equal(x[i:i + FEW], y) for x, y in zip(a, b))


@pytest.mark.parametrize("kind", ["f16", "q8", "q4"])
@pytest.mark.parametrize("hq,hkv,d,t", SHAPES)
@pytest.mark.parametrize("how", TURNS)
def test_append(sage, kind, hq, hkv, d, t, how):
    dt = torch.float16
    make = lambda: (Problem4([t], [t], hkv, hkv, d, 16, "NHD", dt, seed=5, poison=False, offset=1.0)
                    if kind == "q4" else
                    Problem([t], [t], hkv, hkv, d, 16, "NHD", kind, dt, seed=5, poison=False, offset=1.0))
    whole, parts = make(), make()
    k, v, q = randn(3, t, hkv, d, dt=dt), randn(4, t, hkv, d, dt=dt), randn(5, t, max(hq, 1), d, dt=dt)
    kw, with_q = turned(sage, d, how), how is not None and hq > 0
    ws = sage.alloc_workspace_paged()
    a = sage.kv_append(*whole.sage(sage), k, v, q=q if with_q else None, ws=ws, **kw)
    for i in range(0, t, FEW):
        n = min(FEW, t - i)
        parts.cu.copy_(torch.tensor([0, n]))
        parts.lens.fill_(i + n)
        b = sage.kv_append(*parts.sage(sage), k[i:i + n], v[i:i + n], q=q[i:i + n] if with_q else None,
                           ws=ws, **kw)
        assert not with_q or torch.equal(a[i:i + n], b)
    assert sage.device_status(ws) == sage.OK, sage.last_error()
    raw = lambda x: x.contiguous().view(torch.uint8)
    for name in ("k", "v") + (("k_scale",) if kind == "q8" else ("k_groups", "v_groups") if kind == "q4" else ()):
        assert torch.equal(raw(getattr(whole, name)), raw(getattr(parts, name))), name
