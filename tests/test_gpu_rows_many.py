"""Rotations and appends of thousands of tokens: the kernels for many rows, and CTAs whose tokens
are no power of two (whole waves of CTAs)."""
import pytest

torch = pytest.importorskip("torch")
from tests import test_gpu_rows as rows  # noqa: E402
from tests.paged_ref import Problem, turn  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sage():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_attention_smooth_gb300 import sage
    return sage


MANY = ([7000, 0, 1, 999], [7100, 0, 5, 900])
SHAPES = [(128, 2, 16, "NHD", False), (80, 3, 32, "HND", True), (40, 1, 48, "HND", False)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,r", [(128, 128), (64, 16), (40, 20)])
@pytest.mark.parametrize("t", [761, 3649, 9121, 29185])
def test_rope(sage, interleaved, d, r, t):
    rows.test_rope(sage, torch.bfloat16, interleaved, d, r, t)


@pytest.mark.parametrize("d,hkv,page,layout,both", SHAPES)
@pytest.mark.parametrize("r,interleaved", [(0, False), (-1, False), (-1, True)])
def test_append_16bit(sage, monkeypatch, d, hkv, page, layout, both, r, interleaved):
    monkeypatch.setattr(rows, "CASES", [MANY])
    rows.test_append_16bit(sage, torch.float16, d, hkv, page, layout, both, r, interleaved, 0)


@pytest.mark.parametrize("d,hkv,page,layout,both", SHAPES)
@pytest.mark.parametrize("r", [0, -1])
def test_append_q8(sage, monkeypatch, d, hkv, page, layout, both, r):
    monkeypatch.setattr(rows, "CASES", [MANY])
    rows.test_append_q8(sage, torch.bfloat16, d, hkv, page, layout, both, r, 0)


@pytest.mark.parametrize("n", [[900, 1, 300], [7000, 1, 900]])
def test_append_q8_interleaved(sage, n):
    """Both kernels, neighbouring pairs: the bound of the half layout's test."""
    p = Problem(n, [m + 11 for m in n], 2, 2, 128, 16, "NHD", "q8", torch.bfloat16, seed=61,
                poison=False, offset=3.0)
    k, v = rows.randn(62, sum(n), 2, 128), rows.randn(63, sum(n), 2, 128)
    cache, batch = p.sage(sage)
    at, pages, slots, pos = rows.places(p)
    f, gain = sage.rope_freqs(128)
    q = sage.kv_append(cache, batch, k, v, q=p.q, inv_freq=f, interleaved=True, mscale=gain)
    assert torch.equal(q[at], sage.rope(p.q[at], None, pos, f, True, gain)[0])
    x = turn(k[at], pos, f, True, gain) - p.k_mean.double()
    top = x.abs().amax(-1)
    err = (2.0 ** -20 * rows.magnitude(k[at], 128, True, gain) + 2.0 ** -24 * x.abs()).amax(-1)
    codes, s = rows.slot_view(p, p.k)[pages, slots], p.k_scale[pages, :, slots].double()
    assert ((s - top / 127).abs() <= (err + 2.0 ** -23 * top) / 127 + 1e-38).all()
    bound = (s * 0.5 * (1 + 2.0 ** -15) + 2 * err)[..., None] + 1e-30
    assert ((codes.double() * s[..., None] - x).abs() <= bound).all()
