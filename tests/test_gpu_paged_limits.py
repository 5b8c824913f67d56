"""Attention over the paged cache at the ends of its ranges."""
import pytest

torch = pytest.importorskip("torch")
from tests.paged_ref import Problem  # noqa: E402
from tests.test_gpu_paged import check, sage  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,dt", [("bf16", torch.bfloat16), ("f16", torch.float16),
                                     ("q8", torch.bfloat16), ("q8", torch.float16)])
@pytest.mark.parametrize("n", [1, 5, 200])
@pytest.mark.parametrize("scale", [1e-8, 1e-30])
def test_scale_near_zero_and_rows_of_zeros(sage, kind, dt, n, scale):  # noqa: F811
    """All logits are next to zero, among them those of rows without a number in them."""
    p = Problem([n, 40], [300, 40], 4, 2, 64, 16, "NHD", kind, dt, seed=71)
    p.q[::2] = 0.0
    p.q[1::4] = (p.q[1::4].float() * 1e-7).to(dt)
    check(sage, p, scale)


def test_declared_bounds_near_2_31(sage):  # noqa: F811
    """Bounds say what may come; 1024 sequences of a few keys each."""
    n = 1024
    p = Problem([1 + i % 2 * 20 for i in range(n)], [21 + i % 9 for i in range(n)], 2, 2, 8, 65536,
                "NHD", "bf16", seed=72, poison=False, pool=n)
    table = torch.full((n, 32768), -1, dtype=torch.int32, device="cuda")
    table[:, :1] = p.table[:, :1]
    p.table, p.max_q, p.max_kv = table, 2 ** 30 - 1, 2 ** 31 - 1
    check(sage, p)
