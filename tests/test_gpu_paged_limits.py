"""Attention over the paged cache at the ends of its ranges."""
import pytest

torch = pytest.importorskip("torch")
from tests.paged_ref import Problem  # noqa: E402
from tests.test_gpu_paged import check, sage  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def test_declared_bounds_near_2_31(sage):  # noqa: F811
    """Bounds say what may come; 1024 sequences of a few keys each."""
    n = 1024
    p = Problem([1 + i % 2 * 20 for i in range(n)], [21 + i % 9 for i in range(n)], 2, 2, 8, 65536,
                "NHD", "bf16", seed=72, poison=False, pool=n)
    table = torch.full((n, 32768), -1, dtype=torch.int32, device="cuda")
    table[:, :1] = p.table[:, :1]
    p.table, p.max_q, p.max_kv = table, 2 ** 30 - 1, 2 ** 31 - 1
    check(sage, p)
