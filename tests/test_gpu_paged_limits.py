"""Attention over the paged cache at the ends of its ranges: weights far below the
largest one, scales near zero, declared bounds near 2^31."""
import pytest

torch = pytest.importorskip("torch")
from tests.paged_ref import HALF, Problem  # noqa: E402
from tests.test_gpu_paged import check, sage  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,dt", [("f16", torch.float16), ("q8", torch.float16),
                                     ("q8", torch.bfloat16), ("bf16", torch.bfloat16)])
@pytest.mark.parametrize("n,sequences", [(1, 700), (5, 700), (20, 160)])
@pytest.mark.parametrize("first", [0, 1500])
def test_many_small_weights_beside_a_large_one(sage, kind, dt, n, sequences, first):  # noqa: F811
    """In every sequence one key of weight 1 and 3999 of 2^-26, whose values alone make
    up the output; enough sequences that a CTA keeps one for itself.  Of
    Problem.tolerance only the term of fp16's smallest steps differs: the reference
    that P is taken against lies at least 2^7 below the row's largest weight, so
    that a weight w (the largest being 1) stands as w 2^7 or more in steps of 2^-24
    and is off by 2^-25 / 2^7 = 2^-32 at most."""
    total, d = 4000, 64
    p = Problem([n] * sequences, [total] * sequences, 2, 1, d, 16, "NHD", kind, dt, seed=70,
                poison=False)
    page, slot = p.table[:, first // 16].long(), first % 16
    p.k.zero_()
    p.q.zero_()
    p.q[..., 0] = 12.0
    if kind == "q8":
        p.k[page, slot, 0, 0] = 127
        p.k_scale.fill_(12.0 / 127.0)
        p.v_scale.fill_(1.0)
    else:
        p.k[page, slot, 0, 0] = 12.0
    ones = torch.ones(p.v.shape, device="cuda")
    ones[page, slot] = 0.0
    p.v = ones.to(p.v.dtype)
    out = sage.attn_paged(*p.sage(sage), p.q)
    ref, _, mean, spread = p.reference()
    u, up = HALF[dt], HALF[torch.bfloat16 if kind == "bf16" else torch.float16]
    step = 2.0 ** -25 if dt == torch.float16 else 0.0
    low = 0.0 if kind == "bf16" else 2.0 ** -32
    bound = u * ref.abs() + (up + 3 * 2.0 ** -16) * mean * (1 + u) + low * spread + step
    diff = (out.double() - ref).abs()
    assert float(ref.min()) > 4e-5
    assert (diff <= bound).all(), float((diff / bound).max())


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
