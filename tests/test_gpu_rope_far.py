"""Rotations at far positions, against angles reduced in whole numbers."""
import math
from fractions import Fraction

import pytest

torch = pytest.importorskip("torch")
from tests.paged_ref import HALF  # noqa: E402
from tests.test_gpu_rows import magnitude, randn, sage  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_far_positions_within_the_stated_bound(sage, interleaved):  # noqa: F811
    """The phase is off by |pos| (f 2^-52 + 2^-62) rad: 1 / (2 pi) and the product with
    it are rounded once each (2^-53 of the turns, f pos / 2 pi), the turn's
    fraction to 2^-65 (2 pi 2^-65 < 2^-62 rad).  A phase error e moves a channel by e
    (|x1| + |x2|); the angle here is exact in integers, so the reference is too."""
    pos = torch.tensor([2 ** 40 + 3, -2 ** 40 - 1, 2 ** 33 + 12345, 2 ** 46 + 7, 2 ** 28 + 1],
                       device="cuda")
    f = torch.tensor([1.0, 0.37, 1e-4, 100.25, 2.0 ** -20, 6.5], dtype=torch.float64)
    # pi to 2^-240: 100 terms of the Machin series in whole numbers
    one = 1 << 260

    def arctan(n):
        s = t = one // n
        i = 1
        while t:
            t //= n * n
            i += 2
            s += -t // i if i % 4 == 3 else t // i
        return s
    two_pi = Fraction(8 * (4 * arctan(5) - arctan(239)), one)
    angle = torch.tensor([[float(Fraction(int(a)) * Fraction(float(b)) % two_pi) for b in f]
                          for a in pos], dtype=torch.float64, device="cuda")
    assert abs(float(two_pi) - 2 * math.pi) < 1e-15
    q = randn(85, 5, 2, 16, dt=torch.float16)
    got, _ = sage.rope(q, None, pos, f.cuda(), interleaved)
    i, j = (slice(0, 12, 2), slice(1, 12, 2)) if interleaved else (slice(0, 6), slice(6, 12))
    ref = q.double().clone()
    x1, x2, c, s = ref[..., i].clone(), ref[..., j].clone(), angle.cos()[:, None], angle.sin()[:, None]
    ref[..., i], ref[..., j] = x1 * c - x2 * s, x2 * c + x1 * s
    phase = torch.zeros_like(ref)
    e = (pos.double().abs()[:, None] * (f.cuda() * 2.0 ** -52 + 2.0 ** -62))[:, None].expand(5, 2, 6)
    phase[..., i] = phase[..., j] = e
    bound = HALF[torch.float16] * ref.abs() + (2.0 ** -20 + phase) * magnitude(q, 12, interleaved) \
        + 2.0 ** -25
    assert ((got.double() - ref).abs() <= bound).all()
