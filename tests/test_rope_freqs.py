"""Every frequency of the scaled forms, against forms that go pair by pair."""
import math

import pytest

torch = pytest.importorskip("torch")
from quantized_attention_smooth_gb300 import sage  # noqa: E402

CASES = [(128, 10000.0, 4096, 8.0, 1.0, 32.0), (64, 500000.0, 8192, 4.0, 1.0, 4.0),
         (128, 1e6, 32768, 4.0, 1.0, 32.0), (96, 10000.0, 2048, 16.0, 2.0, 20.0),
         (16, 500.0, 100, 2.0, 1.0, 32.0), (128, 10000.0, 10 ** 7, 3.0, 1.0, 32.0),
         (2, 10000.0, 4096, 8.0, 1.0, 32.0)]


def pairs(r, base, length):
    """Each pair's frequency, and the turns it makes in `length` positions."""
    f = [base ** (-2.0 * i / r) for i in range(r // 2)]
    return f, [length * x / (2 * math.pi) for x in f]


def same(got, want):
    assert got.dtype == torch.float64 and got.shape == (len(want),)
    assert all(abs(a - b) <= 1e-13 * b for a, b in zip(got.tolist(), want)), (got.tolist(), want)


@pytest.mark.parametrize("r,base,length,factor,low,high", CASES)
def test_by_parts_ramps_in_the_turns(r, base, length, factor, low, high):
    f, turns = pairs(r, base, length)
    want = []
    for x, n in zip(f, turns):
        keep = 1.0 if n > high else 0.0 if n < low else (n - low) / (high - low)
        want.append(keep * x + (1 - keep) * x / factor)
    got, gain = sage.rope_freqs(r, base, "by_parts", factor, length, low, high, device="cpu")
    same(got, want)
    assert gain == 1.0


@pytest.mark.parametrize("r,base,length,factor,low,high", CASES)
def test_yarn_ramps_in_the_pairs_index(r, base, length, factor, low, high):
    """The ramp's ends found by counting: the last pair (as the index goes on past
    the head's own) that still turns `high` times, and the first that turns no
    more than `low` times."""
    f, _ = pairs(r, base, length)
    at = [length * base ** (-2.0 * i / r) / (2 * math.pi) for i in range(r)]
    first = max([i for i in range(r) if at[i] >= high], default=0)
    last = min([i for i in range(r) if at[i] <= low], default=r - 1)
    want = []
    for i, x in enumerate(f):
        away = 0.0 if i <= first else 1.0 if i >= last else (i - first) / (last - first)
        want.append((1 - away) * x + away * x / factor)
    got, gain = sage.rope_freqs(r, base, "yarn", factor, length, low, high, device="cpu")
    same(got, want)
    assert abs(gain - (0.1 * math.log(factor) + 1.0)) < 1e-15


def test_yarn_refuses_a_ramp_without_ends():
    for kw in (dict(low=0.0), dict(high=0.5), dict(base=1.0), dict(original_len=0)):
        with pytest.raises(ValueError, match="yarn"):
            sage.rope_freqs(64, scaling="yarn", factor=2.0, device="cpu", **kw)
