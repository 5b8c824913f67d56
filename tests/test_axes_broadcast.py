"""Positions that all axes share: axis stride 0."""
import pytest

from quantized_attention_smooth_gb300 import sage as lib
from tests.test_q4_refusals import append_axes, rope


def test_stride_0_is_not_refused():
    """The next check's refusal is what comes back (no GPU needed: validation comes first)."""
    for call in (rope, append_axes):
        assert call(step=0, R=74) == lib.ERR_INVALID_ARG and "even" in lib.last_error()
        for step in (1, 2, -1, -4, 1 << 39):
            assert call(step=step, R=74) == lib.ERR_INVALID_ARG and "axis_stride" in lib.last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("t", [1, 5, 900, 8000])
def test_expanded_positions(t):
    torch = pytest.importorskip("torch")
    from tests.paged_ref import Problem
    from tests.q4_ref import Problem4
    from tests.test_gpu_rows import randn
    q, k = randn(1, t, 4, 64), randn(2, t, 2, 64)
    one = torch.randint(0, 5000, (1, t), device="cuda")
    axes, (f, _) = lib.rope_axes((10, 11, 11)), lib.rope_freqs(64)
    for pos in (one.expand(3, t), one.int().expand(3, t)):
        want = lib.rope(q, k, pos.contiguous(), f, axes=axes)
        got = lib.rope(q, k, pos, f, axes=axes)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        # and these are the positions of one axis
        assert torch.equal(got[0], lib.rope(q, None, pos[0].contiguous(), f)[0])
    for make in (lambda: Problem([t], [t + 3], 4, 2, 64, 16, poison=False),
                 lambda: Problem4([t], [t + 3], 4, 2, 64, 16, poison=False)):
        a, b = make(), make()
        lib.kv_append(*a.sage(lib), k, k, inv_freq=f, positions=one.expand(3, t), axes=axes)
        lib.kv_append(*b.sage(lib), k, k, inv_freq=f, positions=one.expand(3, t).contiguous(), axes=axes)
        assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
