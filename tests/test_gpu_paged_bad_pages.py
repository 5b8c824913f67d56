"""Table entries outside the cache: each is reported, none is followed, and all of them read the
same zeros, whatever number they are."""
import pytest

torch = pytest.importorskip("torch")
from tests.paged_ref import Problem  # noqa: E402
from tests.q4_ref import Problem4  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sage():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_attention_smooth_gb300 import sage
    return sage


@pytest.mark.parametrize("kind", ["q4", "q8", "bf16"])
@pytest.mark.parametrize("q_len", [1, 5, 150])
def test_every_entry_outside_is_reported(sage, kind, q_len):
    make = dict(seed=12, poison=False)
    p = (Problem4([q_len, q_len], [200, 200], 4, 2, 64, 16, **make) if kind == "q4" else
         Problem([q_len, q_len], [200, 200], 4, 2, 64, 16, "NHD", kind, **make))
    ws = sage.alloc_workspace_paged()
    good = sage.attn_paged(*p.sage(sage), p.q, ws=ws)
    assert sage.device_status(ws) == sage.OK
    outs = []
    for bad in (-1, -2, -3, -2 ** 31, p.k.shape[0], 2 ** 31 - 1):
        p.table[1, 3] = bad
        ws = sage.alloc_workspace_paged()
        outs.append(sage.attn_paged(*p.sage(sage), p.q, ws=ws))
        assert sage.device_status(ws) == sage.ERR_INVALID_ARG, bad
        assert "block table" in sage.last_error()
        assert torch.equal(outs[-1][:q_len], good[:q_len]) and torch.isfinite(outs[-1]).all()
        assert torch.equal(outs[-1], outs[0])
    assert not torch.equal(outs[0], good)
