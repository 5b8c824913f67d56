"""A NaN among a row's keys or values shows in its result, whichever kernel joins it."""
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
@pytest.mark.parametrize("q_len,kv_len,hkv,d", [
    (1, 40, 2, 64), (1, 40, 2, 128), (4, 900, 2, 64),    # an item on one CTA, or on several
    (1, 30000, 2, 128), (3, 30000, 2, 64),               # joined by the second launch
    (1, 9000, 16, 128),                                  # joined by a CTA
    (150, 400, 2, 64), (200, 30000, 2, 128),             # many rows
])
def test_a_nan_shows(sage, kind, q_len, kv_len, hkv, d):
    make = dict(seed=3, poison=False)
    p = (Problem4([q_len], [kv_len], 2 * hkv, hkv, d, 16, **make) if kind == "q4" else
         Problem([q_len], [kv_len], 2 * hkv, hkv, d, 16, "NHD", kind, **make))
    page, slot = int(p.table[0, 0]), 5                   # key 5, which every row sees
    ws = sage.alloc_workspace_paged()

    def run():
        lse = torch.zeros(p.q.shape[:2], device="cuda")
        out = sage.attn_paged(*p.sage(sage), p.q, lse=lse, ws=ws)
        assert sage.device_status(ws) == sage.OK
        return out, lse

    clean, lse0 = run()
    assert torch.isfinite(clean).all() and torch.isfinite(lse0).all()
    where = {"q4": lambda t, g: (g, (page, 0, slot, 0)), "q8": lambda t, g: (p.k_scale, (page, 0, slot)),
             "bf16": lambda t, g: (t, (page, slot, 0, 7))}[kind]
    t, at = where(p.k, getattr(p, "k_groups", None))
    keep = t[at].clone()
    t[at] = float("nan")
    out, lse = run()
    assert torch.isnan(out[:, :2]).all() and torch.isnan(lse[:, :2]).all()
    assert torch.equal(out[:, 2:], clean[:, 2:]) and torch.equal(lse[:, 2:], lse0[:, 2:])
    t[at] = keep
    if kind == "q8":                                     # (e4m3's NaN is a code)
        t, at = p.v.view(torch.uint8), (page, slot, 0, 7)
        keep, t[at] = t[at].clone(), 0x7F
        mine = [7]
    else:
        t, at = where(p.v, getattr(p, "v_groups", None))
        keep, t[at] = t[at].clone(), float("nan")
        mine = list(range(32)) if kind == "q4" else [7]
    out, lse = run()
    assert torch.isnan(out[:, :2][..., mine]).all()
    others = [c for c in range(d) if c not in mine]
    assert torch.equal(out[:, 2:], clean[:, 2:]) and torch.equal(lse, lse0)
    assert torch.equal(out[..., others], clean[..., others])
