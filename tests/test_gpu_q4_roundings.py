"""The roundings that the 4-bit cache's two kernels make, at large logits: the same tokens alone (few
rows: K exact) and at the end of a chunk (many rows: every element of K and V rounded to fp16)."""
import pytest

torch = pytest.importorskip("torch")
from tests.paged_ref import HALF  # noqa: E402
from tests.q4_ref import GROUP, Problem4  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sage():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_attention_smooth_gb300 import sage
    return sage


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128, 104])
@pytest.mark.parametrize("large", [1.0, 8.0, 20.0])
def test_few_and_many_rows_within_their_bounds(sage, dt, d, large):
    n, kv, few = 200, 700, 12
    p = Problem4([n], [kv], 2, 2, d, 16, "NHD", dt, seed=d, poison=False)
    scale = large * d ** -0.5
    ws = sage.alloc_workspace_paged()
    cache, batch = p.sage(sage)
    lse = torch.empty(n, 2, device="cuda")
    many = sage.attn_paged(cache, batch, p.q, sm_scale=scale, lse=lse, ws=ws)[-few:].double()
    many_lse = lse[-few:].double()
    last = sage.PagedBatch(torch.tensor([0, few], dtype=torch.int32, device="cuda"), p.lens, p.table, few, kv)
    lse = torch.empty(few, 2, device="cuda")
    alone = sage.attn_paged(cache, last, p.q[-few:], sm_scale=scale, lse=lse, ws=ws).double()
    alone_lse = lse.double()
    assert sage.device_status(ws) == sage.OK
    out, ref_lse, mean, _ = (x[-few:] for x in p.reference(scale))

    # What moves a logit x = scale sum q k.  Few rows: fp32 sums of exact products, in each group
    # of q times codes up to 15 and of -8 q, four tensor instructions of 2^-22 each on 23 sum |q|
    # s, so 2^-15 of scale sum |q| s.  Many rows: each k rounded to fp16, 2^-11 of it, and sums
    # of 2^-16.  Both: exp2's argument, |x| log2 e < 2^8 in fp32, 2^-16.
    k, _ = p.keys(0)
    s = p.k_groups.new_zeros(kv, 2, d, dtype=torch.float64)
    j = torch.arange(kv, device="cuda")
    s[:] = p.k_groups[p.table[0].long()[j // 16], :, j % 16][..., :p.groups].double().repeat_interleave(
        GROUP, -1)[..., :d]
    q = p.q[-few:].double().abs()
    big = lambda x: torch.einsum("thd,jhd->thj", q, x.abs()).amax(-1) * scale
    e_few = 2.0 ** -15 * big(s) + 2.0 ** -16
    e_many = (2.0 ** -11 + 3 * 2.0 ** -16) * big(k) + 2.0 ** -16
    assert large < 8 or float(big(k).max()) > 40         # (logits of some size, or the test says little)
    # lse moves by the largest move of a logit (and 2^-14 of fp32's logarithm)
    for got, e in ((alone_lse, e_few), (many_lse, e_many)):
        assert ((got - ref_lse).abs() <= e + 2.0 ** -14).all()
    assert ((alone_lse - many_lse).abs() <= e_few + e_many + 2.0 ** -13).all()
    # out: its own rounding; P times the scale, or P and V, to fp16; a weight moves by 2 e relative.
    # Below 2^-14 fp16 has steps of 2^-24 (weights of 2^7 at the largest, values to 512 v_scale).
    u = HALF[dt]
    steps = 512 * p.v_scale[:, :d].double() * kv * 2.0 ** -31 + (2.0 ** -25 if dt == torch.float16 else 0)

    def bound(e, roundings):
        e = e[..., None]
        return u * out.abs() + (roundings * 2.0 ** -11 + 2.0 ** -16 + 2 * e * (1 + e)) * mean * (1 + u) + steps

    few_bound, many_bound = bound(e_few, 1), bound(e_many, 2)
    assert ((alone - out).abs() <= few_bound).all()
    assert ((many - out).abs() <= many_bound).all()
    assert ((alone - many).abs() <= few_bound + many_bound).all()
