"""The 8-bit cache as views whose strides are odd multiples of 8: rows then start
on 8 bytes only.  The writer and both attention kernels."""
import pytest

torch = pytest.importorskip("torch")
from tests.paged_ref import Problem  # noqa: E402
from tests.test_gpu_paged import check, sage  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def apart(p, head, token, page):
    """Moves p's codes into buffers with `head`, `token` and `page` bytes more from
    one head, token and page to the next; returns the buffers of K and V and the
    mask of the bytes that belong to no slot."""
    shape, d = p.k.shape, p.d
    n, slots, heads = p.k.shape[0], p.page, p.hkv
    if p.layout == "NHD":
        h = d + head
        t = heads * h + token
        g = slots * t + page
        strides = (g, t, h, 1)
    else:
        t = d + token
        h = slots * t + head
        g = heads * h + page
        strides = (g, h, t, 1)
    gaps = torch.ones(n * g, dtype=torch.bool, device=p.q.device)
    gaps.as_strided(shape, strides).fill_(False)
    bufs = []
    for x in (p.k, p.v):
        buf = torch.full((n * g,), 0x7F, dtype=torch.uint8, device=p.q.device)
        buf.as_strided(shape, strides).copy_(x.view(torch.uint8))
        bufs.append(buf)
    p.k = bufs[0].view(torch.int8).as_strided(shape, strides)
    p.v = bufs[1].view(torch.float8_e4m3fn).as_strided(shape, strides)
    return bufs, gaps


VIEWS = [(8, 0, 0), (0, 8, 0), (0, 0, 8), (24, 16, 40)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,page,layout", [(128, 16, "NHD"), (64, 64, "HND"), (80, 48, "NHD"),
                                           (16, 128, "HND"), (72, 32, "NHD"), (128, 256, "HND")])
@pytest.mark.parametrize("view", VIEWS)
def test_attention_over_narrow_rows(sage, dt, d, page, layout, view):  # noqa: F811
    for q_lens, kv_lens in (([1, 1, 1], [1, 300, 129]), ([5, 1], [90, 700]), ([150, 20], [400, 20]),
                            ([260], [260])):
        p = Problem(q_lens, kv_lens, 6, 2, d, page, layout, "q8", dt, seed=d + sum(view))
        apart(p, *view)
        check(sage, p)


@pytest.mark.parametrize("view", VIEWS)
def test_window_over_narrow_rows(sage, view):  # noqa: F811
    for q_lens, kv_lens in (([1, 3], [700, 20]), ([140], [420])):
        p = Problem(q_lens, kv_lens, 4, 1, 128, 32, "NHD", "q8", torch.bfloat16, 50, 5, seed=60)
        apart(p, *view)
        check(sage, p)


@pytest.mark.parametrize("d", [128, 64, 80, 72])
@pytest.mark.parametrize("view", VIEWS)
@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("q_lens", [[1, 1, 3], [900, 1, 30]])
def test_append_and_attend_over_narrow_rows(sage, d, view, layout, q_lens):  # noqa: F811
    """The same codes as in a cache without gaps, nothing written between the slots,
    and attention over what was written."""
    kv_lens = [n + 17 for n in q_lens]
    two = [Problem(q_lens, kv_lens, 4, 2, d, 32, layout, "q8", torch.bfloat16, seed=61, poison=False)
           for _ in range(2)]
    p = two[1]
    bufs, gaps = apart(p, *view)
    g = torch.Generator(device="cuda").manual_seed(62)
    k, v = (torch.randn(p.q.shape[0], 2, d, generator=g, device="cuda").to(torch.bfloat16)
            for _ in range(2))
    for x in two:
        sage.kv_append(*x.sage(sage), k, v)
    assert torch.equal(two[0].k, p.k) and torch.equal(two[0].k_scale, p.k_scale)
    assert torch.equal(two[0].v.view(torch.uint8), bufs[1].as_strided(p.k.shape, p.k.stride()))
    assert all((buf[gaps] == 0x7F).all() for buf in bufs)
    check(sage, p)
