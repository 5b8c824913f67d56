"""Attention of new tokens over the 4-bit cache, against the formula in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
from tests.q4_ref import Problem4  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def sage():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_attention_smooth_gb300 import sage
    return sage


def check(sage, p, scale=None, **kw):
    ws = sage.alloc_workspace_paged()
    cache, batch = p.sage(sage)
    rows = sum(p.q_lens)
    out = torch.full(p.q.shape, 7.0, dtype=p.q.dtype, device="cuda")
    lse = torch.full(p.q.shape[:2], 7.0, device="cuda")
    got = sage.attn_paged(cache, batch, p.q, out=out, window=p.window, sinks=p.sinks,
                          sm_scale=scale, lse=lse, ws=ws, **kw)
    assert got is out
    assert sage.device_status(ws) == sage.OK, sage.last_error()
    ref, ref_lse, mean, spread = p.reference(scale)
    diff = (out.double() - ref).abs()[:rows]
    tol = p.bound(ref, mean, spread, scale)[:rows]
    assert torch.isfinite(out[:rows]).all()
    assert (diff <= tol).all(), f"worst {float((diff / tol).max()):.3g} of the bound"
    empty = torch.isinf(ref_lse[:rows])
    assert torch.equal(torch.isinf(lse[:rows]) & (lse[:rows] < 0), empty)
    # a key's rounding to fp16 moves every logit by e at most
    e = 2.0 ** -11 * 40 + 2.0 ** -14
    assert ((lse[:rows].double() - ref_lse[:rows])[~empty].abs() <= e).all()
    assert (out[rows:] == 7.0).all() and (lse[rows:] == 7.0).all()
    return out


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (8, 2, 128), (6, 2, 80), (5, 1, 40), (16, 1, 128),
                                      (3, 3, 8), (12, 2, 72), (20, 1, 120), (4, 2, 32), (8, 1, 96)])
@pytest.mark.parametrize("page,layout,both", [(16, "NHD", True), (64, "HND", False)])
def test_single_tokens(sage, dt, hq, hkv, d, page, layout, both):
    check(sage, Problem4([1, 1, 1, 1, 1], [1, 17, 300, 64, 129], hq, hkv, d, page, layout, dt,
                         seed=hq * 100 + d, both=both))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("page,layout,both", [(16, "HND", True), (48, "NHD", False),
                                              (128, "NHD", True), (256, "HND", False),
                                              (32, "NHD", False)])
@pytest.mark.parametrize("q_lens,kv_lens", [
    ([3, 0, 1, 40, 7], [3, 20, 0, 200, 500]),       # an empty sequence and one without keys
    ([130, 1, 17], [130, 300, 1000]),
    ([5, 300], [2, 260]),                            # more new tokens than positions
])
def test_chunks(sage, dt, page, layout, both, q_lens, kv_lens):
    check(sage, Problem4(q_lens, kv_lens, 6, 2, 96, page, layout, dt, seed=len(q_lens) + page,
                         both=both, spare_rows=3))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("d", [8, 32, 40, 56, 64, 72, 104, 112, 128])
@pytest.mark.parametrize("page,layout,both", [(16, "HND", False), (80, "NHD", True),
                                              (64, "NHD", False), (384, "HND", True)])
def test_chunks_of_odd_head_sizes(sage, dt, d, page, layout, both):
    check(sage, Problem4([140, 30, 1], [140, 400, 300], 6, 2, d, page, layout, dt, seed=d, both=both))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("group", [1, 3, 7, 16, 40, 129])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [90, 700]), ([4, 37], [60, 300])])
@pytest.mark.parametrize("d", [64, 128])
def test_groups(sage, dt, group, q_lens, kv_lens, d):
    """Any number of query heads on a kv head, also more than a row tile holds."""
    check(sage, Problem4(q_lens, kv_lens, group, 1, d, 32, "NHD", dt, seed=group))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (16, 16), (100, 0), (100, 40),
                                          (129, 5), (600, 2), (5000, 4), (30, 2000)])
@pytest.mark.parametrize("q_lens,kv_lens,d", [([1, 5, 1, 33], [700, 700, 20, 64], 64),
                                              ([300, 2], [420, 900], 128)])
def test_window_and_sinks(sage, dt, window, sinks, q_lens, kv_lens, d):
    check(sage, Problem4(q_lens, kv_lens, 8, 2, d, 32, "NHD", dt, window, sinks, seed=window))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("scale", [0.01, 0.3])
def test_scale_and_strided_queries(sage, dt, scale):
    p = Problem4([2, 70, 1], [90, 200, 33], 4, 2, 64, 16, "NHD", dt, seed=3)
    wide = torch.randn(p.q.shape[0], 11, 64, device="cuda").to(dt)
    wide[:, 3:7] = p.q
    p.q = wide[:, 3:7]                                # heads of a wider projection
    a = check(sage, p, scale)
    odd = torch.randn(p.q.shape[0], 4, 65, device="cuda").to(dt)
    odd[..., 1:] = p.q
    p.q = odd[..., 1:]                                # rows on 2-byte boundaries
    assert torch.equal(check(sage, p, scale), a)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("q_lens,kv_lens,page", [([1, 2], [20001, 333], 16), ([150, 20], [6000, 4000], 64)])
def test_long_split_sequences(sage, dt, q_lens, kv_lens, page):
    """Sequences over every SM; results do not depend on the run."""
    p = Problem4(q_lens, kv_lens, 8, 2, 128, page, "NHD", dt, seed=5)
    a = check(sage, p)
    for _ in range(3):
        assert torch.equal(check(sage, p), a)


def test_many_sequences(sage):
    q_lens = [(i * 7) % 3 for i in range(700)]
    kv_lens = [q_lens[i] + (i * 13) % 90 for i in range(700)]
    check(sage, Problem4(q_lens, kv_lens, 4, 1, 64, 16, "NHD", torch.bfloat16, seed=8))


def test_many_short_chunks_among_longer_ones(sage):
    q_lens = [200 if i % 10 == 0 else 33 + i % 60 for i in range(1500)]
    kv_lens = [n + i % 70 for i, n in enumerate(q_lens)]
    check(sage, Problem4(q_lens, kv_lens, 1, 1, 64, 16, "NHD", torch.float16, seed=17))


def test_declared_lengths_may_be_larger(sage):
    p = Problem4([1, 40], [100, 70], 4, 2, 64, 16, "NHD", seed=9, max_kv=112)
    p.max_q = 1000
    check(sage, p)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("q_len", [1, 30, 200])
@pytest.mark.parametrize("down", [2.0 ** -20, 2.0 ** 10])
def test_queries_of_any_size(sage, dt, q_len, down):
    """Queries far from 1, whose logits the softmax's scale brings back."""
    p = Problem4([q_len], [300], 4, 2, 128, 16, "NHD", dt, seed=10)
    base = check(sage, p).double()
    if dt == torch.float16 and down < 1:
        p.q = (p.q.float() * 2.0 ** -6).to(dt)        # fp16: only so far without rounding
        p.q = torch.where(p.q.abs() < 2.0 ** -13, 0.0, p.q.float()).to(dt)
        base, down = check(sage, p, 128 ** -0.5 * 64).double(), 1.0
    big = Problem4([q_len], [300], 4, 2, 128, 16, "NHD", dt, seed=10)
    big.q = (p.q.float() * down).to(dt)
    scale = 128 ** -0.5 * (64 if down == 1.0 else 1.0) / down
    got = check(sage, big, scale).double()
    assert float((got - base).abs().max()) <= 2.0 ** -7 * float(base.abs().max())


@pytest.mark.parametrize("q_len", [1, 150])
def test_values_of_zero_scale(sage, q_len):
    p = Problem4([q_len], [200], 4, 2, 128, 16, flat=True, poison=False)
    cache, batch = p.sage(sage)
    assert (sage.attn_paged(cache, batch, p.q) == 0).all()


@pytest.mark.parametrize("q_len", [1, 200])
def test_a_small_weight_counts(sage, q_len):
    """One key of weight 2^-20 with the largest value beside one of weight 1 whose value is 0."""
    p = Problem4([q_len], [16], 1, 1, 64, 16, q_dtype=torch.float16, poison=False)
    p.k.fill_(0x88)                                   # zeros
    p.v.fill_(0x88)
    page = int(p.table[0, 0])
    p.k_groups.fill_(1.0)
    p.v_groups.fill_(1.0)
    p.v_scale.fill_(1.0)
    p.q.zero_()
    p.q[..., 0] = 1.0
    p.k[page, 0, 0, 0] = 0x8F                         # the first key's channel 0: 7
    p.v[page, 1, 0, 0] = 0x8F                         # the second one's value: 7 * 64
    scale = 20 * 0.6931471805599453 / 7               # logits 20 ln 2 and 0
    out = sage.attn_paged(*p.sage(sage), p.q, sm_scale=scale)
    last = out[-1, 0, 0].double()                     # sees all 16 keys
    want = 448 * 2.0 ** -20 / (1 + 15 * 2.0 ** -20)
    assert abs(float(last) - want) <= want * 2.0 ** -8


@pytest.mark.parametrize("q_len", [1, 200])
def test_cache_beyond_32_bit_offsets(sage, q_len):
    """Pages whose byte offsets pass 2^32, scales whose offsets pass 2^30."""
    page, hkv, d = 128, 8, 128
    far_pages = (1 << 32) // (page * hkv * d // 2) + 600
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    p = Problem4([q_len], [1000], 16, hkv, d, page, "NHD", seed=11, poison=False, pool=8)
    small = check(sage, p)
    far = far_pages - 8

    def spread(t):
        out = torch.empty(far_pages, *t.shape[1:], dtype=t.dtype, device="cuda")
        out[far:] = t
        return out

    p.k, p.v, p.k_groups, p.v_groups = (spread(t) for t in (p.k, p.v, p.k_groups, p.v_groups))
    p.table = torch.where(p.table < 8, p.table + far, p.table)
    assert torch.equal(sage.attn_paged(*p.sage(sage), p.q), small)


@pytest.mark.parametrize("q_len", [1, 150])
def test_bad_page_is_reported_and_never_followed(sage, q_len):
    p = Problem4([q_len, q_len], [200, 200], 4, 2, 64, 16, seed=12)
    good = check(sage, p)
    p.table[1, 3] = p.k.shape[0]                       # one past the pool
    p.table[1, 5] = -1
    ws = sage.alloc_workspace_paged()
    out = sage.attn_paged(*p.sage(sage), p.q, ws=ws)
    assert sage.device_status(ws) == sage.ERR_INVALID_ARG
    assert "block table" in sage.last_error()
    assert torch.equal(out[:q_len], good[:q_len])      # the other sequence is as it was
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("q_len", [1, 150])
@pytest.mark.parametrize("what", ["kv", "q", "order"])
def test_bad_lengths_skip_their_sequence(sage, q_len, what):
    p = Problem4([q_len, q_len], [200, 200], 4, 2, 64, 16, seed=13)
    ref, _, mean, spread = p.reference()
    tol = p.bound(ref, mean, spread)
    if what == "kv":
        p.lens[1] = 201                                # beyond max_kv
    elif what == "q":
        p.max_q = q_len
        p.cu[2] = 2 * q_len + 1                        # beyond the packed rows
    else:
        p.cu[2] = q_len - 1
    ws = sage.alloc_workspace_paged()
    out = torch.full_like(p.q, 7.0)
    sage.attn_paged(*p.sage(sage), p.q, out=out, ws=ws)
    assert sage.device_status(ws) == sage.ERR_INVALID_ARG
    assert ((out.double() - ref).abs() <= tol)[:q_len].all()
    assert (out[q_len:] == 7.0).all()


def test_graphs_share_a_workspace(sage):
    """Two captured graphs and eager calls take turns on one workspace; lengths change between
    replays without a new capture."""
    ws = sage.alloc_workspace_paged()
    ps = [Problem4([1, 1, 60], [3000, 40, 500], 8, 2, 128, 16, "NHD", seed=s, poison=False)
          for s in (14, 15)]
    runs = []
    for p in ps:
        cache, batch = p.sage(sage)
        out = torch.zeros_like(p.q)
        sage.attn_paged(cache, batch, p.q, out=out, ws=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sage.attn_paged(cache, batch, p.q, out=out, ws=ws)
        runs.append((p, cache, batch, out, graph))
    for lens in ([3000, 40, 500], [1700, 1, 61]):
        for p, *_ in runs:
            p.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        for p, cache, batch, out, graph in runs:
            out.zero_()
            graph.replay()
        for p, cache, batch, out, graph in runs:
            assert torch.equal(out, sage.attn_paged(cache, batch, p.q, ws=ws))
            p.kv_lens = lens
            check(sage, p)
    assert sage.device_status(ws) == sage.OK


def test_two_calls_at_once(sage):
    ps = [Problem4([1, 1, 90], [4000, 300, 900], 8, 2, 128, 16, "NHD", seed=s) for s in (18, 19)]
    want = [check(sage, p) for p in ps]
    args = [p.sage(sage) + (p.q,) for p in ps]
    ws = [sage.alloc_workspace_paged() for _ in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(sage.attn_paged(*args[i], ws=ws[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert sage.device_status(ws[i]) == sage.OK
        assert all(torch.equal(x, want[i]) for x in got[i])


def test_what_the_binding_refuses(sage):
    p = Problem4([1], [20], 2, 2, 64, 16, poison=False)
    args = dict(k_mean=p.k_mean, v_scale=p.v_scale, k_groups=p.k_groups, v_groups=p.v_groups, head_dim=64)

    def bad(match, k=p.k, v=p.v, **kw):
        with pytest.raises((ValueError, TypeError), match=match):
            sage.PagedCache(k, v, "NHD", **{**args, **kw})

    bad("head_dim", head_dim=None)
    bad("rows of", head_dim=80)
    bad("k_groups", k_groups=None)
    bad("v_groups", v_groups=p.v_groups.float())
    bad("k_mean", k_mean=None)
    bad("does not belong", k_scale=torch.zeros(p.k.shape[0], 2, 16, device="cuda"))
    bad("uint8", v=p.v.view(torch.int8))
    bad("strides", v=p.v.transpose(1, 2).contiguous().transpose(1, 2))
    half = torch.zeros(4, 16, 2, 64, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError, match="quantised"):
        sage.PagedCache(half, half.clone(), "NHD", k_groups=p.k_groups)
    with pytest.raises(ValueError, match="head_dim"):
        sage.PagedCache(half, half.clone(), "NHD", head_dim=32)
