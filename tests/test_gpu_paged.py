"""Attention of new tokens over the paged cache, against the formula in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
from tests.paged_ref import Problem  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sage():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_attention_smooth_gb300 import sage
    return sage


def check(sage, p, scale=None, status=None, **kw):
    ws = sage.alloc_workspace_paged()
    cache, batch = p.sage(sage)
    rows = sum(p.q_lens)
    out = torch.full(p.q.shape, 7.0, dtype=p.q.dtype, device="cuda")
    lse = torch.full(p.q.shape[:2], 7.0, device="cuda")
    got = sage.attn_paged(cache, batch, p.q, out=out, window=p.window, sinks=p.sinks,
                          sm_scale=scale, lse=lse, ws=ws, **kw)
    assert got is out
    assert sage.device_status(ws) == (sage.OK if status is None else status), sage.last_error()
    ref, ref_lse, mean, spread = p.reference(scale)
    diff = (out.double() - ref).abs()[:rows]
    tol = p.tolerance(ref, mean, spread)[:rows]
    assert torch.isfinite(out[:rows]).all()
    assert (diff <= tol).all(), f"worst {float((diff / tol).max()):.3g} of the bound"
    empty = torch.isinf(ref_lse[:rows])
    assert torch.equal(torch.isinf(lse[:rows]) & (lse[:rows] < 0), empty)
    assert ((lse[:rows].double() - ref_lse[:rows])[~empty].abs() <= 2.0 ** -14).all()
    assert (out[rows:] == 7.0).all() and (lse[rows:] == 7.0).all()
    return out


KINDS = [("bf16", torch.bfloat16), ("f16", torch.float16), ("q8", torch.bfloat16),
         ("q8", torch.float16)]


@pytest.mark.parametrize("kind,dt", KINDS)
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (8, 2, 128), (6, 2, 80), (5, 1, 40), (16, 1, 128),
                                      (3, 3, 8), (12, 2, 72), (20, 1, 120)])
@pytest.mark.parametrize("page,layout", [(16, "NHD"), (64, "HND")])
def test_single_tokens(sage, kind, dt, hq, hkv, d, page, layout):
    check(sage, Problem([1, 1, 1, 1, 1], [1, 17, 300, 64, 129], hq, hkv, d, page, layout, kind, dt,
                        seed=hq * 100 + d))


@pytest.mark.parametrize("kind,dt", KINDS)
@pytest.mark.parametrize("page,layout,both", [(16, "HND", True), (48, "NHD", False),
                                              (128, "NHD", True), (256, "HND", False),
                                              (32, "NHD", False)])
@pytest.mark.parametrize("q_lens,kv_lens", [
    ([3, 0, 1, 40, 7], [3, 20, 0, 200, 500]),       # an empty sequence and one without keys
    ([130, 1, 17], [130, 300, 1000]),
    ([5, 300], [2, 260]),                            # more new tokens than positions
])
def test_chunks(sage, kind, dt, page, layout, both, q_lens, kv_lens):
    check(sage, Problem(q_lens, kv_lens, 6, 2, 96, page, layout, kind, dt, seed=len(q_lens) + page,
                        both=both, spare_rows=3))


@pytest.mark.parametrize("kind,dt", KINDS)
@pytest.mark.parametrize("d", [8, 40, 56, 72, 104, 112, 120])
@pytest.mark.parametrize("page,layout,both", [(16, "HND", False), (80, "NHD", True),
                                              (64, "NHD", False), (384, "HND", True)])
def test_chunks_of_odd_head_sizes(sage, kind, dt, d, page, layout, both):
    check(sage, Problem([140, 30, 1], [140, 400, 300], 6, 2, d, page, layout, kind, dt, seed=d,
                        both=both))


@pytest.mark.parametrize("kind,dt", KINDS)
@pytest.mark.parametrize("group", [1, 3, 7, 16, 40, 129])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [90, 700]), ([4, 37], [60, 300])])
def test_groups(sage, kind, dt, group, q_lens, kv_lens):
    """Any number of query heads on a kv head, also more than a row tile holds."""
    check(sage, Problem(q_lens, kv_lens, group, 1, 64, 32, "NHD", kind, dt, seed=group))


@pytest.mark.parametrize("kind,dt", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (16, 16), (100, 0), (100, 40),
                                          (129, 5), (600, 2), (5000, 4), (30, 2000)])
@pytest.mark.parametrize("q_lens,kv_lens,d", [([1, 5, 1, 33], [700, 700, 20, 64], 64),
                                              ([300, 2], [420, 900], 128)])
def test_window_and_sinks(sage, kind, dt, window, sinks, q_lens, kv_lens, d):
    check(sage, Problem(q_lens, kv_lens, 8, 2, d, 32, "NHD", kind, dt, window, sinks, seed=window))


@pytest.mark.parametrize("kind,dt", KINDS)
@pytest.mark.parametrize("scale", [0.01, 1.0])
def test_scale_and_strided_queries(sage, kind, dt, scale):
    p = Problem([2, 70, 1], [90, 200, 33], 4, 2, 64, 16, "NHD", kind, dt, seed=3)
    p.q = p.q * (0.3 if scale == 1.0 else 1.0)
    wide = torch.randn(p.q.shape[0], 11, 64, device="cuda").to(dt)
    wide[:, 3:7] = p.q
    p.q = wide[:, 3:7]                                # heads of a wider projection
    a = check(sage, p, scale)
    odd = torch.randn(p.q.shape[0], 4, 65, device="cuda").to(dt)
    odd[..., 1:] = p.q
    p.q = odd[..., 1:]                                # rows on 2-byte boundaries
    assert torch.equal(check(sage, p, scale), a)


@pytest.mark.parametrize("kind,dt", KINDS)
def test_long_split_sequences(sage, kind, dt):
    """One long sequence over every SM; results do not depend on the run."""
    p = Problem([1, 2], [20001, 333], 8, 2, 128, 16, "NHD", kind, dt, seed=5)
    a = check(sage, p)
    for _ in range(3):
        assert torch.equal(check(sage, p), a)


@pytest.mark.parametrize("kind,dt", KINDS)
def test_long_split_chunk(sage, kind, dt):
    p = Problem([150, 20], [6000, 4000], 8, 2, 128, 64, "HND", kind, dt, seed=6)
    a = check(sage, p)
    assert torch.equal(check(sage, p), a)


def test_many_sequences(sage):
    q_lens = [(i * 7) % 3 for i in range(700)]
    kv_lens = [q_lens[i] + (i * 13) % 90 for i in range(700)]
    check(sage, Problem(q_lens, kv_lens, 4, 1, 64, 16, "NHD", "bf16", torch.bfloat16, seed=8))


@pytest.mark.parametrize("kind,dt", KINDS)
def test_many_short_chunks_among_longer_ones(sage, kind, dt):
    """Several hundred chunks of one row tile after chunks of two: the roles of a
    CTA run ahead of each other by several items."""
    q_lens = [200 if i % 10 == 0 else 33 + i % 60 for i in range(1500)]
    kv_lens = [n + i % 70 for i, n in enumerate(q_lens)]
    check(sage, Problem(q_lens, kv_lens, 1, 1, 64, 16, "NHD", kind, dt, seed=17))


def test_declared_lengths_may_be_larger(sage):
    p = Problem([1, 40], [100, 70], 4, 2, 64, 16, "NHD", seed=9, max_kv=112)
    p.max_q = 1000
    check(sage, p)


@pytest.mark.parametrize("kind,dt", KINDS)
def test_large_queries_and_keys(sage, kind, dt):
    """Logits in the thousands: a softmax that picks one key."""
    p = Problem([1, 20], [300, 300], 4, 2, 64, 16, "NHD", kind, dt, seed=10)
    p.q = (p.q.float() * 100).to(dt)
    cache, batch = p.sage(sage)
    out = sage.attn_paged(cache, batch, p.q)
    ref = p.reference()[0]
    # a logit of 2^12 has an fp32 step of 2^-11: weights move by 2^-9 at most
    assert torch.isfinite(out).all()
    assert float((out.double() - ref).abs().max()) <= 2.0 ** -6 * float(ref.abs().max())


@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("q_len", [1, 200])
def test_cache_beyond_32_bit_offsets(sage, kind, q_len):
    """Pages whose element offsets pass 2^32."""
    page, hkv, d = 128, 8, 128
    pool = (1 << 32) // (page * hkv * d) + 600
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    p = Problem([q_len], [1000], 16, hkv, d, page, "NHD", kind, seed=11, poison=False, pool=8)
    small = check(sage, p)
    dt8 = kind == "q8"
    far = pool - 8
    k = torch.empty(pool, page, hkv, d, dtype=torch.int8 if dt8 else torch.bfloat16, device="cuda")
    v = torch.empty(pool, page, hkv, d, dtype=torch.uint8 if dt8 else torch.bfloat16, device="cuda")
    k[far:] = p.k
    v[far:] = p.v.view(torch.uint8) if dt8 else p.v
    p.k, p.v = k, v.view(torch.float8_e4m3fn) if dt8 else v
    if dt8:
        scale = torch.zeros(pool, hkv, page, device="cuda")
        scale[far:] = p.k_scale
        p.k_scale = scale
    p.table = torch.where(p.table < 8, p.table + far, p.table)
    cache, batch = p.sage(sage)
    assert torch.equal(sage.attn_paged(cache, batch, p.q), small)


@pytest.mark.parametrize("q_len", [1, 150])
def test_bad_page_is_reported_and_never_followed(sage, q_len):
    p = Problem([q_len, q_len], [200, 200], 4, 2, 64, 16, seed=12)
    good = check(sage, p)
    p.table[1, 3] = p.k.shape[0]                       # one past the pool
    p.table[1, 5] = -1
    ws = sage.alloc_workspace_paged()
    out = sage.attn_paged(*p.sage(sage), p.q, ws=ws)
    assert sage.device_status(ws) == sage.ERR_INVALID_ARG
    assert "block table" in sage.last_error()
    assert torch.equal(out[:q_len], good[:q_len])      # the other sequence is as it was


@pytest.mark.parametrize("q_len", [1, 150])
@pytest.mark.parametrize("what", ["kv", "q", "order"])
def test_bad_lengths_skip_their_sequence(sage, q_len, what):
    p = Problem([q_len, q_len], [200, 200], 4, 2, 64, 16, seed=13)
    ref, _, mean, spread = p.reference()
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
    # the other sequence is right (its split into parts goes by the whole batch, so not to the bit)
    tol = p.tolerance(ref, mean, spread)
    assert ((out.double() - ref).abs() <= tol)[:q_len].all()
    assert (out[q_len:] == 7.0).all()


@pytest.mark.parametrize("kind", ["bf16", "q8"])
def test_graphs_share_a_workspace(sage, kind):
    """Two captured graphs and eager calls take turns on one workspace; lengths
    change between replays without a new capture."""
    ws = sage.alloc_workspace_paged()
    ps = [Problem([1, 1, 60], [3000, 40, 500], 8, 2, 128, 16, "NHD", kind, seed=s, poison=False)
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


@pytest.mark.parametrize("kind", ["bf16", "q8"])
def test_two_calls_at_once(sage, kind):
    """Calls on two streams, each with its own workspace, do not disturb each other."""
    ps = [Problem([1, 1, 90], [4000, 300, 900], 8, 2, 128, 16, "NHD", kind, seed=s)
          for s in (18, 19)]
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


def test_another_stream(sage):
    p = Problem([1, 30], [500, 90], 8, 2, 128, 16, seed=16)
    want = check(sage, p)
    cache, batch = p.sage(sage)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        got = sage.attn_paged(cache, batch, p.q, stream=stream)
        s.synchronize()
        assert torch.equal(got, want)
    with torch.cuda.stream(s):
        got = sage.attn_paged(cache, batch, p.q)
    s.synchronize()
    assert torch.equal(got, want)
