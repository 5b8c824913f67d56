"""The serving operators as a server runs them: a step's tables on the device, rotations of
several axes, the append into four bits, attention over it, and rejected tokens given back."""
import pytest

torch = pytest.importorskip("torch")
from tests.q4_ref import Problem4  # noqa: E402
from tests.test_gpu_rows import randn  # noqa: E402

pytestmark = pytest.mark.gpu
HQ, HKV, D, PAGE, PAGES = 8, 2, 64, 16, 40


@pytest.fixture(scope="module")
def sage():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_attention_smooth_gb300 import sage
    return sage


class Server:
    def __init__(self, sage, dt):
        self.sage, self.dt = sage, dt
        shape = (PAGES, PAGE, HKV, 32)
        new = lambda *s, **kw: torch.zeros(*s, device="cuda", **kw)
        self.k, self.v = new(*shape, dtype=torch.uint8), new(*shape, dtype=torch.uint8)
        self.k_groups, self.v_groups = (new(PAGES, HKV, PAGE, 2, dtype=torch.float16) for _ in range(2))
        for t in (self.k_groups, self.v_groups):
            t.fill_(float("nan"))                       # a slot that nobody wrote
        self.k_mean, self.v_scale = randn(1, HKV, 64, dt=torch.float32), new(HKV, 64) + 4 / 448
        self.cache = sage.PagedCache(self.k, self.v, "NHD", k_mean=self.k_mean, v_scale=self.v_scale,
                                     k_groups=self.k_groups, v_groups=self.v_groups, head_dim=D)
        self.pool = sage.PagePool.new(PAGES, PAGE, 6, 200)
        self.ws = sage.alloc_workspace_paged()
        self.axes, (self.freqs, _) = sage.rope_axes((8, 12, 12)), sage.rope_freqs(D)

    def step(self, plan, requests, new, q, k, v, pos):
        sage = self.sage
        batch = sage.paged_step(self.pool, plan, requests, new, ws=self.ws)
        qr = sage.kv_append(self.cache, batch, k, v, q=q, inv_freq=self.freqs, positions=pos,
                            axes=self.axes, ws=self.ws)
        return qr, sage.attn_paged(self.cache, batch, qr, ws=self.ws)

    def check(self, plan, qr, out):
        """out against the formula over what the cache holds."""
        cu, lens = plan.cu_q.tolist(), plan.kv_lens.tolist()
        q_lens = [b - a for a, b in zip(cu, cu[1:])]
        p = Problem4(q_lens, lens, HQ, HKV, D, PAGE, "NHD", self.dt, poison=False, pool=PAGES)
        p.k, p.v, p.k_groups, p.v_groups = self.k, self.v, self.k_groups, self.v_groups
        p.k_mean, p.v_scale, p.table, p.q = self.k_mean, self.v_scale, plan.block_table, qr
        ref, _, mean, spread = p.reference()
        assert ((out.double() - ref).abs() <= p.bound(ref, mean, spread)).all()
        assert self.sage.device_status(self.ws) == self.sage.OK, self.sage.last_error()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def inputs(seed, rows, dt):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [randn(seed + i, rows, h, D, dt=dt) for i, h in enumerate((HQ, HKV, HKV))] + [
        torch.randint(0, 300, (3, rows), generator=g, device="cuda")]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_prompts_drafts_and_a_captured_loop(sage, dt):
    s = Server(sage, dt)
    # prompts of three requests, one of them in two chunks
    plan = sage.PagedPlan(s.pool, 3, 90, 60, 200)
    qr, out = s.step(plan, i32([4, 0, 2]), i32([60, 13, 17]), *inputs(10, 90, dt))
    s.check(plan, qr, out)
    plan = sage.PagedPlan(s.pool, 1, 40, 40, 200)
    qr, out = s.step(plan, i32([2]), i32([40]), *inputs(20, 40, dt))
    s.check(plan, qr, out)
    # four drafted tokens each, of which some are rejected
    before = s.pool.lens.clone()
    plan = sage.PagedPlan(s.pool, 3, 12, 4, 200)
    reqs = i32([0, 2, 4])
    qr, out = s.step(plan, reqs, i32([4, 4, 4]), *inputs(30, 12, dt))
    s.check(plan, qr, out)
    keep = before[reqs.long()] + i32([4, 1, 0])
    sage.paged_trim(s.pool, reqs, keep.int(), ws=s.ws)
    assert s.pool.lens[reqs.long()].tolist() == keep.tolist()
    # single tokens in a captured graph
    plan, ones = sage.PagedPlan(s.pool, 3, 3, 1, 200), i32([1, 1, 1])
    buf = inputs(40, 3, dt)
    s.step(plan, reqs, ones, *buf)                      # (this token counts)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qr, out = s.step(plan, reqs, ones, *buf)
    for i in range(12):
        for a, b in zip(buf, inputs(50 + 7 * i, 3, dt)):
            a.copy_(b)
        graph.replay()
        s.check(plan, qr, out)
        assert int(plan.denied) == 0
    # finished requests' pages serve the next one
    left = int(s.pool.left)
    sage.paged_trim(s.pool, i32([0, 4]), ws=s.ws)
    assert int(s.pool.left) > left
    plan = sage.PagedPlan(s.pool, 1, 150, 150, 200)
    qr, out = s.step(plan, i32([5]), i32([150]), *inputs(60, 150, dt))
    s.check(plan, qr, out)
    assert int(plan.denied) == 0


def test_a_denied_sequence_is_left_out(sage):
    """A pool with too few pages: the denied sequence stores nothing and gives zeros."""
    s = Server(sage, torch.bfloat16)
    plan = sage.PagedPlan(s.pool, 2, 200, 190, 200)
    s.step(plan, i32([0, 1]), i32([190, 10]), *inputs(70, 200, torch.bfloat16))
    sage.paged_step(s.pool, sage.PagedPlan(s.pool, 1, 190, 190, 200), i32([2]), i32([190]), ws=s.ws)
    sage.paged_step(s.pool, sage.PagedPlan(s.pool, 1, 190, 190, 200), i32([3]), i32([190]), ws=s.ws)
    assert int(s.pool.left) == 3
    k, v = s.k.clone(), s.v.clone()
    plan = sage.PagedPlan(s.pool, 2, 70, 60, 200)
    qr, out = s.step(plan, i32([4, 1]), i32([60, 6]), *inputs(80, 70, torch.bfloat16))
    assert int(plan.denied) == 1 and plan.kv_lens.tolist() == [0, 16]
    assert (plan.slots[:60] == -1).all() and (plan.positions[:60] == -1).all()
    assert (out[:60] == 0).all() and s.pool.lens.tolist() == [190, 16, 190, 190, 0, 0]
    page = int(plan.block_table[1, 0])
    k[page, 10:] = s.k[page, 10:]
    v[page, 10:] = s.v[page, 10:]
    assert torch.equal(k, s.k) and torch.equal(v, s.v)
    assert sage.device_status(s.ws) == sage.OK
