"""What a step that is denied for its own lengths means for the calls after it, and what a plan that
serves several steps holds behind a shorter one."""
import pytest

torch = pytest.importorskip("torch")
from tests.test_gpu_pool import Model  # noqa: E402
from tests.test_gpu_serving_step import D, HKV, Server, i32, inputs  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sage():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_attention_smooth_gb300 import sage
    return sage


# the second request: more than max_q; rows behind the plan's; more than max_kv; not in the pool
@pytest.mark.parametrize("request_id,new,rows,max_kv,written", [
    (3, 41, 60, 200, False), (3, 30, 35, 200, False), (3, 30, 60, 25, True), (9, 30, 60, 200, True)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_a_sequence_beyond_the_bounds_beside_a_good_one(sage, dt, request_id, new, rows, max_kv, written):
    """Nothing is stored of it; its rows of out are zeros if the batch's bounds hold, else they are
    left as they were."""
    s = Server(sage, dt)
    plan = sage.PagedPlan(s.pool, 2, rows, 40, max_kv)
    q, k, v, pos = inputs(90, rows, dt)
    before = [t.clone() for t in (s.k, s.v, s.k_groups, s.v_groups)]
    batch = sage.paged_step(s.pool, plan, i32([1, request_id]), i32([10, new]), ws=s.ws)
    assert int(plan.denied) == 1 and plan.kv_lens.tolist() == [10, 0]
    assert s.pool.lens.tolist() == [0, 10, 0, 0, 0, 0]
    end = min(10 + new, rows)
    assert (plan.slots[10:end] == -1).all() and (plan.positions[10:end] == -1).all()
    assert sage.device_status(s.ws) == sage.ERR_INVALID_ARG
    qr = torch.full_like(q, 5.0)
    sage.kv_append(s.cache, batch, k, v, q=q, q_out=qr, inv_freq=s.freqs, positions=pos, axes=s.axes,
                   ws=s.ws)
    assert (qr[10:] == 5.0).all()
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    sage.attn_paged(s.cache, batch, qr, out=out, lse=lse, ws=s.ws)
    page = int(plan.block_table[1 - 1, 0])
    for t, was in zip((s.k, s.v), before):
        assert not torch.equal(t[page, :10], was[page, :10])
        t = t.clone()
        t[page, :10] = was[page, :10]
        assert torch.equal(t, was)
    # the good sequence is what it is alone
    ws = sage.alloc_workspace_paged()
    alone = sage.PagedBatch(i32([0, 10]), i32([10]), plan.block_table[:1].contiguous(), 40, max_kv)
    assert torch.equal(out[:10], sage.attn_paged(s.cache, alone, qr[:10].contiguous(), ws=ws))
    want, want_lse = (0.0, -float("inf")) if written else (7.0, 7.0)
    assert (out[10:end] == want).all() and (lse[10:end] == want_lse).all()
    assert (out[end:] == 7.0).all()
    kb, vb = (torch.full((rows, HKV, D), 7.0, dtype=dt, device="cuda") for _ in range(2))
    sage.kv_gather(s.cache, batch, rows, k_out=kb, v_out=vb, ws=ws)
    assert (kb[10:end] == 0).all() and (vb[10:end] == 0).all()
    assert (kb[end:] == 7.0).all() and (vb[end:] == 7.0).all() and torch.isfinite(kb[:10]).all()


def test_a_captured_plan_whose_steps_get_shorter(sage):
    """Rows below cu_q[n] are this step's; those behind keep what a longer one left."""
    pool = sage.PagePool.new(40, 16, 4, 100)
    model = Model(range(39, -1, -1), 16, 4, pool.table.shape[1])
    plan = sage.PagedPlan(pool, 3, 30, 10, 100)
    reqs, new, ws = i32([2, 0, 3]), i32([0, 0, 0]), sage.alloc_workspace_paged()
    sage.paged_step(pool, plan, reqs, new, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sage.paged_step(pool, plan, reqs, new, ws=ws)
    held = [[-1] * 30, [-1] * 30]
    for lens in ([10, 10, 10], [3, 0, 9], [0, 1, 0], [10, 2, 1], [0, 0, 0]):
        new.copy_(i32(lens))
        graph.replay()
        cu, kv, tables, positions, slots, denied, bad = model.step([2, 0, 3], lens, 30, 10, 100, 7)
        held = [now[:cu[-1]] + was[cu[-1]:] for now, was in zip((positions, slots), held)]
        assert plan.cu_q.tolist() == cu and plan.kv_lens.tolist() == kv and denied == 0 and not bad
        assert [plan.positions.tolist(), plan.slots.tolist()] == held
    assert sage.device_status(ws) == sage.OK
