"""A pool and a plan made on the stream that uses them, while the current stream is busy."""
import pytest

torch = pytest.importorskip("torch")
from tests.test_gpu_pool import Model, i32, same  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sage():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_attention_smooth_gb300 import sage
    return sage


@pytest.mark.parametrize("raw", [False, True])       # a stream, or its handle
def test_made_on_the_stream_of_the_calls(sage, raw):
    s = torch.cuda.Stream()
    on = s.cuda_stream if raw else s
    reqs, new, keep = i32([3, 1]), i32([40, 50]), i32([20, 50])
    # memory that held something else, for the fills to matter
    with torch.cuda.stream(s):
        junk = [torch.full((64,), 77, dtype=torch.int32, device="cuda") for _ in range(64)]
    torch.cuda.synchronize()
    del junk
    torch.cuda._sleep(200_000_000)                   # about a tenth of a second
    pool = sage.PagePool.new(30, 16, 6, 100, stream=on)
    plan = sage.PagedPlan(pool, 2, 95, 64, 100, stream=on)
    ws = sage.alloc_workspace_paged(stream=on)
    sage.paged_step(pool, plan, reqs, new, ws=ws, stream=on)
    sage.paged_trim(pool, reqs, keep, ws=ws, stream=on)
    s.synchronize()
    torch.cuda.synchronize()
    model = Model(range(29, -1, -1), 16, 6, pool.table.shape[1])
    cu, lens, tables, positions, slots, denied, bad = model.step([3, 1], [40, 50], 95, 64, 100, 7)
    model.trim([3, 1], [20, 50])
    assert plan.cu_q.tolist() == cu and plan.kv_lens.tolist() == lens and not bad
    assert plan.block_table.tolist() == tables and int(plan.denied) == denied == 0
    assert plan.positions.tolist() == positions and plan.slots.tolist() == slots
    assert sage.device_status(ws) == sage.OK
    same(pool, model)


def test_a_pool_around_given_tables(sage):
    s = torch.cuda.Stream()
    base = sage.PagePool.new(30, 16, 6, 100)
    reqs, new = i32([0, 5]), i32([17, 1])
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    pool = sage.PagePool(base.free, base.left, base.table, base.lens, 16, stream=s)
    plan = sage.PagedPlan(pool, 2, 18, 20, 100, stream=s)
    sage.paged_step(pool, plan, reqs, new, stream=s)
    s.synchronize()
    model = Model(range(29, -1, -1), 16, 6, pool.table.shape[1])
    model.step([0, 5], [17, 1], 18, 20, 100, 7)
    same(pool, model)
