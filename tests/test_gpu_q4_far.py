"""The 4-bit append, the reading back and the pool at their largest: offsets beyond 32 bits, 65536
sequences; and several calls at once."""
import random

import pytest

torch = pytest.importorskip("torch")
from tests.q4_ref import Problem4  # noqa: E402
from tests.test_gpu_pool import Model, i32, run_step, same  # noqa: E402
from tests.test_gpu_rows import randn  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sage():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_attention_smooth_gb300 import sage
    return sage


@pytest.mark.parametrize("n", [3, 900])
def test_append_and_gather_beyond_32_bit_offsets(sage, n):
    page, hkv, d = 128, 8, 128
    far_pages = (1 << 32) // (page * hkv * d // 2) + 600
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    near = Problem4([n], [1000], hkv, hkv, d, page, seed=1, poison=False, pool=8, offset=1.0)
    k, v = randn(2, n, hkv, d), randn(3, n, hkv, d)
    sage.kv_append(*near.sage(sage), k, v)
    want = sage.kv_gather(*near.sage(sage), n, torch.bfloat16)
    p = Problem4([n], [1000], hkv, hkv, d, page, seed=1, poison=False, pool=8, offset=1.0)
    far = far_pages - 8

    def spread(t):
        out = torch.empty(far_pages, *t.shape[1:], dtype=t.dtype, device="cuda")
        out[far:] = t
        return out

    p.k, p.v, p.k_groups, p.v_groups = (spread(t) for t in (p.k, p.v, p.k_groups, p.v_groups))
    p.table = torch.where(p.table < 8, p.table + far, p.table)
    sage.kv_append(*p.sage(sage), k, v)
    for a, b in ((p.k, near.k), (p.v, near.v), (p.k_groups, near.k_groups), (p.v_groups, near.v_groups)):
        assert torch.equal(a[far:].view(torch.uint8), b.view(torch.uint8))
    got = sage.kv_gather(*p.sage(sage), n, torch.bfloat16)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_the_most_sequences(sage):
    n = 65536
    rng = random.Random(5)
    pool = sage.PagePool.new(3 * n, 16, n, 64)
    model = Model(range(3 * n - 1, -1, -1), 16, n, pool.table.shape[1])
    reqs = rng.sample(range(n), n)
    run_step(sage, pool, model, reqs, [rng.randint(0, 20) for _ in reqs], 20, 64)
    keep = [rng.randint(0, 20) for _ in reqs]
    sage.paged_trim(pool, i32(reqs), i32(keep))
    model.trim(reqs, keep)
    same(pool, model)
    with pytest.raises(sage.SageError, match="sequences"):
        sage.paged_trim(pool, torch.zeros(n + 1, dtype=torch.int32, device="cuda"))


def test_nothing_to_do(sage):
    pool = sage.PagePool.new(4, 16, 2, 64)
    plan = sage.PagedPlan(pool, 0, 0, 1, 64)
    plan.cu_q.fill_(9)
    plan.denied.fill_(9)
    sage.paged_step(pool, plan, i32([]), i32([]))
    sage.paged_trim(pool, i32([]))
    assert plan.cu_q.tolist() == [0] and int(plan.denied) == 0 and int(pool.left) == 4
    p = Problem4([1], [20], 2, 2, 64, 16, poison=False)
    cache, _ = p.sage(sage)
    none = sage.PagedBatch(i32([0, 0]), i32([20]), p.table, 1, 20)
    x = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    f, _ = sage.rope_freqs(64)
    sage.kv_append(cache, none, x, x)
    sage.kv_append(cache, none, x, x, inv_freq=f, positions=torch.empty(3, 0, dtype=torch.int64, device="cuda"),
                   axes=sage.rope_axes((10, 11, 11)))
    assert sage.attn_paged(cache, none, x).shape == (0, 2, 64)
    assert sage.kv_gather(cache, none, 0, torch.bfloat16)[0].shape == (0, 2, 64)


def test_steps_and_appends_at_once(sage):
    """Two pools with their caches on two streams, each with its own workspace."""
    def make(seed):
        p = Problem4([5, 70], [40, 70], 4, 2, 64, 16, seed=seed, poison=False)
        pool = sage.PagePool.new(60, 16, 4, 300)
        return dict(p=p, args=p.sage(sage), pool=pool, plan=sage.PagedPlan(pool, 2, 14, 7, 300),
                    ws=sage.alloc_workspace_paged(), k=randn(seed, 75, 2, 64), v=randn(seed + 1, 75, 2, 64))

    def go(s, n):
        outs = []
        for i in range(n):
            sage.paged_step(s["pool"], s["plan"], i32([1, 3]), i32([7, 7]), ws=s["ws"])
            outs.append(s["plan"].slots.clone())
            sage.kv_append(*s["args"], s["k"] + i, s["v"], ws=s["ws"])
            outs.append(sage.kv_gather(*s["args"], 75, torch.bfloat16, ws=s["ws"])[0])
        return outs

    want = [go(make(seed), 15) for seed in (3, 9)]
    both = [make(seed) for seed in (3, 9)]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    got = []
    for s, stream in zip(both, streams):
        with torch.cuda.stream(stream):
            got.append(go(s, 15))
    torch.cuda.synchronize()
    for s, a, b in zip(both, want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        assert sage.device_status(s["ws"]) == sage.OK
