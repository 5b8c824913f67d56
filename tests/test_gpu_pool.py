"""Steps and cuts of a page pool against a plain model of it."""
import random

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sage():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_attention_smooth_gb300 import sage
    return sage


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Model:
    """The pool in plain Python."""

    def __init__(self, stack, page, requests, width):
        self.stack, self.page, self.width = list(stack), page, width
        self.pages, self.lens = [[] for _ in range(requests)], [0] * requests

    def step(self, reqs, new, rows, max_q, max_kv, width):
        """cu_q, kv_lens, tables, positions, slots, denied, whether something was reported."""
        at, cu, out, taken, dry, bad, seen = 0, [0], [], 0, False, False, set()
        positions, slots = [-1] * rows, [-1] * rows
        denied = 0
        for r, n in zip(reqs, new):
            start, at = at, at + max(n, 0)
            cu.append(at)
            fine = 0 <= r < len(self.lens) and r not in seen and 0 <= n <= max_q and at <= rows
            own = 0 <= r < len(self.lens) and r not in seen
            if own:
                seen.add(r)
            end = 0
            if fine:
                end = -(-(self.lens[r] + n) // self.page)
                fine = self.lens[r] + n <= max_kv and end <= min(width, self.width)
            bad |= not fine
            need = end - len(self.pages[r]) if fine else 0
            if fine and need > 0 and (dry or need > len(self.stack)):
                dry, fine = True, False
            if not fine:
                denied += 1
                out.append((0, list(self.pages[r][:width]) if own else []))
                continue
            old = self.lens[r]
            self.pages[r] += [self.stack.pop() for _ in range(need)]
            self.lens[r] += n
            out.append((self.lens[r], list(self.pages[r])))
            for t in range(n):
                positions[start + t] = old + t
                slots[start + t] = self.pages[r][(old + t) // self.page] * self.page + (old + t) % self.page
        tables = [t + [-1] * (width - len(t)) for _, t in out]
        return cu, [x for x, _ in out], tables, positions, slots, denied, bad

    def trim(self, reqs, keep):
        gone, seen, bad = [], set(), False
        for i, r in enumerate(reqs):
            k = 0 if keep is None else keep[i]
            if not 0 <= r < len(self.lens) or r in seen or k < 0:
                bad = True
                if 0 <= r < len(self.lens):
                    seen.add(r)
                continue
            seen.add(r)
            if k < self.lens[r]:
                stay = -(-k // self.page)
                gone += self.pages[r][stay:]
                del self.pages[r][stay:]
                self.lens[r] = k
        self.stack += gone[::-1]
        return bad


def same(pool, model):
    torch.cuda.synchronize()
    left = int(pool.left)
    assert left == len(model.stack)
    assert pool.free[:left].tolist() == model.stack
    assert pool.lens.tolist() == model.lens
    table = pool.table.tolist()
    assert all(table[r][:len(p)] == p for r, p in enumerate(model.pages))
    assert not pool.marks.any()


def run_step(sage, pool, model, reqs, new, max_q, max_kv, rows=None, spare=0):
    rows = sum(max(x, 0) for x in new) + spare if rows is None else rows
    plan = sage.PagedPlan(pool, len(reqs), rows, max_q, max_kv)
    plan.positions.fill_(-9)
    plan.slots.fill_(-9)
    ws = sage.alloc_workspace_paged()
    batch = sage.paged_step(pool, plan, i32(reqs), i32(new), ws=ws)
    assert batch is plan.batch
    cu, lens, tables, positions, slots, denied, bad = model.step(reqs, new, rows, max_q, max_kv,
                                                                 plan.block_table.shape[1])
    assert sage.device_status(ws) == (sage.ERR_INVALID_ARG if bad else sage.OK)
    assert plan.cu_q.tolist() == cu and plan.kv_lens.tolist() == lens
    assert plan.block_table.tolist() == tables
    used = min(cu[-1], rows)
    assert plan.positions.tolist()[:used] == positions[:used]
    assert plan.slots.tolist()[:used] == slots[:used]
    assert (plan.positions[used:] == -9).all() and (plan.slots[used:] == -9).all()
    assert int(plan.denied) == denied
    same(pool, model)
    return plan


@pytest.mark.parametrize("seed", range(8))
def test_random_steps_and_cuts(sage, seed):
    rng = random.Random(seed)
    page = rng.choice([16, 48, 64])
    requests = rng.choice([1, 5, 40])
    pages = rng.choice([3, 30, 400])
    max_len = rng.choice([60, 500, 3000])
    pool = sage.PagePool.new(pages, page, requests, max_len)
    model = Model(range(pages - 1, -1, -1), page, requests, pool.table.shape[1])
    for _ in range(25):
        reqs = rng.sample(range(requests), rng.randint(0, requests))
        if rng.random() < 0.6:
            new = [rng.choice([0, 1, 1, rng.randint(0, 100)]) for _ in reqs]
            run_step(sage, pool, model, reqs, new, 100, rng.choice([max_len, max_len // 2]),
                     spare=rng.choice([0, 7]))
        else:
            keep = None if rng.random() < 0.3 else [rng.randint(0, max_len) for _ in reqs]
            ws = sage.alloc_workspace_paged()
            sage.paged_trim(pool, i32(reqs), None if keep is None else i32(keep), ws=ws)
            assert model.trim(reqs, keep) is False and sage.device_status(ws) == sage.OK
            same(pool, model)


@pytest.mark.parametrize("n", [1, 1023, 1024, 1025, 5000])
def test_many_requests(sage, n):
    rng = random.Random(n)
    pool = sage.PagePool.new(4 * n, 16, n + 3, 100)
    model = Model(range(4 * n - 1, -1, -1), 16, n + 3, pool.table.shape[1])
    reqs = rng.sample(range(n + 3), n)
    for _ in range(3):
        run_step(sage, pool, model, reqs, [rng.randint(0, 30) for _ in reqs], 30, 100)


def test_a_cut_undoes_a_step(sage):
    rng = random.Random(3)
    pool = sage.PagePool.new(500, 16, 30, 1000)
    model = Model(range(499, -1, -1), 16, 30, pool.table.shape[1])
    reqs = list(range(30))
    run_step(sage, pool, model, reqs, [rng.randint(1, 90) for _ in reqs], 90, 1000)
    free, before = pool.free.clone(), pool.lens.clone()
    left = int(pool.left)
    order = rng.sample(reqs, 30)
    run_step(sage, pool, model, order, [rng.randint(0, 90) for _ in reqs], 90, 1000)
    sage.paged_trim(pool, i32(order), before[i32(order).long()].contiguous())
    model.trim(order, before[i32(order).long()].tolist())
    same(pool, model)
    assert int(pool.left) == left and torch.equal(pool.free, free)


def test_bad_entries_are_denied_and_reported(sage):
    pool = sage.PagePool.new(50, 16, 6, 200)
    model = Model(range(49, -1, -1), 16, 6, pool.table.shape[1])
    run_step(sage, pool, model, [0, 1, 2], [20, 30, 40], 50, 200)
    for reqs, new in [([0, 6, 1], [3, 4, 5]), ([-1, 2, 2 ** 31 - 1], [1, 1, 1]),
                      ([3, 3, 4, 3], [10, 10, 10, 10]),              # the same one three times
                      ([0, 1], [-5, 2]), ([4, 5], [51, 3]),          # below zero, beyond max_q
                      ([2, 5, 5], [40, 2, 1])]:
        run_step(sage, pool, model, reqs, new, 50, 200)
    run_step(sage, pool, model, [5, 0, 1], [10, 10, 10], 50, 200, rows=15)     # rows beyond the plan's
    run_step(sage, pool, model, [4, 2], [10, 20], 50, 90)            # beyond max_kv
    ws = sage.alloc_workspace_paged()
    sage.paged_trim(pool, i32([1, 9, 1, 2, -4, 0]), i32([5, 0, 0, -2, 0, 7]), ws=ws)
    assert model.trim([1, 9, 1, 2, -4, 0], [5, 0, 0, -2, 0, 7])
    assert sage.device_status(ws) == sage.ERR_INVALID_ARG
    same(pool, model)


def test_an_empty_stack(sage):
    pool = sage.PagePool.new(4, 16, 5, 64)
    model = Model(range(3, -1, -1), 16, 5, 4)
    run_step(sage, pool, model, [0, 1, 2, 3, 4], [16, 33, 1, 0, 5], 64, 64)    # 2 does not fit
    run_step(sage, pool, model, [0, 1, 2, 3], [0, 10, 1, 0], 64, 64)           # no new pages for 0, 1, 3
    sage.paged_trim(pool, i32([1, 4]))
    model.trim([1, 4], None)
    run_step(sage, pool, model, [4, 2], [16, 17], 64, 64)


def test_a_count_that_cannot_be(sage):
    """More free pages than the stack holds, or fewer than none: reported, nothing out of range."""
    for left in (99, -3):
        pool = sage.PagePool.new(4, 16, 2, 64)
        pool.left.fill_(left)
        plan = sage.PagedPlan(pool, 2, 20, 20, 64)
        ws = sage.alloc_workspace_paged()
        sage.paged_step(pool, plan, i32([0, 1]), i32([17, 3]), ws=ws)
        assert sage.device_status(ws) != sage.OK
        assert int(pool.left) == (1 if left == 99 else 0)
    pool = sage.PagePool.new(4, 16, 2, 64)
    pool.lens.copy_(i32([60, 10]))                       # pages that are on the stack as well
    pool.table.zero_()
    ws = sage.alloc_workspace_paged()
    sage.paged_trim(pool, i32([0, 1]), ws=ws)
    assert sage.device_status(ws) != sage.OK and int(pool.left) == 4


def test_tables_within_larger_ones_and_streams(sage):
    wide = torch.full((6, 40), -5, dtype=torch.int32, device="cuda")
    base = sage.PagePool.new(30, 16, 6, 100)
    pool = sage.PagePool(base.free, base.left, wide[:, 3:10], base.lens, 16)
    model = Model(range(29, -1, -1), 16, 6, 7)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        run_step(sage, pool, model, [3, 1], [40, 50], 64, 100)
    plan = sage.PagedPlan(pool, 2, 9, 9, 100)
    torch.cuda.synchronize()
    sage.paged_step(pool, plan, i32([0, 3]), i32([4, 5]), stream=s)
    s.synchronize()
    model.step([0, 3], [4, 5], 9, 9, 100, plan.block_table.shape[1])
    same(pool, model)
    assert (wide[:, :3] == -5).all() and (wide[:, 10:] == -5).all()


def test_a_captured_step(sage):
    """A decoding loop in a graph: every replay takes the next places."""
    pool = sage.PagePool.new(40, 16, 4, 100)
    model = Model(range(39, -1, -1), 16, 4, pool.table.shape[1])
    plan = sage.PagedPlan(pool, 3, 3, 1, 100)
    reqs, new, ws = i32([2, 0, 3]), i32([1, 1, 1]), sage.alloc_workspace_paged()
    sage.paged_step(pool, plan, reqs, new, ws=ws)
    model.step([2, 0, 3], [1, 1, 1], 3, 1, 100, 7)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sage.paged_step(pool, plan, reqs, new, ws=ws)
    for _ in range(40):
        graph.replay()
        _, lens, tables, positions, slots, _, _ = model.step([2, 0, 3], [1, 1, 1], 3, 1, 100, 7)
        assert plan.kv_lens.tolist() == lens and plan.block_table.tolist() == tables
        assert plan.positions.tolist() == positions and plan.slots.tolist() == slots
    same(pool, model)
    assert sage.device_status(ws) == sage.OK


def test_what_the_binding_refuses(sage):
    pool = sage.PagePool.new(8, 16, 4, 64)
    plan = sage.PagedPlan(pool, 2, 4, 2, 64)
    two = i32([0, 1])
    for args, match in [((two.long(), two), "requests"), ((two, two.long()), "new_lens"),
                        ((two[:1], two[:1]), "1 requests"), ((two.cpu(), two), "requests is not on"),
                        ((two[None], two), "1-D"), ((two, i32([1])), "new_lens")]:
        with pytest.raises(ValueError, match=match):
            sage.paged_step(pool, plan, *args)
    with pytest.raises(ValueError, match="keep_lens"):
        sage.paged_trim(pool, two, two.float())
    with pytest.raises(ValueError, match="table"):
        sage.PagePool(pool.free, pool.left, pool.table.long(), pool.lens, 16)
    with pytest.raises(ValueError, match="lens"):
        sage.PagePool(pool.free, pool.left, pool.table, pool.lens[:2], 16)
    with pytest.raises(ValueError, match="negative"):
        sage.PagedPlan(pool, -1, 4, 2, 64)
    with pytest.raises(sage.SageError, match="page_size"):
        odd = sage.PagePool(pool.free, pool.left, pool.table, pool.lens, 24)
        sage.paged_trim(odd, two)
