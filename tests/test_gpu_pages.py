"""Page tables, slots and positions built on the GPU against a request-by-request model (whole numbers, equal)."""
import numpy as np
import pytest
import torch

import exl3_trellis_quantized_gb300 as E

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


class Model:
    """Plain lists: the requests' pages, lengths and the stack."""

    def __init__(self, rows, lens, stack, page, width):
        self.rows, self.lens, self.stack, self.page, self.width = rows, lens, stack, page, width

    def plan(self, new, total):
        cu, positions, slots, granted, dry = [0], [], [], [], False
        for b, n in enumerate(new):
            n = max(0, n)
            want = -(-(self.lens[b] + n) // self.page)
            need = max(0, want - len(self.rows[b])) if n else 0
            ok = sum(max(0, x) for x in new[:b + 1]) <= total and want <= self.width
            if ok and need:
                dry = dry or need > len(self.stack)
                ok = not dry
            if ok:
                self.rows[b] += [self.stack.pop() for _ in range(need)]
            for i in range(n):
                p = self.lens[b] + i
                positions.append(p)
                slots.append(self.rows[b][p // self.page] * self.page + p % self.page if ok else -1)
            self.lens[b] += n if ok else 0
            granted.append(ok)
            cu.append(min(total, cu[-1] + n))
        positions, slots = positions[:total], slots[:total]
        pad = total - len(positions)
        return cu, positions + [0] * pad, slots + [-1] * pad, granted

    def release(self, ended, shared, capacity):
        for b, done in enumerate(ended):
            if done:
                self.stack += self.rows[b][min(len(self.rows[b]), shared[b]):]
                self.rows[b], self.lens[b] = [], 0
        del self.stack[capacity:]


def make(batch, longest, page, spare, seed, ahead=0.1):
    rng = np.random.default_rng(seed)
    lens = [int(v) for v in rng.integers(0, longest + 1, batch)]
    held = [-(-n // page) + int(rng.random() < ahead) for n in lens]
    width = longest // page + 4
    order = rng.permutation(sum(held) + spare).tolist()
    rows = []
    for h in held:
        rows.append(order[:h])
        order = order[h:]
    table = np.full((batch, width), -7, dtype=np.int32)
    for b, r in enumerate(rows):
        table[b, :len(r)] = r
    capacity = sum(held) + spare + 3
    stack = np.full(capacity, -9, dtype=np.int32)
    stack[:spare] = order
    tables = E.KVTables(i32(table), i32(lens), i32(held), i32(stack), i32([spare]), page)
    return tables, Model(rows, lens, order, page, width), rng


def assert_state(tables, model):
    lens, held, table = tables.kv_lens.tolist(), tables.held.tolist(), tables.block_table.cpu().numpy()
    assert lens == model.lens and held == [len(r) for r in model.rows]
    for b, r in enumerate(model.rows):
        assert table[b, :len(r)].tolist() == r
    n = int(tables.free_count)
    assert n == len(model.stack) and tables.free_pages[:n].tolist() == model.stack


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("batch,longest,top,extra", [(1, 0, 1, 0), (1, 40, 3000, 5), (3, 500, 1, -2), (61, 3000, 1, 3),
                                                     (200, 900, 700, 0), (255, 33, 40, 9), (1025, 100, 6, 0),
                                                     (2049, 64, 5, 100), (5000, 300, 4, -300)])
def test_plan_steps(batch, longest, top, extra, page):
    """Two steps and what they leave; the rows may be too few (extra < 0), and pages run out."""
    for spare in (4 * batch + 2 * batch * top // page, batch // 3):
        tables, model, rng = make(batch, longest, page, spare, 1000 * batch + page)
        for _ in range(2):
            new = [int(v) for v in rng.integers(-1, top + 1, batch)]
            total = max(0, sum(max(0, n) for n in new) + extra)
            before = tables.block_table.clone()
            got = E.kv_plan(tables, i32(new), total)
            held = [len(r) for r in model.rows]
            want = model.plan(new, total)
            assert [g.dtype for g in got] == [torch.int32, torch.int32, torch.int64, torch.bool]
            for g, w in zip(got, want):
                assert g.tolist() == w
            assert_state(tables, model)
            # nothing else in the table changed
            after = tables.block_table.cpu().numpy()
            for b, r in enumerate(model.rows):
                before[b, held[b]:len(r)] = i32(r[held[b]:])
            assert (after == before.cpu().numpy()).all()


@pytest.mark.parametrize("batch,longest", [(1, 0), (1, 900), (7, 3000), (250, 2000), (2500, 100)])
@pytest.mark.parametrize("with_shared", [False, True])
def test_release(batch, longest, with_shared):
    tables, model, rng = make(batch, longest, 16, 11, batch)
    ended = rng.random(batch) < 0.6
    ended[0] = True
    shared = [int(v) for v in rng.integers(-1, 9, batch)] if with_shared else None
    E.kv_release(tables, torch.tensor(ended, device=DEV), None if shared is None else i32(shared))
    model.release(ended.tolist(), [max(0, v) for v in shared] if shared else [0] * batch, tables.free_pages.numel())
    assert_state(tables, model)
    E.kv_release(tables, torch.tensor(ended, device=DEV))  # nothing is left of them
    assert_state(tables, model)


def test_stack_too_small_for_what_comes_back():
    tables, model, _ = make(9, 400, 16, 5, 3)
    small = E.KVTables(tables.block_table, tables.kv_lens, tables.held, tables.free_pages[:20].clone(), tables.free_count, 16)
    guard = small.free_pages.clone()
    E.kv_release(small, torch.ones(9, dtype=torch.bool, device=DEV))
    model.release([True] * 9, [0] * 9, 20)
    assert int(small.free_count) == 20 and small.free_pages.tolist() == model.stack
    assert small.free_pages[:5].tolist() == guard[:5].tolist()


def test_state_out_of_range_is_clamped():
    """Counts and lengths that cannot be: taken as the nearest that can, and nothing outside the tensors is touched."""
    table = torch.full((4, 3), -1, dtype=torch.int32, device=DEV)
    table[:, 0] = i32([4, 5, 6, 7])
    stack = i32([0, 1, 2, 3])
    tables = E.KVTables(table, i32([-5, 10**9, 40, 3]), i32([1, 99, -4, 1]), stack, i32([70]), 16)
    cu, positions, slots, granted = E.kv_plan(tables, i32([2, 2, 2, 2**31 - 1]), 8)
    assert cu.tolist() == [0, 2, 4, 6, 8]
    # request 0 stands at 0; 1 is full; 2 holds nothing and wants three pages; 3 brings more than there is room for
    assert granted.tolist() == [True, False, True, False]
    assert positions.tolist() == [0, 1, 48, 49, 40, 41, 3, 4]
    assert slots.tolist() == [64, 65, -1, -1, 24, 25, -1, -1]
    assert int(tables.free_count) == 1 and tables.held.tolist() == [1, 3, 3, 1]
    assert table[2].tolist() == [3, 2, 1] and tables.kv_lens.tolist() == [2, 48, 42, 3]


@pytest.mark.parametrize("batch", [2048, 2049, 6000])
def test_rows_far_beyond_32_bits(batch):
    """Requests of 2^31 - 1 new tokens each, so that sums of sums pass 2^31: the first that fits is served, the rest wait."""
    page, width, total = 16, 8, 1 << 20
    tables = E.KVTables(i32(np.full((batch, width), -1)), i32([3] * batch), i32([0] * batch), i32(np.arange(64)), i32([64]), page)
    new = [5] + [2**31 - 1] * (batch - 2) + [0]
    cu, positions, slots, granted = E.kv_plan(tables, i32(new), total)
    assert cu.tolist() == [0, 5] + [total] * (batch - 1)
    assert granted.tolist() == [True] + [False] * (batch - 1)
    want = 3 + torch.cat([torch.arange(5), torch.arange(total - 5)])
    assert torch.equal(positions.cpu().long(), want)
    assert slots[:5].tolist() == [63 * page + 3 + i for i in range(5)] and bool((slots[5:] == -1).all())
    assert int(tables.free_count) == 63 and tables.held.tolist() == [1] + [0] * (batch - 1)
    assert tables.kv_lens.tolist() == [8] + [3] * (batch - 1)


def test_pages_far_beyond_32_bits():
    """Requests that lack 2^26 pages each, so that the needs of the batch pass 2^31: none is granted, and none behind them."""
    batch, page, width = 70, 16, 1 << 26
    table = torch.empty(batch, width, dtype=torch.int32, device=DEV)  # held 0: nothing of it is read
    table[:, 0] = -3
    lens = [4] + [2**30 - 1] * (batch - 2) + [4]
    tables = E.KVTables(table, i32(lens), i32([0] * batch), i32(np.arange(64)), i32([64]), page)
    cu, positions, slots, granted = E.kv_plan(tables, i32([1] * batch), batch)
    assert cu.tolist() == list(range(batch + 1)) and positions.tolist() == lens
    assert granted.tolist() == [True] + [False] * (batch - 1)
    assert slots.tolist() == [63 * page + 4] + [-1] * (batch - 1)
    assert int(tables.free_count) == 63 and tables.held.tolist() == [1] + [0] * (batch - 1)
    assert tables.kv_lens.tolist() == [5] + lens[1:] and table[:, 0].tolist() == [63] + [-3] * (batch - 1)


def test_into_leaves_the_state():
    tables, model, rng = make(300, 700, 32, 400, 8)
    keep = [t.clone() for t in (tables.kv_lens, tables.held, tables.free_count, tables.free_pages)]
    into = E.KVTables(tables.block_table, i32([0] * 300), i32([0] * 300), tables.free_pages, i32([0]), 32)
    new = [int(v) for v in rng.integers(0, 50, 300)]
    first = E.kv_plan(tables, i32(new), sum(new), into=into)
    again = E.kv_plan(tables, i32(new), sum(new), into=into)
    for a, b in zip(first, again):
        assert torch.equal(a, b)
    for t, k in zip((tables.kv_lens, tables.held, tables.free_count, tables.free_pages), keep):
        assert torch.equal(t, k)
    model.plan(new, sum(new))
    assert_state(into, model)


def test_captured_steps():
    """A graph of a step with a fixed number of rows, replayed as the lengths move on; given outputs on another stream."""
    batch, page, total = 37, 16, 160
    tables, model, rng = make(batch, 300, page, 600, 4)
    new = i32([0] * batch)
    outs = dict(cu_q=i32([0] * (batch + 1)), positions=i32([0] * total),
                slots=torch.zeros(total, dtype=torch.int64, device=DEV), granted=torch.zeros(batch, dtype=torch.bool, device=DEV))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        E.kv_plan(tables, new, total, **outs)  # no new tokens: nothing moves
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            E.kv_plan(tables, new, total, **outs)
        for _ in range(5):
            step = [int(v) for v in rng.integers(0, 5, batch)]
            new.copy_(i32(step))
            graph.replay()
            want = model.plan(step, total)
            for t, w in zip(outs.values(), want):
                assert t.tolist() == w
            assert_state(tables, model)


def test_empty_batch():
    tables = E.KVTables(i32(np.zeros((0, 4))), i32([]), i32([]), i32([1, 2]), i32([2]), 16)
    cu, positions, slots, granted = E.kv_plan(tables, i32([]), 3)
    assert cu.tolist() == [0] and positions.tolist() == [0] * 3 and slots.tolist() == [-1] * 3 and granted.numel() == 0
    E.kv_release(tables, torch.zeros(0, dtype=torch.bool, device=DEV))
    assert int(tables.free_count) == 2


def test_every_row_of_a_long_prompt():
    """One request of more rows than the cluster takes at a time, and pages named far beyond 2^31 rows: slots in 64 bits."""
    total, page = 70001, 256
    need = (total + page - 1) // page
    far = 2**31 - 1 - need
    stack = torch.arange(far, far + need, dtype=torch.int32, device=DEV)
    tables = E.KVTables(i32(np.full((1, need + 1), -1)), i32([0]), i32([0]), stack, i32([need]), page)
    cu, positions, slots, granted = E.kv_plan(tables, i32([total]), total)
    at = torch.arange(total, device=DEV)
    assert granted.item() and cu.tolist() == [0, total] and torch.equal(positions.long(), at)
    assert torch.equal(slots, (far + need - 1 - at // page) * page + at % page)
    assert int(tables.free_count) == 0 and torch.equal(tables.block_table[0, :need], stack.flip(0))
