"""GPU tests of page allocation against a stack and a page table kept as Python lists."""
import random

import pytest
import torch

import flash_attention_forward_gb300 as fa

pytestmark = pytest.mark.gpu

DEV = "cuda"


class Pages:
    """The definition: a stack, pushed to and popped from page by page."""

    def __init__(self, B, page, max_pages, n_pages, seed):
        self.page, self.max_pages = page, max_pages
        self.store = list(range(n_pages))
        random.Random(seed).shuffle(self.store)
        self.n_free = n_pages
        self.table = [[-1] * max_pages for _ in range(B)]
        self.len = [0] * B

    def pages(self, rows):
        return -(-rows // self.page)

    def resize(self, change, total):
        """(cu, positions, slots), or None and nothing changed."""
        new = [n + d for n, d in zip(self.len, change)]
        cu = [0]
        for d in change:
            cu.append(cu[-1] + max(d, 0))
        if min(new) < 0 or max(new) > self.page * self.max_pages or cu[-1] > total:
            return None
        stack = self.store[:self.n_free]
        for b, (o, n) in enumerate(zip(self.len, new)):
            stack += self.table[b][self.pages(n):self.pages(o)]
        if sum(max(0, self.pages(n) - self.pages(o)) for o, n in zip(self.len, new)) > len(stack):
            return None
        positions, slots = [], []
        for b, (o, n) in enumerate(zip(self.len, new)):
            for p in range(self.pages(o), self.pages(n)):
                self.table[b][p] = stack.pop()
            for t in range(o, n):
                positions.append(t)
                slots.append(self.table[b][t // self.page] * self.page + t % self.page)
        self.store[self.n_free:len(stack)] = stack[self.n_free:]
        self.n_free, self.len = len(stack), new
        pad = total - cu[-1]
        return cu, positions + [0] * pad, slots + [-1] * pad


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def tensors(m):
    return ints(m.table), ints(m.len), ints(m.store), ints([m.n_free])


def check(m, table, kv_len, free, n_free, got, want):
    torch.cuda.synchronize()
    assert kv_len.tolist() == m.len and n_free.tolist() == [m.n_free]
    assert table.tolist() == m.table and free.tolist() == m.store
    assert [x.tolist() for x in got] == [list(x) for x in want]


# the small tables are laid out by one block, the others by two kernels
@pytest.mark.parametrize("B,page,max_pages,most", [(1, 16, 8, 100), (7, 16, 20, 60), (64, 64, 256, 400), (1500, 32, 64, 200),
                                                   (3, 256, 40000, 9000)])
def test_steps_of_a_scheduler(B, page, max_pages, most):
    rng = random.Random(B)
    m = Pages(B, page, max_pages, 2 + min(B * max_pages, 3 * B * (most // page + 1)), B)
    table, kv_len, free, n_free = tensors(m)
    done = 0
    for step in range(12):
        change = []
        for b in range(B):
            x = rng.random()
            if m.len[b] == 0 or x < 0.2:
                change.append(min(rng.randint(0, most), page * max_pages - m.len[b]))
            elif x < 0.35:
                change.append(-m.len[b])
            elif x < 0.5:
                change.append(-rng.randint(0, min(m.len[b], 2 * page)))
            else:
                change.append(min(1, page * max_pages - m.len[b]))
        total = max(1, sum(max(d, 0) for d in change) + rng.choice([0, 3]))
        want = m.resize(change, total)
        if want is None:
            want = [0] * (B + 1), [0] * total, [-1] * total
        else:
            done += 1
        got = fa.sdpa_cache_resize(table, kv_len, ints(change), free, n_free, page, total, kv_len_out=kv_len, n_free_out=n_free)
        assert got[0] is kv_len and got[1] is n_free
        check(m, table, kv_len, free, n_free, got[2:], want)
        fa.sdpa_check_device_status()
    assert done >= 3


def test_pages_given_back_are_taken_by_the_same_call():
    m = Pages(3, 16, 4, 4, 0)
    table, kv_len, free, n_free = tensors(m)
    for change in ([64, 0, 0], [-64, 33, 0], [0, -33, 64], [0, 0, -48], [20, 9, 0]):  # four pages in all
        want = m.resize(change, 70)
        got = fa.sdpa_cache_resize(table, kv_len, ints(change), free, n_free, 16, 70)
        assert want is not None
        kv_len, n_free = got[:2]
        check(m, table, kv_len, free, n_free, got[2:], want)
    assert fa.sdpa_check_device_status() == fa.SDPA_OK


def test_same_inputs_same_call():
    m = Pages(5, 32, 50, 100, 3)
    m.resize([40, 500, 0, 31, 64], 1000)
    table, kv_len, free, n_free = tensors(m)
    m.resize([-40, 100, 7, 1, -33], 110)
    for _ in range(2):
        got = fa.sdpa_cache_resize(table, kv_len, ints([-40, 100, 7, 1, -33]), free, n_free, 32, 110)
        torch.cuda.synchronize()
        assert table.tolist() == m.table and free.tolist() == m.store and got[0].tolist() == m.len


@pytest.mark.parametrize("B,max_pages", [(4, 8), (2000, 64)])
@pytest.mark.parametrize("what", ["short", "negative", "long", "tokens", "n_free", "stack", "length"])
def test_a_change_that_cannot_be_made_changes_nothing(B, max_pages, what):
    page = 16
    m = Pages(B, page, max_pages, 2 * B, 5)
    assert m.resize([20, 16, 0, 1] * (B // 4), 50 * B)
    before = tensors(m)
    table, kv_len, free, n_free = tensors(m)
    change, total = [0] * B, 40 * B
    if what == "short":
        change = [40] * B
    elif what == "negative":
        change[1] = -17
    elif what == "long":
        change[3] = page * max_pages
    elif what == "tokens":
        change, total = [1] * B, B - 1
    elif what == "n_free":
        n_free[0] = -1
    elif what == "stack":
        n_free[0] = 2 * B + 1
    else:
        kv_len[2] = -5
    before = [t.clone() for t in (table, kv_len, free, n_free)]
    got = fa.sdpa_cache_resize(table, kv_len, ints(change), free, n_free, page, total)
    assert fa.sdpa_check_device_status() == fa.SDPA_ERR_INVALID
    assert torch.equal(got[0], kv_len) and torch.equal(got[1], n_free)
    assert (got[2] == 0).all() and (got[3] == 0).all() and (got[4] == -1).all()
    assert all(torch.equal(a, b) for a, b in zip(before, (table, kv_len, free, n_free)))
    assert fa.sdpa_check_device_status() == fa.SDPA_OK


def test_wide_table_views_canaries_streams_and_other_workspaces():
    m = Pages(6, 64, 30, 200, 7)
    m.resize([100, 0, 64, 65, 1, 640], 2000)
    wide = torch.full((6, 41), -7, dtype=torch.int32, device=DEV)
    wide[:, 5:35] = ints(m.table)
    _, kv_len, free, n_free = tensors(m)
    outs = {n: torch.full((k,), 77, dtype=d, device=DEV) for n, k, d in
            (("kv_len_out", 8, torch.int32), ("n_free_out", 3, torch.int32), ("cu_seqlens", 9, torch.int32),
             ("positions", 1002, torch.int32), ("slots", 1002, torch.int64))}
    sizes = {"kv_len_out": 6, "n_free_out": 1, "cu_seqlens": 7, "positions": 1000, "slots": 1000}
    change = [-100, 300, 1, -1, 63, 64]
    want = m.resize(change, 1000)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fa.sdpa_cache_resize(wide[:, 5:35], kv_len, ints(change), free, n_free, 64, 1000, stream=s,
                               **{n: t[1:1 + sizes[n]] for n, t in outs.items()})
    torch.cuda.synchronize()
    check(m, wide[:, 5:35], got[0], free, got[1], got[2:], want)
    assert (wide[:, :5] == -7).all() and (wide[:, 35:] == -7).all()
    for n, t in outs.items():
        assert t[0] == 77 and (t[1 + sizes[n]:] == 77).all()


def test_replayed_steps():
    # two captured calls share nothing; each replay is a step of decoding
    m = Pages(9, 16, 12, 80, 1)
    m.resize([5 * b for b in range(9)], 500)
    table, kv_len, free, n_free = tensors(m)
    change = ints([1] * 9)
    fa.sdpa_cache_resize(table, kv_len, change, free, n_free, 16, 9)   # the first call, outside the capture
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        got = fa.sdpa_cache_resize(table, kv_len, change, free, n_free, 16, 9, kv_len_out=kv_len, n_free_out=n_free)
    for step in range(40):
        if step % 3 == 2:
            change.copy_(ints([2 if b % 2 else -1 for b in range(9)]))
            want = m.resize([2 if b % 2 else -1 for b in range(9)], 9)
        else:
            change.copy_(ints([1] * 9))
            want = m.resize([1] * 9, 9)
        if want is None:
            want = [0] * 10, [0] * 9, [-1] * 9
        g.replay()
        check(m, table, kv_len, free, n_free, got[2:], want)
    fa.sdpa_check_device_status()
