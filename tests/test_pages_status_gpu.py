"""GPU tests of page allocation's status: raised by a step that cannot be made, and by no other, whether one block lays it out
or two kernels do, in eager and in replayed steps."""
import random

import pytest
import torch

import flash_attention_forward_gb300 as fa
from test_pages_gpu import Pages, check, ints, tensors

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,page,max_pages,most", [(1, 16, 8, 100), (7, 16, 20, 60), (64, 64, 256, 400), (1500, 32, 64, 200),
                                                   (3, 256, 40000, 9000)])
def test_steps_that_can_and_cannot_be_made(B, page, max_pages, most):
    rng = random.Random(B + 1)
    m = Pages(B, page, max_pages, 1 + B * (most // page + 1), B)
    table, kv_len, free, n_free = tensors(m)
    outcomes = []
    for step in range(14):
        change = [rng.choice([0, 1, -n, min(most, page * max_pages - n)]) for n in m.len]
        change = [min(d, page * max_pages - n) for d, n in zip(change, m.len)]
        total = max(1, sum(max(d, 0) for d in change))
        if step % 4 == 3:   # one row too many dropped, or a token more than announced
            if step % 8 == 3:
                change[0] = -m.len[0] - 1
            else:
                change[0], total = min(most, page * max_pages - m.len[0]), max(1, total - most)
        want = m.resize(change, total)
        outcomes.append(want is not None)
        if want is None:
            want = [0] * (B + 1), [0] * total, [-1] * total
        got = fa.sdpa_cache_resize(table, kv_len, ints(change), free, n_free, page, total, kv_len_out=kv_len, n_free_out=n_free)
        check(m, table, kv_len, free, n_free, got[2:], want)
        assert fa.sdpa_check_device_status() == (fa.SDPA_OK if outcomes[-1] else fa.SDPA_ERR_INVALID), (step, outcomes)
        assert fa.sdpa_check_device_status() == fa.SDPA_OK
    assert any(outcomes) and not all(outcomes)


@pytest.mark.parametrize("B", [9, 1100])
def test_replayed_steps(B):
    m = Pages(B, 16, 12, 4 * B, 1)
    assert m.resize([5 * (b % 9) for b in range(B)], 30 * B)
    table, kv_len, free, n_free = tensors(m)
    change = ints([0] * B)
    fa.sdpa_cache_resize(table, kv_len, change, free, n_free, 16, 2 * B)   # the first call, outside the capture
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        got = fa.sdpa_cache_resize(table, kv_len, change, free, n_free, 16, 2 * B, kv_len_out=kv_len, n_free_out=n_free)
    outcomes = []
    for step in range(12):
        d = [[1] * B, [2 if b % 2 else -1 for b in range(B)], [40] + [0] * (B - 1), [3] * B][step % 4]   # the last: too many tokens
        change.copy_(ints(d))
        want = m.resize(d, 2 * B)
        outcomes.append(want is not None)
        if want is None:
            want = [0] * (B + 1), [0] * (2 * B), [-1] * (2 * B)
        g.replay()
        check(m, table, kv_len, free, n_free, got[2:], want)
        assert fa.sdpa_check_device_status() == (fa.SDPA_OK if outcomes[-1] else fa.SDPA_ERR_INVALID), (step, outcomes)
    assert any(outcomes) and not all(outcomes)


def test_single_row_of_any_stride():
    # a table of one sequence made by a transpose: contiguous, with a row stride of 1
    m = Pages(1, 16, 6, 9, 2)
    _, kv_len, free, n_free = tensors(m)
    table = torch.full((6, 1), -1, dtype=torch.int32, device="cuda").t()
    assert table.is_contiguous() and table.stride(0) < 6
    want = m.resize([50], 50)
    got = fa.sdpa_cache_resize(table, kv_len, ints([50]), free, n_free, 16, 50, kv_len_out=kv_len, n_free_out=n_free)
    check(m, table, kv_len, free, n_free, got[2:], want)
    assert fa.sdpa_check_device_status() == fa.SDPA_OK
