"""GPU parity of the chunk attention over paged caches (16-bit and quantised) against the fp64 oracle.

Tolerance.  The probabilities are rounded to the 16-bit type of the P.V product (half a step u_p: bf16
2^-8, fp16 2^-11; quantised caches use fp16 whatever the query's type), the row sums are fp32 of the
unrounded ones, exp2 and the fp32 score carry 2^-21 |s| (scores below 2^6 here: 2^-15, twice: numerator and
sum), and the output is rounded once (half a step u).  With |V| <= vmax over the visible keys
    |dO| <= u |O| + (u_p + 2^-14 + 2^-16) vmax,   |dLSE| <= 2^-15 + 2^-16.
A quantised V row adds at most 2^-25 of its block's largest magnitude (fp16's smallest step below the
scaled codes), inside the 2^-16.
"""
import numpy as np
import pytest
import torch

import flash_attention_forward_gb300 as fa
import oracle

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
TOL_LSE = 2.0 ** -15 + 2.0 ** -16


def make(new, lens, Hq, Hkv, D, Dv, page, dtype, quant, seed=0, spare=2, gain=None):
    """Packed queries and a paged cache: rows past a length and spare pages are NaN (codes and scales), table
    entries past a sequence's pages are wild."""
    g = torch.Generator().manual_seed(seed)
    pages = [(L + page - 1) // page for L in lens]
    n_pages, max_pages = sum(pages) + spare, max(max(pages), 1) + 1
    perm = torch.randperm(n_pages, generator=g).to(torch.int32)
    wild = torch.tensor([-7, 1 << 30, n_pages, 3], dtype=torch.int32)
    table = wild[torch.arange(len(lens) * max_pages) % 4].view(len(lens), max_pages).clone()
    k = torch.full((n_pages, page, Hkv, D), float("nan"))
    v = torch.full((n_pages, page, Hkv, Dv), float("nan"))
    at = 0
    for b, L in enumerate(lens):
        ids = perm[at:at + pages[b]].long()
        table[b, :pages[b]] = ids.to(torch.int32)
        at += pages[b]
        for pool, d in ((k, D), (v, Dv)):
            rows = torch.full((pages[b] * page, Hkv, d), float("nan"))
            rows[:L] = torch.randn((L, Hkv, d), generator=g)
            if gain is not None:
                rows = rows * gain(g, rows)
            pool[ids] = rows.view(pages[b], page, Hkv, d)
    q = torch.randn((sum(new), Hq, D), generator=g).to(DT[dtype])
    if quant:
        pools = []
        for pool in (k, v):
            codes, scales = oracle.quantise_pool(pool)
            nan = torch.isnan(pool).all(-1).transpose(1, 2)
            pools += [codes, torch.where(nan, torch.full_like(scales, float("nan")), scales).contiguous()]
    else:
        pools = [k.to(DT[dtype]), v.to(DT[dtype])]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
    return q, pools, table, torch.tensor(lens, dtype=torch.int32), cu


def run(q, pools, table, kv, cu, maxq, **kw):
    d = [t.to(DEV) for t in pools]
    if len(pools) == 4:
        o, lse = fa.sdpa_fwd_paged_fp8(q.to(DEV), d[0], d[2], d[1], d[3], table.to(DEV), kv.to(DEV), cu.to(DEV), maxq, **kw)
    else:
        o, lse = fa.sdpa_fwd_paged(q.to(DEV), d[0], d[1], table.to(DEV), kv.to(DEV), cu.to(DEV), maxq, **kw)
    torch.cuda.synchronize()
    assert fa.sdpa_check_device_status() == fa.SDPA_OK
    return o, lse


def values(pools):
    if len(pools) == 4:
        return oracle.dequantise_pool(*pools[:2]), oracle.dequantise_pool(*pools[2:])
    return pools


def check(q, pools, table, kv, cu, o, lse, scale, causal):
    k, v = values(pools)
    kvl = kv.tolist()
    ref, ref_lse = oracle.sdpa_fwd_paged(q, k, v, table, kvl, cu, scale=scale, causal=causal)
    got, got_lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    u = torch.finfo(o.dtype).eps / 2
    u_p = 2.0 ** -11 if len(pools) == 4 or o.dtype == torch.float16 else 2.0 ** -8
    vg = oracle.gather_pages(v, table, kvl)
    for b in range(len(kvl)):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        if rows.stop == rows.start:
            continue
        L = max(0, min(kvl[b], vg.shape[1]))
        vmax = float(vg[b, :L].abs().max()) if L else 0.0
        assert np.isfinite(got[rows]).all(), f"sequence {b}: NaN or Inf"
        err = np.abs(got[rows] - ref[rows])
        assert (err <= u * np.abs(ref[rows]) + (u_p + 2.0 ** -14 + 2.0 ** -16) * vmax).all(), (b, err.max(), vmax)
        dead = np.isneginf(ref_lse[:, rows])
        assert np.array_equal(np.isneginf(got_lse[:, rows]), dead)
        assert (got[rows][dead.T] == 0).all()
        if (~dead).any():
            e = np.abs(got_lse[:, rows] - ref_lse[:, rows])[~dead].max()
            assert e <= TOL_LSE, (b, e)


NEW = [1, 3, 0, 33, 64, 130, 5, 20, 1, 2]
LENS = [1, 3, 5, 33, 700, 131, 127, 128, 129, 1500]


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hq,Hkv,D,Dv,page", [(8, 2, 128, 128, 64), (14, 2, 128, 128, 16), (3, 3, 64, 64, 32),
                                              (16, 1, 192, 128, 128), (4, 4, 192, 128, 16), (24, 2, 64, 64, 256)])
@pytest.mark.parametrize("causal", [True, False])
def test_ragged_chunks(quant, dtype, Hq, Hkv, D, Dv, page, causal):
    x = make(NEW, LENS, Hq, Hkv, D, Dv, page, dtype, quant)
    o, lse = run(*x, max(NEW), scale=D ** -0.5, causal=causal)
    check(*x, o, lse, D ** -0.5, causal)


@pytest.mark.parametrize("quant", [False, True])
def test_tokens_without_keys(quant):
    # an empty cache, and more new tokens than rows: the first ones sit at negative positions
    x = make([4, 10, 2], [0, 6, 2], 8, 2, 128, 128, 16, "bf16", quant)
    o, lse = run(*x, 10, scale=0.1, causal=True)
    check(*x, o, lse, 0.1, True)
    assert torch.isneginf(lse[:, :8]).all() and (o[:8] == 0).all()
    o, lse = run(*x, 10, scale=0.1, causal=False)
    check(*x, o, lse, 0.1, False)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("new,lens", [([5], [20000]), ([1, 8, 3], [9000, 300, 6000]), ([300], [8000]), ([2000], [2000])])
def test_cut_key_ranges(quant, new, lens):
    # few rows over long caches: the plan cuts the keys; a workspace for the plan alone must give the same
    x = make(new, lens, 8, 2, 128, 128, 64, "bf16", quant, seed=4)
    o, lse = run(*x, max(new), scale=0.09, causal=True)
    check(*x, o, lse, 0.09, True)
    plan = fa.sdpa_fwd_paged_workspace_size(len(new), 8, 2, sum(new), max(new), 1, 128)
    small = torch.empty(plan, dtype=torch.uint8, device=DEV)
    o2, lse2 = run(*x, max(new), scale=0.09, causal=True, workspace=small)
    check(*x, o2, lse2, 0.09, True)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("B,new", [(40, 1), (300, 2)])
def test_many_sequences_on_each_sm(quant, B, new):
    # every CTA walks several units, most of one ragged block
    g = torch.Generator().manual_seed(6)
    lens = torch.randint(new, 400, (B,), generator=g).tolist()
    x = make([new] * B, lens, 4, 2, 128, 128, 16, "bf16", quant, seed=7)
    o, lse = run(*x, new, scale=0.09, causal=True)
    check(*x, o, lse, 0.09, True)


@pytest.mark.parametrize("quant", [False, True])
def test_sequences_without_new_tokens_between_short_chunks(quant):
    # one query tile a sequence: the plan passes over the empty ones, at both ends too
    x = make([0, 0, 3, 0, 1, 16, 0, 2, 0], [9, 0, 900, 40, 1, 5000, 300, 70, 128], 8, 2, 128, 128, 64, "bf16", quant, seed=11)
    o, lse = run(*x, 16, scale=0.09, causal=True)
    check(*x, o, lse, 0.09, True)


@pytest.mark.parametrize("quant", [False, True])
def test_more_sequences_than_the_plan_keeps_in_shared_memory(quant):
    g = np.random.default_rng(12)
    new, lens = g.integers(0, 4, 1100).tolist(), g.integers(1, 150, 1100).tolist()
    x = make(new, lens, 4, 2, 64, 64, 16, "f16", quant, seed=12)
    o, lse = run(*x, max(new), scale=0.125, causal=True)
    check(*x, o, lse, 0.125, True)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("D", [64, 192])
def test_the_widest_group_and_more_tiles_than_the_plan_keeps_in_shared_memory(quant, D):
    # 128 heads of one KV head: a query tile is one token, 2300 tokens are 1150 units
    x = make([2203, 97], [200, 64], 128, 1, D, 64 if D == 64 else 128, 32, "bf16", quant, seed=13)
    o, lse = run(*x, 2203, scale=D ** -0.5, causal=False)
    check(*x, o, lse, D ** -0.5, False)


def test_rows_of_very_different_scales():
    # scales up to 2^12 apart inside a block, bf16 queries far outside fp16's range
    gain = lambda g, rows: torch.exp2(torch.randint(-12, 1, rows.shape[:-1], generator=g).float())[..., None]  # noqa: E731
    for qg in (2.0 ** -20, 2.0 ** 20):
        q, pools, table, kv, cu = make([9, 40], [500, 140], 8, 2, 128, 128, 32, "bf16", True, gain=gain)
        q = (q.float() * qg).to(q.dtype)
        o, lse = run(q, pools, table, kv, cu, 40, scale=0.09 / qg, causal=True)
        check(q, pools, table, kv, cu, o, lse, 0.09 / qg, True)


def test_small_values_keep_their_precision_beside_large_ones():
    # all the weight on a key whose V row is 2^-18 of its block's others: the output is that row.  Its codes
    # reach fp16 times 2^-18 * 2^6 of the block's factor, exact down to codes of 2^-12 * 2^-24
    q, pools, table, kv, cu = make([3], [200], 4, 1, 128, 128, 16, "bf16", False)
    k, v = torch.zeros(pools[0].shape), pools[1].float()
    p, r = int(table[0, 77 // 16]), 77 % 16
    k[p, r, 0] = 20.0  # score 2560 against 0
    v[p, r] *= 2.0 ** -18
    pools = [*oracle.quantise_pool(k), *oracle.quantise_pool(torch.nan_to_num(v))]
    o, _ = run(torch.ones_like(q), pools, table, kv, cu, 3, scale=1.0, causal=True)
    want = oracle.dequantise_pool(*pools[2:])[p, r, 0]
    err = (o[0, 0].double().cpu() - want).abs()
    assert (err <= 2.0 ** -8 * want.abs() + 2.0 ** -25 * 2.0 ** -6 * float(pools[3].max()) * 2).all()


def test_zero_queries_and_zero_keys():
    # a zero query row against a zero K block: every score is 0 and the mask must stay a mask
    q, pools, table, kv, cu = make([4], [130], 4, 1, 128, 128, 16, "bf16", False)
    k, v = torch.nan_to_num(pools[0].float()) * 0, torch.nan_to_num(pools[1].float())
    pools = [*oracle.quantise_pool(k), *oracle.quantise_pool(v)]
    q[:2] = 0
    o, lse = run(q, pools, table, kv, cu, 4, scale=0.09, causal=True)
    check(q, pools, table, kv, cu, o, lse, 0.09, True)


@pytest.mark.parametrize("quant", [False, True])
def test_strides_interleaved_pools_and_untouched_rows(quant):
    new, lens, page = [7, 20], [50, 40], 16
    q, pools, table, kv, cu = make(new, lens, 8, 2, 128, 128, page, "f16", quant)
    k, v = pools[0], pools[-2] if quant else pools[1]
    # K and V pages alternate in one pool; q and o are slices of wider rows; two rows belong to nobody
    both = torch.stack([k.view(torch.uint8 if quant else torch.int16), v.view(torch.uint8 if quant else torch.int16)], 1).to(DEV)
    both = both.view(torch.float8_e4m3fn if quant else torch.float16)
    wide = torch.zeros((29, 10, 256), dtype=q.dtype, device=DEV)
    wide[:27, 1:9, 128:] = q.to(DEV)
    out = torch.full((29, 9, 192), 5.0, dtype=q.dtype, device=DEV)
    tab = torch.full((2, table.shape[1] + 5), -1, dtype=torch.int32, device=DEV)
    tab[:, : table.shape[1]] = table.to(DEV)
    args = (table.shape[1],)
    qs, os_ = wide[:, 1:9, 128:], out[:, :8, 64:]
    common = (tab[:, : args[0]], kv.to(DEV), cu.to(DEV), 20)
    if quant:
        _, lse = fa.sdpa_fwd_paged_fp8(qs, both[:, 0], both[:, 1], pools[1].to(DEV), pools[3].to(DEV), *common, scale=0.1,
                                       causal=True, out=os_)
    else:
        _, lse = fa.sdpa_fwd_paged(qs, both[:, 0], both[:, 1], *common, scale=0.1, causal=True, out=os_)
    torch.cuda.synchronize()
    assert (out[27:] == 5).all() and (out[..., :64] == 5).all() and (out[:, 8] == 5).all()
    check(q, pools, table, kv, cu, os_[:27].contiguous(), lse[:, :27].contiguous(), 0.1, True)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("new", [[3, 2, 4], [150, 70, 200]])
def test_lengths_outside_the_table_are_clamped(quant, new):
    q, pools, table, kv, cu = make(new, [100, 40, 300], 8, 2, 128, 128, 32, "bf16", quant, seed=15)
    for i, t in enumerate(pools):  # every row of every page may be visible now
        pools[i] = torch.nan_to_num(t.float(), nan=0.5).to(t.dtype)
    table[1] = torch.arange(table.shape[1], dtype=torch.int32) % pools[0].shape[0]
    cap = table.shape[1] * 32
    kv = torch.tensor([-(1 << 31), (1 << 31) - 1, 300], dtype=torch.int32)
    clamped = torch.tensor([0, cap, 300], dtype=torch.int32)
    o, lse = run(q, pools, table, kv, cu, max(new), scale=0.09, causal=False)
    check(q, pools, table, clamped, cu, o, lse, 0.09, False)
    # a position far behind the table sees all of it, one before the first row nothing
    o, lse = run(q, pools, table, kv, cu, max(new), scale=0.09, causal=True)
    ref, ref_lse = oracle.sdpa_fwd_paged(q, *values(pools), table, clamped, cu, scale=0.09, causal=False)
    rows = slice(int(cu[1]), int(cu[2]))
    vmax = float(oracle.gather_pages(values(pools)[1], table, clamped.tolist())[1].abs().max())
    u_p = 2.0 ** -11 if quant else 2.0 ** -8
    err = np.abs(o.double().cpu().numpy()[rows] - ref[rows])
    assert (err <= 2.0 ** -8 * np.abs(ref[rows]) + (u_p + 2.0 ** -14 + 2.0 ** -16) * vmax).all()
    assert np.abs(lse.double().cpu().numpy()[:, rows] - ref_lse[:, rows]).max() <= TOL_LSE
    assert (o[:new[0]] == 0).all() and torch.isneginf(lse[:, :new[0]]).all()


def test_bad_offsets_store_nothing_and_are_reported():
    q, pools, table, kv, cu = make([5, 6], [50, 40], 4, 2, 128, 128, 16, "bf16", False)
    d = [t.to(DEV) for t in pools]
    for bad, maxq in (([0, 12, 11], 11), ([0, 5, 12], 11), ([-1, 5, 11], 11), ([0, 5, 11], 5)):
        out = torch.full((11, 4, 128), 3.0, dtype=q.dtype, device=DEV)
        fa.sdpa_fwd_paged(q.to(DEV), d[0], d[1], table.to(DEV), kv.to(DEV), torch.tensor(bad, dtype=torch.int32, device=DEV),
                          maxq, out=out)
        torch.cuda.synchronize()
        assert fa.sdpa_check_device_status() == fa.SDPA_ERR_INVALID
        assert (out == 3).all()


@pytest.mark.parametrize("new", [[200, 90], [1] * 300])
def test_bad_offsets_where_a_kernel_of_its_own_plans(new):
    # long chunks, and more sequences than the attention kernel plans for
    q, pools, table, kv, cu = make(new, [250] * len(new), 4, 2, 128, 128, 16, "bf16", False)
    d = [t.to(DEV) for t in pools]
    cu[1] = cu[2] + 1
    out = torch.full((sum(new), 4, 128), 3.0, dtype=q.dtype, device=DEV)
    fa.sdpa_fwd_paged(q.to(DEV), d[0], d[1], table.to(DEV), kv.to(DEV), cu.to(DEV), max(new), out=out)
    torch.cuda.synchronize()
    assert fa.sdpa_check_device_status() == fa.SDPA_ERR_INVALID
    assert (out == 3).all()


@pytest.mark.parametrize("quant", [False, True])
def test_pages_outside_the_pool_read_as_zeros(quant):
    x = make([3], [64], 4, 1, 128, 128, 16, "bf16", quant)
    q, pools, table, kv, cu = x
    table[0, 1], table[0, 3] = -1, pools[0].shape[0]
    o, lse = run(*x, 3, scale=0.1, causal=False)
    k, v = (t.clone().double() for t in values(pools))
    zk = torch.cat([k, torch.zeros_like(k[:1])])
    zv = torch.cat([v, torch.zeros_like(v[:1])])
    table[0, 1] = table[0, 3] = k.shape[0]
    ref, ref_lse = oracle.sdpa_fwd_paged(q, zk, zv, table, [64], cu, scale=0.1, causal=False)
    vmax = float(torch.nan_to_num(v).abs().max())
    u_p = 2.0 ** -11 if quant else 2.0 ** -8
    assert (np.abs(o.double().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + (u_p + 2.0 ** -13) * vmax).all()
    assert np.abs(lse.cpu().numpy() - ref_lse).max() <= TOL_LSE


@pytest.mark.parametrize("quant", [False, True])
def test_streams_graph_and_repeatability(quant):
    q, pools, table, kv, cu = make([3, 70, 1], [9000, 900, 77], 8, 2, 128, 128, 64, "bf16", quant, seed=2)
    d = [t.to(DEV) for t in pools]
    args = (q.to(DEV), d[0], d[2], d[1], d[3]) if quant else (q.to(DEV), d[0], d[1])
    args += (table.to(DEV), kv.to(DEV), cu.to(DEV), 70)
    fn = fa.sdpa_fwd_paged_fp8 if quant else fa.sdpa_fwd_paged
    want, want_lse = fn(*args, causal=True)
    torch.cuda.synchronize()
    outs = []
    for _ in range(2):
        with torch.cuda.stream(torch.cuda.Stream()):
            outs += [fn(*args, causal=True) for _ in range(3)]
    torch.cuda.synchronize()
    for o, lse in outs:
        assert torch.equal(o, want) and torch.equal(lse, want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = fn(*args, causal=True)
    o.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, want_lse)
    assert fa.sdpa_check_device_status() == fa.SDPA_OK


def test_what_a_call_allocates_belongs_to_its_stream(monkeypatch):
    q, pools, table, kv, cu = make([3, 2], [900, 77], 8, 2, 128, 128, 64, "bf16", True, seed=6)
    kc, ks, vc, vs = (t.to(DEV) for t in pools)
    q, table, kv, cu = (t.to(DEV) for t in (q, table, kv, cu))
    rows = torch.tensor([0, 900, 977], dtype=torch.int32, device=DEV)
    pools16 = [oracle.dequantise_pool(*pools[i:i + 2]).to(torch.bfloat16).to(DEV) for i in (0, 2)]
    calls = [lambda **kw: fa.sdpa_fwd_paged_fp8(q, kc, vc, ks, vs, table, kv, cu, 3, causal=True, **kw),
             lambda **kw: fa.sdpa_fwd_paged(q, *pools16, table, kv, cu, 3, causal=True, **kw),
             lambda **kw: fa.sdpa_decode_paged_fp8(q[:2], kc, vc, ks, vs, table, kv, **kw),
             lambda **kw: fa.sdpa_cache_read_fp8(kc, vc, ks, vs, table, rows, 977, **kw)]
    want = [call() for call in calls]
    torch.cuda.synchronize()
    side, used, empty = torch.cuda.Stream(), [], torch.empty

    def noted(*a, **kw):
        used.append(torch.cuda.current_stream())
        return empty(*a, **kw)

    monkeypatch.setattr(torch, "empty", noted)
    got = [call(stream=side) for call in calls]
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert len(used) == 3 + 3 + 3 + 2 and all(s == side for s in used)
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


@pytest.mark.parametrize("quant", [False, True])
def test_a_wait_that_gives_up_is_reported(quant):
    x = make([3, 200], [300, 900], 8, 2, 128, 128, 64, "bf16", quant)
    fa.library().sdpa_debug_stall_next_call()
    q, pools, table, kv, cu = x
    d = [t.to(DEV) for t in pools]
    args = (q.to(DEV), d[0], d[2], d[1], d[3]) if quant else (q.to(DEV), d[0], d[1])
    fn = fa.sdpa_fwd_paged_fp8 if quant else fa.sdpa_fwd_paged
    fn(*args, table.to(DEV), kv.to(DEV), cu.to(DEV), 200, causal=True)
    torch.cuda.synchronize()
    assert fa.sdpa_check_device_status() == fa.SDPA_ERR_TIMEOUT
    o, lse = run(*x, 200, scale=128 ** -0.5, causal=True)
    check(*x, o, lse, 128 ** -0.5, True)


def test_a_quantised_cache_in_use():
    # prompts written in chunks, then single tokens: write, attend, decode and read back agree with the
    # oracle on the values the cache holds
    g = torch.Generator().manual_seed(9)
    B, Hq, Hkv, D, page, dt = 3, 8, 2, 128, 16, torch.bfloat16
    n_pages = 40
    kp, vp = (torch.zeros((n_pages, page, Hkv, D), device=DEV).to(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.zeros((n_pages, Hkv, page), device=DEV) for _ in range(2))
    table = torch.randperm(n_pages, generator=g)[:36].view(B, 12).to(torch.int32)
    lens = [0, 0, 0]
    for step in ([70, 5, 33], [30, 60, 0], [1, 1, 1]):
        lens = [a + b for a, b in zip(lens, step)]
        total = sum(step)
        k, v = (torch.randn((total, Hkv, D), generator=g).to(dt) for _ in range(2))
        q = torch.randn((total, Hq, D), generator=g).to(dt)
        kv = torch.tensor(lens, dtype=torch.int32)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(step)]), dtype=torch.int32)
        t, kvd, cud = table.to(DEV), kv.to(DEV), cu.to(DEV)
        fa.sdpa_cache_write_fp8(k.to(DEV), v.to(DEV), kp, vp, ks, vs, t, kvd, cud)
        o, lse = fa.sdpa_fwd_paged_fp8(q.to(DEV), kp, vp, ks, vs, t, kvd, cud, max(step), causal=True)
        torch.cuda.synchronize()
        pools = [x.cpu() for x in (kp, ks, vp, vs)]
        check(q, pools, table, kv, cu, o, lse, D ** -0.5, True)
        if step == [1, 1, 1]:
            od, lsed = fa.sdpa_decode_paged_fp8(q.to(DEV), kp, vp, ks, vs, t, kvd)
            torch.cuda.synchronize()
            check(q, pools, table, kv, cu, od, lsed.t().contiguous(), D ** -0.5, True)
    cuk = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    rk, rv = fa.sdpa_cache_read_fp8(kp, vp, ks, vs, table.to(DEV), cuk.to(DEV), sum(lens))
    torch.cuda.synchronize()
    for got, i in ((rk, 0), (rv, 2)):
        val = oracle.gather_pages(oracle.dequantise_pool(*pools[i:i + 2]), table, lens)
        assert torch.equal(got.double().cpu(), torch.cat([val[b, :L] for b, L in enumerate(lens)]))
    # the packed rows feed the packed prefill: the last token of each sequence sees the same keys
    o2, _ = fa.sdpa_fwd_varlen(q.to(DEV), rk, rv, torch.arange(B + 1, dtype=torch.int32, device=DEV), cuk.to(DEV), 1)
    torch.cuda.synchronize()
    assert (o2.float() - od.float()).abs().max().item() <= 2 * 2.0 ** -8 * 4.5
    assert fa.sdpa_check_device_status() == fa.SDPA_OK


def nan_workspace(q, pools, table, cu, maxq, Hkv):
    """A workspace of the full size filled with NaN: a partial that nobody wrote shows in the result."""
    n = fa.sdpa_fwd_paged_workspace_size(len(cu) - 1, q.shape[1], Hkv, q.shape[0], maxq, table.shape[1] * pools[0].shape[1],
                                         pools[-2].shape[-1] if len(pools) == 4 else pools[1].shape[-1])
    return torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("new,lens,Hq,Hkv", [([4, 0, 2], [8600, 6600, 1200], 8, 2), ([1, 0, 1], [550, 5, 3000], 1, 1),
                                             ([1, 0, 1], [550, 5, 5000], 1, 1), ([1, 0, 1], [550, 5, 8000], 1, 1)])
def test_a_cut_next_to_a_sequence_without_tokens(quant, new, lens, Hq, Hkv):
    x = make(new, lens, Hq, Hkv, 128, 128, 64, "bf16", quant, seed=21)
    ws = nan_workspace(x[0], x[1], x[2], x[4], max(new), Hkv)
    o, lse = run(*x, max(new), scale=0.09, causal=True, workspace=ws)
    check(*x, o, lse, 0.09, True)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("seed", range(6))
def test_cuts_anywhere_in_batches_with_idle_sequences(quant, seed):
    # the equal stretches of the SMs cut units next to their edges, several times, and beside sequences without
    # new tokens; odd seeds have chunks of more than a query tile, which a kernel of its own plans
    g = np.random.default_rng(40 + seed)
    B, Hkv = int(g.integers(2, 21)), [1, 2, 8][seed % 3]
    new = g.integers(1, 9 if seed % 2 == 0 else 90, B) * (g.random(B) >= 0.33)
    new[int(g.integers(B))] = 3
    lens = np.exp(g.uniform(np.log(500), np.log(6000), B)).astype(int).tolist()
    x = make(new.tolist(), lens, 4 * Hkv, Hkv, 64, 64, 64, "f16", quant, seed=seed)
    ws = nan_workspace(x[0], x[1], x[2], x[4], int(new.max()), Hkv)
    o, lse = run(*x, int(new.max()), scale=0.125, causal=True, workspace=ws)
    check(*x, o, lse, 0.125, True)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("new", [[18, 17], [300, 210]])
def test_rows_of_a_tile_without_a_token_change_nothing(quant, dtype, new):
    # 7 heads a KV head fill 126 of a tile's 128 rows; the other two hold what an earlier kernel left in shared memory,
    # here the queries of calls whose rows are all in use and whose scores are small or very large
    x = make(new, [3000, 1700], 14, 2, 128, 128, 64, dtype, quant, seed=31)
    q8, *rest = make([64, 64], [3000, 1700], 16, 2, 128, 128, 64, dtype, quant, seed=32)
    got = []
    for gain in (0.0, 1.0, 100.0):
        for _ in range(2):
            run((q8 * gain).to(q8.dtype), *rest, 64, scale=0.09, causal=True)
        got.append(run(*x, max(new), scale=0.09, causal=True))
    same = [torch.equal(o, got[0][0]) and torch.equal(lse, got[0][1]) for o, lse in got]
    assert all(same), same
    check(*x, *got[0], 0.09, True)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("new,Hq,D", [([1, 3, 8, 2], 8, 128), ([1, 40, 300, 5], 8, 128), ([7, 1, 130, 9], 4, 192)])
def test_scales_that_are_no_powers_of_two(dtype, new, Hq, D):
    # A K or V value takes two fp16 roundings, (1 + 2^-11)^2 - 1 <= r = 2^-10 + 2^-22 of itself (the factors lie in
    # [16, 128) here, so nothing is subnormal).  A score moves by at most d = r * scale * sum |q_i K_i|, so a weight by
    # e^(2 d), the output by (e^(2 d) - 1 + r) vmax beside the bound at the top, and the log-sum-exp by d.
    lens = [1, 700, 350, 90]
    q, pools, table, kv, cu = make(new, lens, Hq, 2, D, 128, 32, dtype, True, seed=51)
    g = torch.Generator().manual_seed(52)
    for i in (1, 3):  # power-of-two scales of randn rows: 2^-7 and 2^-6, now within a factor of 4 of one another
        pools[i] = torch.where(torch.isnan(pools[i]), pools[i], 2.0 ** -7 * (0.5 + 1.5 * torch.rand(pools[i].shape, generator=g)))
    o, lse = run(q, pools, table, kv, cu, max(new), scale=0.03, causal=True)
    k, v = values(pools)
    ref, ref_lse = oracle.sdpa_fwd_paged(q, k, v, table, lens, cu, scale=0.03, causal=True)
    got, got_lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    kg, vg = oracle.gather_pages(k, table, lens), oracle.gather_pages(v, table, lens)
    r, u = 2.0 ** -10 + 2.0 ** -22, torch.finfo(o.dtype).eps / 2
    for b, L in enumerate(lens):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        vmax = float(vg[b, :L].abs().max())
        kh = kg[b, :L].abs().repeat_interleave(Hq // 2, 1)  # [L, Hq, D]
        d = r * 0.03 * torch.einsum("nhd,lhd->nhl", q[rows].double().abs(), kh.double()).amax(-1).numpy()  # [n, Hq]
        tol = u * np.abs(ref[rows]) + (2.0 ** -11 + 2.0 ** -14 + 2.0 ** -16 + r + np.expm1(2 * d)[..., None]) * vmax
        assert (np.abs(got[rows] - ref[rows]) <= tol).all(), b
        seen = np.isfinite(ref_lse[:, rows])
        assert np.array_equal(np.isfinite(got_lse[:, rows]), seen)
        e = np.abs(np.where(seen, got_lse[:, rows], 0) - np.where(seen, ref_lse[:, rows], 0))
        assert (e <= TOL_LSE + d.T).all(), b
    # one visible key: the output is its V row, off by the two roundings and its own
    if new[0] == 1 and o.dtype == torch.float16:
        want = vg[0, 0].repeat_interleave(Hq // 2, 0).numpy()
        assert (np.abs(got[0] - want) <= (r + 2.0 ** -11 * (1 + r)) * np.abs(want) + 2.0 ** -25).all()


@pytest.mark.parametrize("new", [[3, 8, 1], [90, 200, 1]])
@pytest.mark.parametrize("exps", [(80,), (-80,), (-80, 0, 80)])
def test_scales_at_the_ends_of_their_range(new, exps):
    # V's scales at 2^-80, 2^80 or a mixture, K's 2^60 with the softmax scale taking it back.  Beside the bounds at the
    # top: y - m is rounded where it is below 2^7 (2^-18, twice), and the sum's logarithm, up to 100 now, carries 2^-22
    # of itself (2^-15.4); times ln 2 all that is below 2^-15.  A row under 2^-30 of its block's largest scale reads as
    # zero, far inside the 2^-16 of vmax.
    lens = [700, 1300, 77]
    q, pools, table, kv, cu = make(new, lens, 8, 2, 128, 128, 32, "bf16", True, seed=55)
    g = torch.Generator().manual_seed(56)
    pools[1] = pools[1] * 2.0 ** 60
    e = torch.tensor(exps, dtype=torch.float64)[torch.randint(len(exps), pools[3].shape, generator=g)]
    pools[3] = torch.where(torch.isnan(pools[3]), pools[3], torch.exp2(e).float())
    scale = 0.09 * 2.0 ** -60
    o, lse = run(q, pools, table, kv, cu, max(new), scale=scale, causal=True)
    k, v = values(pools)
    ref, ref_lse = oracle.sdpa_fwd_paged(q, k, v, table, lens, cu, scale=scale, causal=True)
    vg = oracle.gather_pages(v, table, lens)
    for b, L in enumerate(lens):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        vmax = float(vg[b, :L].abs().max())
        err = np.abs(o.double().cpu().numpy()[rows] - ref[rows])
        assert (err <= 2.0 ** -8 * np.abs(ref[rows]) + (2.0 ** -11 + 2.0 ** -14 + 2.0 ** -15) * vmax).all(), (b, err.max() / vmax)
        assert np.abs(lse.double().cpu().numpy()[:, rows] - ref_lse[:, rows]).max() <= TOL_LSE + 2.0 ** -15, b


def test_pages_behind_two_to_the_32_bytes():
    # the same rows in pages at the front of a small cache and at the end of pools of 4.4 GB: the same results, bit for bit
    g = torch.Generator().manual_seed(61)
    Hq, Hkv, D, page, dt = 8, 8, 128, 64, torch.bfloat16
    new, lens = [5, 70, 1], [300, 450, 64]
    n_small, n_big = 20, (1 << 32) // (page * Hkv * D) + 2000
    total = sum(lens)
    k, v = (torch.randn((total, Hkv, D), generator=g).to(dt).to(DEV) for _ in range(2))
    q = torch.randn((sum(new), Hq, D), generator=g).to(dt).to(DEV)
    kv = torch.tensor(lens, dtype=torch.int32, device=DEV)
    cu_k, cu_q = (torch.tensor(np.concatenate([[0], np.cumsum(x)]), dtype=torch.int32, device=DEV) for x in (lens, new))
    ids = torch.randperm(n_small, generator=g)[:18].to(torch.int32)
    got = []
    for n, off in ((n_small, 0), (n_big, n_big - n_small)):
        assert off == 0 or (off * page * Hkv * D) >= 1 << 32
        kp, vp = (torch.empty((n, page, Hkv, D), dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2))
        ks, vs = (torch.empty((n, Hkv, page), device=DEV) for _ in range(2))
        table = torch.full((3, 8), -1, dtype=torch.int32)
        at = 0
        for b, L in enumerate(lens):
            m = (L + page - 1) // page
            table[b, :m] = ids[at:at + m] + off
            at += m
        table = table.to(DEV)
        fa.sdpa_cache_write_fp8(k, v, kp, vp, ks, vs, table, kv, cu_k)
        out = [*fa.sdpa_cache_read_fp8(kp, vp, ks, vs, table, cu_k, total),
               *fa.sdpa_decode_paged_fp8(q[:3], kp, vp, ks, vs, table, kv),
               *fa.sdpa_fwd_paged_fp8(q, kp, vp, ks, vs, table, kv, cu_q, 70, causal=True)]
        del kp, vp, ks, vs
        # 16-bit pools of half as many pages: as many bytes
        n16, off16 = (n, 0) if off == 0 else (n // 2, n // 2 - n_small)
        pools = [torch.empty((n16, page, Hkv, D), dtype=dt, device=DEV) for _ in range(2)]
        table = torch.where(table >= 0, table - off + off16, table)
        for pool, x in zip(pools, (k, v)):
            at = 0
            for b, L in enumerate(lens):
                for i in range(0, L, page):
                    m = min(page, L - i)
                    pool[table[b, i // page].long(), :m] = x[at + i:at + i + m]
                at += L
        out += fa.sdpa_fwd_paged(q, *pools, table, kv, cu_q, 70, causal=True)
        torch.cuda.synchronize()
        assert fa.sdpa_check_device_status() == fa.SDPA_OK
        got.append(out)
        del pools
        torch.cuda.empty_cache()
    for a, b in zip(*got):
        assert torch.isfinite(a).all() and torch.equal(a, b)
