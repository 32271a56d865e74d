"""GPU tests of latent attention against the definition in 64 bits.

Tolerance, as for the chunk attention over paged caches: the probabilities are rounded to the type (half a step u),
the row sums are fp32 of the unrounded ones, exp2 and the fp32 score carry 2^-21 |s| (scores below 2^6 here: 2^-15, twice:
numerator and sum), and the output is rounded once (u).  With |V| <= vmax over the visible keys
    |dO| <= u |O| + (u + 2^-14 + 2^-16) vmax,   |dLSE| <= 2^-15 + 2^-16."""
import numpy as np
import pytest
import torch

import flash_attention_forward_gb300 as fa

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
TOL_LSE = 2.0 ** -15 + 2.0 ** -16
NEW = [1, 3, 0, 33, 64, 130, 5, 20, 1, 2]
LENS = [1, 3, 5, 33, 700, 131, 127, 128, 129, 1500]


def offsets(n):
    return torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32)


def attention(q, k, v, scale, causal):
    """One sequence in 64 bits: q [n, H, D], k [L, H, D], v [L, H, Dv]; the queries are the last positions."""
    q, k, v = (x.double().to(DEV) for x in (q, k, v))
    n, L = q.shape[0], k.shape[0]
    if n == 0 or L == 0:
        return torch.zeros(n, q.shape[1], v.shape[2], dtype=torch.float64, device=DEV), torch.full((q.shape[1], n), -float("inf"), device=DEV).double()
    s = torch.einsum("nhd,lhd->hnl", q, k) * scale
    if causal:
        hide = torch.arange(L, device=DEV) > torch.arange(L - n, L, device=DEV)[:, None]
        s = s.masked_fill(hide, -float("inf"))
    lse = torch.logsumexp(s, -1)
    p = torch.where(torch.isneginf(lse)[..., None], 0.0, torch.exp(s - lse[..., None]))
    return torch.einsum("hnl,lhd->nhd", p, v), lse


def check(o, lse, ref, ref_lse, vmax):
    u = torch.finfo(o.dtype).eps / 2
    got = o.double()
    assert torch.isfinite(got).all()
    err = (got - ref).abs()
    assert (err <= u * ref.abs() + (u + 2.0 ** -14 + 2.0 ** -16) * vmax).all(), float(err.max())
    dead = torch.isneginf(ref_lse)
    assert torch.equal(torch.isneginf(lse.double()), dead)
    assert (got[dead.T] == 0).all()
    e = (lse.double() - ref_lse).abs()[~dead]
    assert e.numel() == 0 or e.max() <= TOL_LSE, float(e.max())


# ---------------------------------------------------------------- expanded


def packed(new, lens, Hq, Hkv, dtype, seed=0, holes=False):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    q = torch.randn((sum(new), Hq, 192), generator=g).to(dt).to(DEV)
    both = torch.randn((max(1, sum(lens)), Hkv, 256), generator=g).to(dt).to(DEV)
    r = torch.randn((max(1, sum(lens)), 64), generator=g).to(dt).to(DEV)
    return q, both[..., :128], r, both[..., 128:]


def check_expanded(q, k, r, v, new, lens, o, lse, scale, causal, q0=0, k0=0):
    G = q.shape[1] // k.shape[1]
    at, at_k = q0, k0
    for n, L in zip(new, lens):
        kk = torch.cat([k[at_k:at_k + L], r[at_k:at_k + L, None].expand(L, k.shape[1], 64)], -1).repeat_interleave(G, 1)
        vv = v[at_k:at_k + L].repeat_interleave(G, 1)
        ref, ref_lse = attention(q[at:at + n], kk, vv, scale, causal)
        check(o[at:at + n], lse[:, at:at + n], ref, ref_lse, float(vv.abs().max()) if L else 0.0)
        at, at_k = at + n, at_k + L


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (6, 2), (1, 1), (16, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_expanded(dtype, Hq, Hkv, causal):
    q, k, r, v = packed(NEW, LENS, Hq, Hkv, dtype, seed=Hq)
    o, lse = fa.sdpa_fwd_latent(q, k, r, v, offsets(NEW).to(DEV), offsets(LENS).to(DEV), max(NEW), scale=0.08, causal=causal)
    assert fa.sdpa_check_device_status() == fa.SDPA_OK
    check_expanded(q, k, r, v, NEW, LENS, o, lse, 0.08, causal)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("new,lens,Hq,Hkv", [([4, 1, 0, 8, 3], [3000, 1, 700, 127, 5000], 16, 1), ([128, 5], [1024, 128], 3, 3),
                                             ([5, 9, 2], [3, 0, 1], 2, 2), ([1000], [4000], 8, 8), ([1] * 300, [37] * 300, 2, 2)])
def test_expanded_short_chunks_cuts_and_queries_without_keys(dtype, new, lens, Hq, Hkv):
    # one query tile and more, cut key ranges, more queries than keys, an empty sequence
    q, k, r, v = packed(new, lens, Hq, Hkv, dtype, seed=len(new))
    o, lse = fa.sdpa_fwd_latent(q, k, r, v, offsets(new).to(DEV), offsets(lens).to(DEV), max(new), causal=True)
    assert fa.sdpa_check_device_status() == fa.SDPA_OK
    check_expanded(q, k, r, v, new, lens, o, lse, 192 ** -0.5, True)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,lens,H", [([600, 1, 130, 300, 0, 257, 900, 40], [700, 1, 130, 900, 9, 100, 900, 300], 80),
                                        ([129] + [1, 3] * 600, [129] + [5, 3] * 600, 2)])
def test_expanded_many_units(causal, new, lens, H):
    # whole units from a list, some heads at a time; and more tiles than the plan sorts
    q, k, r, v = packed(new, lens, H, H, "bf16", seed=H)
    cu_q, cu_k = offsets(new).to(DEV), offsets(lens).to(DEV)
    o, lse = fa.sdpa_fwd_latent(q, k, r, v, cu_q, cu_k, max(new), scale=0.07, causal=causal)
    assert fa.sdpa_check_device_status() == fa.SDPA_OK
    check_expanded(q, k, r, v, new, lens, o, lse, 0.07, causal)
    o2, lse2 = fa.sdpa_fwd_latent(q, k, r, v, cu_q, cu_k, max(new), scale=0.07, causal=causal)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_expanded_other_sequences_rows_and_the_rest_of_the_output():
    # rows no sequence owns, and the other sequences', may be NaN; the output's are left as they are
    new, lens = [3, 70, 2], [200, 70, 129]
    q, k, r, v = (x.clone() for x in packed([2] + new + [3], [5] + lens + [130], 2, 2, "bf16"))
    cu_q, cu_k = offsets(new) + 2, offsets(lens) + 5
    for x, cu in ((q, cu_q), (k, cu_k), (r, cu_k), (v, cu_k)):
        x[:int(cu[0])] = float("nan")
        x[int(cu[-1]):] = float("nan")
    out = torch.full((q.shape[0], 2, 128), 9.0, dtype=q.dtype, device=DEV)
    o, lse = fa.sdpa_fwd_latent(q, k, r, v, cu_q.to(DEV), cu_k.to(DEV), 70, causal=True, out=out)
    check_expanded(q, k, r, v, new, lens, o, lse, 192 ** -0.5, True, 2, 5)
    assert (out[:2] == 9).all() and (out[-3:] == 9).all()
    # NaN in the middle sequence stays there
    want = o.clone(), lse.clone()
    for x in (k, r, v):
        x[205:275] = float("nan")
    o, lse = fa.sdpa_fwd_latent(q, k, r, v, cu_q.to(DEV), cu_k.to(DEV), 70, causal=True)
    for rows in (slice(2, 5), slice(75, 77)):
        assert torch.equal(o[rows], want[0][rows]) and torch.equal(lse[:, rows], want[1][:, rows])


def test_expanded_past_32_bits():
    # the sequences' rows lie behind 2^32 bytes, and 2^31 values, of every tensor with heads
    H, new, lens = 128, [40, 1, 300], [40, 700, 301]
    total = (1 << 31) // (H * 128) + 1100
    q, k, r, v = packed(new, lens, H, H, "bf16", seed=3)
    wide_q = torch.empty((total, H, 192), dtype=q.dtype, device=DEV)
    wide_kv = torch.empty((total, H, 256), dtype=q.dtype, device=DEV)
    wide_r = torch.empty((total, 64), dtype=q.dtype, device=DEV)
    q0, k0 = total - sum(new), total - sum(lens)
    wide_q[q0:], wide_kv[k0:, :, :128], wide_kv[k0:, :, 128:], wide_r[k0:] = q, k, v, r
    out = torch.full((total, H, 128), 9.0, dtype=q.dtype, device=DEV)
    cu_q, cu_k = offsets(new) + q0, offsets(lens) + k0
    o, lse = fa.sdpa_fwd_latent(wide_q, wide_kv[..., :128], wide_r, wide_kv[..., 128:], cu_q.to(DEV), cu_k.to(DEV), 300,
                                scale=0.07, causal=True, out=out)
    assert fa.sdpa_check_device_status() == fa.SDPA_OK
    check_expanded(q, k, r, v, new, lens, o[q0:], lse[:, q0:], 0.07, True)
    assert (out[:q0] == 9).all()


def test_expanded_equals_the_packed_prefill_with_repeated_keys():
    # equal lengths: bottom-right and top-left masking are one; the same problem with the shared part repeated
    lens = [300, 17, 1000]
    q, k, r, v = packed(lens, lens, 4, 4, "bf16", seed=5)
    cu = offsets(lens).to(DEV)
    o, lse = fa.sdpa_fwd_latent(q, k, r, v, cu, cu, 1000, causal=True)
    full = torch.cat([k, r[:, None].expand(-1, 4, -1)], -1)
    o2, lse2 = fa.sdpa_fwd_varlen(q, full, v, cu, cu, 1000, causal=True)
    vmax = float(v.abs().max())
    assert ((o.double() - o2.double()).abs() <= 2 * (2.0 ** -8 * o2.double().abs() + (2.0 ** -8 + 2.0 ** -13) * vmax)).all()
    assert (lse - lse2).abs().max() <= 2 * TOL_LSE


@pytest.mark.parametrize("cu_q,cu_k", [([0, 5, 4], [0, 9, 20]), ([0, 5, 9], [0, 21, 20]), ([0, 5, 9], [0, 9, 41]), ([-1, 5, 9], [0, 9, 20]),
                                       ([0, 8, 9], [0, 9, 20])])
@pytest.mark.parametrize("maxq", [7, 200])
def test_expanded_bad_offsets_store_nothing(cu_q, cu_k, maxq):
    if maxq == 200 and cu_q == [0, 8, 9]:
        cu_q = [0, 8, 999]
    q, k, r, v = packed([max(9, maxq)], [40], 1, 1, "bf16")
    out = torch.full((q.shape[0], 1, 128), 3.0, dtype=q.dtype, device=DEV)
    t = [torch.tensor(c, dtype=torch.int32, device=DEV) for c in (cu_q, cu_k)]
    fa.sdpa_fwd_latent(q, k, r, v, *t, maxq, causal=True, out=out)
    assert fa.sdpa_check_device_status() == fa.SDPA_ERR_INVALID
    assert (out == 3).all()


def test_expanded_without_room_for_partials_and_repeatable():
    new, lens = [4, 1], [9000, 5000]
    q, k, r, v = packed(new, lens, 8, 1, "bf16", seed=3)
    cu_q, cu_k = offsets(new).to(DEV), offsets(lens).to(DEV)
    a = fa.sdpa_fwd_latent(q, k, r, v, cu_q, cu_k, 4)
    small = torch.empty(fa.sdpa_fwd_latent_workspace_size(2, 8, 1, 5, 4, 1), dtype=torch.uint8, device=DEV)
    b = fa.sdpa_fwd_latent(q, k, r, v, cu_q, cu_k, 4, workspace=small)
    for o, lse in (a, b):
        check_expanded(q, k, r, v, new, lens, o, lse, 192 ** -0.5, False)
    c = fa.sdpa_fwd_latent(q, k, r, v, cu_q, cu_k, 4)
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])


# ---------------------------------------------------------------- absorbed


def cache(new, lens, Hq, page, dtype, seed=0, spare=2):
    """Packed queries and a latent cache: rows past a length and spare pages are NaN, table entries past a sequence's
    pages are wild."""
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    pages = [(max(L, 0) + page - 1) // page for L in lens]
    n_pages, max_pages = sum(pages) + spare, max(max(pages), 1) + 1
    perm = torch.randperm(n_pages, generator=g).to(torch.int32)
    wild = torch.tensor([-7, 1 << 30, n_pages, 3], dtype=torch.int32)
    table = wild[torch.arange(len(lens) * max_pages) % 4].view(len(lens), max_pages).clone()
    pool = torch.full((n_pages, page, 576), float("nan"), dtype=dt)
    at = 0
    for b, L in enumerate(lens):
        ids = perm[at:at + pages[b]]
        table[b, :pages[b]] = ids
        at += pages[b]
        rows = torch.full((pages[b] * page, 576), float("nan"), dtype=dt)
        rows[:max(L, 0)] = torch.randn((max(L, 0), 576), generator=g).to(dt)
        pool[ids.long()] = rows.view(pages[b], page, 576)
    q = torch.randn((max(1, sum(new)), Hq, 576), generator=g).to(dt)
    return [t.to(DEV) for t in (q, pool, table, torch.tensor(lens, dtype=torch.int32), offsets(new))]


def rows_of(pool, table, b, L):
    page = pool.shape[1]
    t = torch.arange(L, device=DEV)
    return pool.view(-1, 576)[table[b].long()[t // page] * page + t % page]


def check_absorbed(q, pool, table, new, lens, o, lse, scale, causal, q0=0):
    at = q0
    for b, (n, L) in enumerate(zip(new, lens)):
        L = max(L, 0)
        x = rows_of(pool, table, b, L)[:, None]
        step = max(1, (1 << 27) // max(1, q.shape[1] * L))
        vmax = float(x[..., :512].abs().max()) if L else 0.0
        for i in range(0, n, step):
            m = min(step, n - i)
            # the last m of the positions up to the last of these tokens
            vis = L - n + i + m if causal else L
            if vis <= 0 and causal:
                ref = torch.zeros(m, q.shape[1], 512, dtype=torch.float64, device=DEV)
                ref_lse = torch.full((q.shape[1], m), -float("inf"), dtype=torch.float64, device=DEV)
            else:
                xs = x[:vis].expand(-1, q.shape[1], -1)
                ref, ref_lse = attention(q[at + i:at + i + m], xs, xs[..., :512], scale, causal)
            check(o[at + i:at + i + m], lse[:, at + i:at + i + m], ref, ref_lse, vmax)
        at += n


def absorbed(args, new, lens, scale=0.05, causal=True, **kw):
    q, pool, table, kv, cu = args
    o, lse = fa.sdpa_fwd_latent_paged(q, pool, table, kv, cu, max(new), scale=scale, causal=causal, **kw)
    assert fa.sdpa_check_device_status() == fa.SDPA_OK
    check_absorbed(q, pool, table, new, lens, o, lse, scale, causal)
    return o, lse


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hq,page", [(16, 64), (1, 16), (20, 128), (32, 32), (5, 256), (64, 64), (128, 16), (96, 64), (37, 128)])
def test_absorbed_decode(dtype, Hq, page):
    lens = [1, 127, 128, 129, 0, 700, 64, 1500, 16, 385]
    absorbed(cache([1] * 10, lens, Hq, page, dtype, seed=Hq), [1] * 10, lens)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,page", [(16, 64), (3, 16), (40, 128), (128, 64), (65, 32)])
def test_absorbed_chunks(dtype, causal, Hq, page):
    absorbed(cache(NEW, LENS, Hq, page, dtype, seed=Hq + 1), NEW, LENS, causal=causal)


@pytest.mark.parametrize("new,lens,Hq", [([4, 1, 0, 8, 3], [30000, 1, 700, 127, 5000], 16), ([1, 1], [70000, 3], 128), ([1], [5000], 64),
                                         ([5, 9, 2, 0, 1], [3, 0, 1, 50, -4], 8), ([1] * 300, [137] * 300, 32), ([300], [9000], 24)])
def test_absorbed_cuts_short_caches_and_many_sequences(new, lens, Hq):
    absorbed(cache(new, lens, Hq, 64, "bf16", seed=len(new)), new, lens)


def test_absorbed_rescales_as_the_maximum_grows():
    # scores grow along the keys, by more than 2^8 again and again, and differently in every column
    args = cache([1, 1], [2000, 2000], 32, 64, "bf16", seed=4)
    q, pool, table = args[:3]
    q[:] = 0.0
    q[:, :, 512] = torch.linspace(0.0, 8.0, 32, device=DEV).to(q.dtype)
    for b in range(2):
        t = torch.arange(2000, device=DEV)
        flat = table[b].long()[t // 64] * 64 + t % 64
        pool.view(-1, 576)[flat, 512] = (t / 32.0 if b == 0 else (2000 - t) / 32.0).to(q.dtype)
    # scores reach 8 * 62 * 0.05 = 25 natural units: 36 powers of two
    absorbed(args, [1, 1], [2000, 2000])


def test_absorbed_other_sequences_rows_and_the_rest_of_the_output():
    new, lens = [3, 70, 2], [200, 70, 129]
    for Hq in (4, 128):
        q, pool, table, kv, cu = cache([2] + new + [3], [5] + lens + [130], Hq, 16, "bf16")
        q[:2], q[-3:] = float("nan"), float("nan")
        cu, kv, table = cu[1:-1].contiguous(), kv[1:-1].contiguous(), table[1:-1]
        out = torch.full((q.shape[0], Hq, 512), 9.0, dtype=q.dtype, device=DEV)
        o, lse = fa.sdpa_fwd_latent_paged(q, pool, table, kv, cu, 70, scale=0.05, causal=True, out=out)
        assert fa.sdpa_check_device_status() == fa.SDPA_OK
        check_absorbed(q, pool, table, new, lens, o, lse, 0.05, True, 2)
        assert (out[:2] == 9).all() and (out[-3:] == 9).all()
        # the results of a sequence do not depend on what the others hold
        o, lse = o.clone(), lse.clone()
        q[5:75] = float("nan")
        o2, lse2 = fa.sdpa_fwd_latent_paged(q, pool, table, kv, cu, 70, scale=0.05, causal=True)
        for rows in (slice(2, 5), slice(75, 77)):
            assert torch.equal(o[rows], o2[rows]) and torch.equal(lse[:, rows], lse2[:, rows])


def test_absorbed_strides_streams_and_no_lse():
    new, lens, Hq = [2, 5], [300, 77], 8
    q, pool, table, kv, cu = cache(new, lens, Hq, 32, "f16")
    wide_q = torch.full((7, Hq + 1, 640), float("nan"), dtype=q.dtype, device=DEV)
    wide_q[:, :Hq, :576] = q
    wide_pool = torch.full((pool.shape[0], 33, 584), float("nan"), dtype=q.dtype, device=DEV)
    wide_pool[:, :32, :576] = pool
    wide_table = torch.full((2, table.shape[1] + 3), 1, dtype=torch.int32, device=DEV)
    wide_table[:, :table.shape[1]] = table
    wide_out = torch.full((7, Hq + 2, 520), 4.0, dtype=q.dtype, device=DEV)
    want = fa.sdpa_fwd_latent_paged(q, pool, table, kv, cu, 5, scale=0.05, causal=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o, lse = fa.sdpa_fwd_latent_paged(wide_q[:, :Hq, :576], wide_pool[:, :32, :576], wide_table[:, :table.shape[1]], kv, cu, 5,
                                      scale=0.05, causal=True, out=wide_out[:, :Hq, :512], return_lse=False, stream=s)
    s.synchronize()
    assert lse is None and torch.equal(o, want[0])
    wide_out[:, :Hq, :512] = 4.0
    assert (wide_out == 4.0).all()


@pytest.mark.parametrize("Hq", [16, 128])
def test_absorbed_bad_offsets_store_nothing(Hq):
    q, pool, table, kv, cu = cache([5, 4], [100, 100], Hq, 64, "bf16")
    for bad, maxq in (([0, 5, 4], 5), ([0, 5, 10], 5), ([-1, 5, 9], 9), ([0, 5, 9], 4)):
        out = torch.full((9, Hq, 512), 3.0, dtype=q.dtype, device=DEV)
        fa.sdpa_fwd_latent_paged(q, pool, table, kv, torch.tensor(bad, dtype=torch.int32, device=DEV), maxq, scale=0.05, out=out)
        assert fa.sdpa_check_device_status() == fa.SDPA_ERR_INVALID
        assert (out == 3).all()


def test_absorbed_bad_pages_read_as_zeros():
    q, pool, table, kv, cu = cache([1, 1], [300, 40], 16, 64, "bf16")
    table[0, 2], table[0, 3] = -1, pool.shape[0]
    o, lse = fa.sdpa_fwd_latent_paged(q, pool, table, kv, cu, 1, scale=0.05)
    assert fa.sdpa_check_device_status() == fa.SDPA_OK
    rows = torch.cat([rows_of(pool, table, 0, 128), torch.zeros(128, 576, dtype=q.dtype, device=DEV),
                      pool[int(table[0, 4]), :44]])
    ref, ref_lse = attention(q[:1], rows[:, None].expand(-1, 16, -1), rows[:, None, :512].expand(-1, 16, -1), 0.05, False)
    check(o[:1], lse[:, :1], ref, ref_lse, float(rows.abs().max()))


def test_absorbed_without_room_for_partials_and_repeatable():
    new, lens = [2, 1], [9000, 5000]
    for Hq in (16, 128):
        args = cache(new, lens, Hq, 64, "bf16", seed=3)
        a = absorbed(args, new, lens)
        small = torch.empty(fa.sdpa_fwd_latent_paged_workspace_size(2, Hq, 3, 2, 1), dtype=torch.uint8, device=DEV)
        absorbed(args, new, lens, workspace=small)
        c = absorbed(args, new, lens)
        assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])


def test_absorbed_pages_past_32_bits():
    # the sequences' pages lie behind 2^32 bytes of their pool
    page = 64
    n_pages = (1 << 32) // (576 * 2 * page) + 40
    pool = torch.empty((n_pages, page, 576), dtype=torch.bfloat16, device=DEV)
    pool[:40] = float("nan")
    g = torch.Generator().manual_seed(2)
    rows = torch.randn((36 * page, 576), generator=g).to(torch.bfloat16).to(DEV)
    ids = torch.randperm(36, generator=g)
    pool[n_pages - 36:] = rows.view(36, page, 576)[ids]
    table = torch.empty(36, dtype=torch.int32)
    table[ids] = torch.arange(n_pages - 36, n_pages, dtype=torch.int32)   # logical page i lies where ids is i
    q = torch.randn((3, 16, 576), generator=g).to(torch.bfloat16).to(DEV)
    new, lens = [1, 2], [20 * page - 5, 16 * page]
    table2 = torch.full((2, 20), -1, dtype=torch.int32)
    table2[0], table2[1, :16] = table[:20], table[20:]
    table2, kv, cu = table2.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), offsets(new).to(DEV)
    o, lse = fa.sdpa_fwd_latent_paged(q, pool, table2, kv, cu, 2, scale=0.05, causal=True)
    assert fa.sdpa_check_device_status() == fa.SDPA_OK
    check_absorbed(q, pool, table2, new, lens, o, lse, 0.05, True)


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_captured_calls_replay(form):
    if form == "absorbed":
        args = cache([3, 1, 40], [500, 9, 3000], 16, 64, "bf16")
        call = lambda: fa.sdpa_fwd_latent_paged(*args, 40, scale=0.05, causal=True)
    else:
        q, k, r, v = packed([300, 5], [700, 5], 16, 16, "bf16")
        cu_q, cu_k = offsets([300, 5]).to(DEV), offsets([700, 5]).to(DEV)
        call = lambda: fa.sdpa_fwd_latent(q, k, r, v, cu_q, cu_k, 300, causal=True)
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):   # each with a workspace of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, call()))
    for g, out in graphs + graphs:
        for t in out:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    assert fa.sdpa_check_device_status() == fa.SDPA_OK


@pytest.mark.parametrize("form,Hq", [("absorbed", 16), ("absorbed", 128), ("expanded", 2), ("expanded", 16)])
def test_stalled_load_times_out_and_context_survives(form, Hq):
    # the test hook withholds the first slots of one launch: every wait gives up, and the next call is right
    if form == "absorbed":
        new, lens = [1, 1], [900, 400]
        args = cache(new, lens, Hq, 64, "bf16")
        call = lambda: fa.sdpa_fwd_latent_paged(*args, 1, scale=0.05, causal=True)
    else:
        new, lens = ([300, 60], [500, 500]) if Hq == 2 else ([100, 60], [500, 500])
        q, k, r, v = packed(new, lens, Hq, Hq, "bf16")
        cu_q, cu_k = offsets(new).to(DEV), offsets(lens).to(DEV)
        call = lambda: fa.sdpa_fwd_latent(q, k, r, v, cu_q, cu_k, max(new), scale=0.05, causal=True)
    assert fa.sdpa_check_device_status() == fa.SDPA_OK
    assert fa.library().sdpa_debug_stall_next_call() == fa.SDPA_OK
    call()
    assert fa.sdpa_check_device_status() == fa.SDPA_ERR_TIMEOUT
    assert fa.sdpa_check_device_status() == fa.SDPA_OK
    o, lse = call()
    assert fa.sdpa_check_device_status() == fa.SDPA_OK
    if form == "absorbed":
        check_absorbed(args[0], args[1], args[2], new, lens, o, lse, 0.05, True)
    else:
        check_expanded(q, k, r, v, new, lens, o, lse, 0.05, True)
