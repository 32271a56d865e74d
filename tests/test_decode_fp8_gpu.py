"""GPU parity of the decode over a quantised paged cache against the fp64 oracle on the same codes.

Tolerance.  With p_j the exact probabilities and V the dequantised values (|V| <= vmax): the kernel's
probability is rounded to fp16 (half a step, 2^-11, or absolute 2^-25 of the row's largest P V weight),
exp2 and the fp32 score carry about 2^-21 |s| (scores here stay below 2^6: 2^-15), and the output is
rounded once to its type (half a step u).  Sums are fp32.  So
    |dO| <= u |O| + (2^-11 + 2 * 2^-15 + 2^-16) vmax,   |dLSE| <= 2^-15 + 2^-16.
"""
import numpy as np
import pytest
import torch

import flash_attention_forward_gb300 as fa
import oracle
import workloads

pytestmark = pytest.mark.gpu

DEV = "cuda"
W = workloads.WORKLOADS["splitkv_decode_bf16_d128"]
TOL_P = 2.0 ** -11 + 2.0 ** -14 + 2.0 ** -16
TOL_LSE = 2.0 ** -15 + 2.0 ** -16


def make(w, lens, page, seed=11, gain=None):
    """16-bit inputs quantised into pages; rows past a length, spare pages and the scales there are NaN,
    and table entries past a sequence's pages are wild."""
    x = workloads.decode_inputs(w, kv_len=lens)
    if gain is not None:
        x["k"], x["v"] = (t.float() * gain(t) for t in (x["k"], x["v"]))
    kp, vp, table = workloads.page_caches(x["k"], x["v"], page, seed=seed, spare_pages=3)
    pools = []
    for pool in (kp, vp):
        codes, scales = oracle.quantise_pool(pool)
        nan = torch.isnan(pool).all(-1).transpose(1, 2)
        pools += [codes, torch.where(nan, torch.full_like(scales, float("nan")), scales).contiguous()]
    for b, L in enumerate(lens):
        used = (L + page - 1) // page
        wild = torch.tensor([-7, 1 << 30, kp.shape[0], 3], dtype=torch.int32).repeat(table.shape[1])
        table[b, used:] = wild[: table.shape[1] - used]
    return x, pools, table


def run(x, pools, table, scale, **kw):
    kc, ks, vc, vs = (t.to(DEV) for t in pools)
    o, lse = fa.sdpa_decode_paged_fp8(x["q"].to(DEV), kc, vc, ks, vs, table.to(DEV), x["kv_len"].to(DEV), scale=scale, **kw)
    torch.cuda.synchronize()
    assert fa.sdpa_check_device_status() == fa.SDPA_OK
    return o, lse


def check(x, pools, table, scale, o, lse):
    k, v = oracle.dequantise_pool(*pools[:2]), oracle.dequantise_pool(*pools[2:])
    ref, ref_lse = oracle.sdpa_decode_paged(x["q"], k, v, table, x["kv_len"], scale=scale)
    got = o.double().cpu().numpy()
    assert np.isfinite(got).all()
    vg = oracle.gather_pages(v, table, x["kv_len"])
    u = torch.finfo(o.dtype).eps / 2
    for b, L in enumerate(x["kv_len"].tolist()):
        vmax = float(vg[b, :L].abs().max()) if L else 0.0
        tol = u * np.abs(ref[b]) + TOL_P * vmax
        assert (np.abs(got[b] - ref[b]) <= tol).all(), (b, L, np.abs(got[b] - ref[b]).max(), vmax)
        gl, rl = lse[b].double().cpu().numpy(), ref_lse[b]
        if L:
            assert np.abs(gl - rl).max() <= TOL_LSE, (b, np.abs(gl - rl).max())
        else:
            assert np.isneginf(gl).all() and (got[b] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hq,Hkv,D,page", [(32, 8, 128, 64), (8, 8, 128, 16), (16, 2, 192, 32), (14, 2, 128, 128),
                                           (16, 1, 192, 16), (12, 1, 128, 256)])
def test_ragged_lengths_and_poisoned_rows(dtype, Hq, Hkv, D, page):
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 255, 256, 257, 1000, 2047, 2048, 2049, 4096]
    w = W.with_shape(B=len(lens), Hq=Hq, Hkv=Hkv, Sk=4096, dtype=dtype, D=D)
    x, pools, table = make(w, lens, page)
    o, lse = run(x, pools, table, w.scale)
    check(x, pools, table, w.scale, o, lse)


def test_few_sequences_take_short_splits():
    w = W.with_shape(B=1, Hq=4, Hkv=1, Sk=8192)
    x, pools, table = make(w, [8000], 64)
    o, lse = run(x, pools, table, w.scale)
    check(x, pools, table, w.scale, o, lse)


@pytest.mark.parametrize("q_gain", [2.0 ** -20, 2.0 ** 20])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rows_of_very_different_scales(dtype, q_gain):
    # V rows (and K rows) whose scales lie up to 2^+-24 apart; queries far outside fp16's normal range
    # for bf16, with the softmax scale taking the factor back
    if dtype == "f16":
        q_gain = 2.0 ** (-6 if q_gain < 1 else 6)
    lens = [700, 65, 1]
    w = W.with_shape(B=3, Hq=8, Hkv=2, Sk=1024, dtype=dtype)
    g = torch.Generator().manual_seed(8)
    x, pools, table = make(w, lens, 32, gain=lambda t: torch.exp2(torch.randint(-12, 1, t.shape[:-1], generator=g).float())[..., None])
    x["q"] = (x["q"].float() * q_gain).to(x["q"].dtype)
    o, lse = run(x, pools, table, w.scale / q_gain)
    check(x, pools, table, w.scale / q_gain, o, lse)


def test_small_values_keep_their_precision_beside_large_ones():
    # all the weight on a key whose V row is 2^-20 of the others': the output is that row
    w = W.with_shape(B=1, Hq=4, Hkv=1, Sk=256)
    x, _, _ = make(w, [200], 16)
    k = torch.zeros_like(x["k"])
    k[0, 77, 0] = 20.0
    x["q"] = torch.ones_like(x["q"])
    v = x["v"].clone()
    v[0, 200:] = 0
    v[0, 77] *= 2.0 ** -20
    kp, vp, table = workloads.page_caches(k, v, 16, seed=3)
    pools = [*oracle.quantise_pool(kp), *oracle.quantise_pool(vp)]
    o, _ = run(x, pools, table, 1.0)  # score 2560 against 0
    want = oracle.gather_pages(oracle.dequantise_pool(*pools[2:]), table, [200])[0, 77, 0]
    assert torch.equal(o[0, 0].double().cpu(), want)


def test_pages_outside_the_pool_read_as_zeros():
    w = W.with_shape(B=1, Hq=4, Hkv=1, Sk=64)
    x, pools, table = make(w, [64], 16)
    table[0, 1], table[0, 3] = -1, pools[0].shape[0]
    o, lse = run(x, pools, table, w.scale)
    k, v = (oracle.gather_pages(oracle.dequantise_pool(*p), table.clamp(0, pools[0].shape[0] - 1), [64])
            for p in (pools[:2], pools[2:]))
    for t in (k, v):
        t[0, 16:32] = 0
        t[0, 48:] = 0
    ref, ref_lse = oracle.sdpa_decode(x["q"], k, v, [64], scale=w.scale)
    vmax = float(v.abs().max())
    assert (np.abs(o.double().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + TOL_P * vmax).all()
    assert np.abs(lse.cpu().numpy() - ref_lse).max() <= TOL_LSE


def test_strided_query_and_output_and_clamped_lengths():
    w = W.with_shape(B=2, Hq=8, Hkv=2, Sk=128)
    x, pools, table = make(w, [128, 30], 16)
    wide = torch.zeros((2, 8, 256), dtype=x["q"].dtype, device=DEV)
    wide[..., 128:] = x["q"].to(DEV)
    out = torch.full((2, 8, 192), 5.0, dtype=x["q"].dtype, device=DEV)
    kc, ks, vc, vs = (t.to(DEV) for t in pools)
    kv = torch.tensor([1000000, 30], dtype=torch.int32, device=DEV)  # clamped to the table's 128 rows
    _, lse = fa.sdpa_decode_paged_fp8(wide[..., 128:], kc, vc, ks, vs, table.to(DEV), kv, scale=w.scale, out=out[..., 64:])
    torch.cuda.synchronize()
    assert (out[..., :64] == 5).all()
    check(x, pools, table, w.scale, out[..., 64:], lse)


def test_two_streams_and_a_captured_graph():
    w = W.with_shape(B=4, Hq=8, Hkv=2, Sk=512)
    x, pools, table = make(w, [512, 100, 1, 0], 64)
    kc, ks, vc, vs = (t.to(DEV) for t in pools)
    args = (x["q"].to(DEV), kc, vc, ks, vs, table.to(DEV), x["kv_len"].to(DEV))
    want, want_lse = fa.sdpa_decode_paged_fp8(*args, scale=w.scale)
    torch.cuda.synchronize()
    outs = []
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        with torch.cuda.stream(s):
            outs.append(fa.sdpa_decode_paged_fp8(*args, scale=w.scale))
    torch.cuda.synchronize()
    for o, lse in outs:
        assert torch.equal(o, want) and torch.equal(lse, want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = fa.sdpa_decode_paged_fp8(*args, scale=w.scale)
    o.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("seed", range(6))
def test_cuts_anywhere(seed):
    # batches whose equal stretches cut units everywhere: next to their edges, several times, in the last unit
    # of a sequence, behind sequences without rows
    g = torch.Generator().manual_seed(100 + seed)
    B = int(torch.randint(1, 60, (1,), generator=g))
    lens = torch.randint(0, 2000 if seed % 2 else 300, (B,), generator=g)
    lens[torch.rand(B, generator=g) < 0.3] = 0
    lens[torch.rand(B, generator=g) < 0.1] = 4096
    w = W.with_shape(B=B, Hq=8, Hkv=4 if seed < 3 else 2, Sk=4096)
    x, pools, table = make(w, lens.tolist(), 64, seed=seed)
    o, lse = run(x, pools, table, w.scale)
    check(x, pools, table, w.scale, o, lse)


@pytest.mark.parametrize("Hq,D", [(8, 128), (32, 192)])
def test_scales_that_are_no_powers_of_two(Hq, D):
    # the decode keeps the scales in fp32, so the bound at the top holds for any of them
    lens = [700, 65, 1]
    w = W.with_shape(B=3, Hq=Hq, Hkv=2, Sk=1024, D=D)
    x, pools, table = make(w, lens, 32)
    g = torch.Generator().manual_seed(53)
    for i in (1, 3):
        pools[i] = pools[i] * (0.5 + torch.rand(pools[i].shape, generator=g))
    o, lse = run(x, pools, table, w.scale)
    check(x, pools, table, w.scale, o, lse)


@pytest.mark.parametrize("exps", [(80,), (-80,), (-80, 0, 80)])
def test_scales_at_the_ends_of_their_range(exps):
    # V's scales at 2^-80, 2^80 or a mixture, K's 2^60 with the softmax scale taking it back.  Beside the bounds at the
    # top: s - m and s + log2(scale) are rounded where they are below 2^7 (2^-18, three times), and the sum's logarithm,
    # up to 90 now, carries 2^-22 of itself (2^-15.5); times ln 2 all that is below 2^-15.
    lens = [700, 65, 1]
    w = W.with_shape(B=3, Hq=8, Hkv=2, Sk=1024)
    x, pools, table = make(w, lens, 32)
    g = torch.Generator().manual_seed(54)
    pools[1] = pools[1] * 2.0 ** 60
    e = torch.tensor(exps, dtype=torch.float64)[torch.randint(len(exps), pools[3].shape, generator=g)]
    pools[3] = torch.where(torch.isnan(pools[3]), pools[3], torch.exp2(e).float())
    scale = w.scale * 2.0 ** -60
    o, lse = run(x, pools, table, scale)
    k, v = oracle.dequantise_pool(*pools[:2]), oracle.dequantise_pool(*pools[2:])
    ref, ref_lse = oracle.sdpa_decode_paged(x["q"], k, v, table, x["kv_len"], scale=scale)
    vg = oracle.gather_pages(v, table, x["kv_len"])
    for b, L in enumerate(lens):
        vmax = float(vg[b, :L].abs().max())
        err = np.abs(o[b].double().cpu().numpy() - ref[b])
        assert (err <= 2.0 ** -8 * np.abs(ref[b]) + (TOL_P + 2.0 ** -15) * vmax).all(), b
        assert np.abs(lse[b].double().cpu().numpy() - ref_lse[b]).max() <= TOL_LSE + 2.0 ** -15, b
