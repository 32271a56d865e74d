"""GPU tests of the quantised paged cache: written codes and scales against the fp64 oracle (bit for bit:
the scaling is exact and the code is one rounding), rows read back, and what must stay untouched."""
import numpy as np
import pytest
import torch

import flash_attention_forward_gb300 as fa
import oracle

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def _cache(lens, new, Hkv, D, Dv, page, dtype, seed=0, spare=3):
    """Empty pools (stale bytes), a page table over a random permutation, and packed new rows."""
    g = torch.Generator().manual_seed(seed)
    pages = [(L + page - 1) // page for L in lens]
    n_pages, max_pages = sum(pages) + spare, max(max(pages), 1)
    perm = torch.randperm(n_pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), max_pages), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    total = sum(new)
    rows = [torch.randn((total, Hkv, d), generator=g) * torch.exp(3 * torch.randn((total, Hkv, 1), generator=g))
            for d in (D, Dv)]
    k, v = (x.clamp(-6e4, 6e4).to(DT[dtype]) for x in rows)
    codes = [torch.randint(0, 256, (n_pages, page, Hkv, d), generator=g, dtype=torch.uint8) for d in (D, Dv)]
    scales = [torch.randn((n_pages, Hkv, page), generator=g) for _ in range(2)]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
    return k, v, codes, scales, table, torch.tensor(lens, dtype=torch.int32), cu


def _expect(x, codes, scales, table, lens, new, page):
    """Oracle pools after the write (uint8 codes)."""
    codes, scales = codes.clone(), scales.clone()
    q, s = oracle.quantise_e4m3_rows(x)
    at = 0
    for b, (L, n) in enumerate(zip(lens, new)):
        for i in range(n):
            pos = L - n + i
            p, r = int(table[b, pos // page]), pos % page
            codes[p, r] = q[at + i].view(torch.uint8)
            scales[p, :, r] = s[at + i]
        at += n
    return codes, scales


def _write(k, v, codes, scales, table, kv_len, cu, **kw):
    d = [c.to(DEV).view(torch.float8_e4m3fn) for c in codes] + [s.to(DEV) for s in scales]
    fa.sdpa_cache_write_fp8(k.to(DEV), v.to(DEV), *d, table.to(DEV), kv_len.to(DEV), cu.to(DEV), **kw)
    torch.cuda.synchronize()
    return [d[0].view(torch.uint8).cpu(), d[1].view(torch.uint8).cpu(), d[2].cpu(), d[3].cpu()]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hkv,D,Dv,page", [(8, 128, 128, 16), (2, 64, 64, 64), (1, 192, 128, 32), (3, 128, 128, 256)])
def test_write_is_the_oracle_bit_for_bit(dtype, Hkv, D, Dv, page):
    lens, new = [1, 16, 17, 300, 40, 65], [1, 16, 3, 300, 0, 7]
    k, v, codes, scales, table, kv_len, cu = _cache(lens, new, Hkv, D, Dv, page, dtype)
    k[3] = 0.0  # a row of zeros takes the smallest scale
    got = _write(k, v, codes, scales, table, kv_len, cu)
    assert fa.sdpa_check_device_status() == fa.SDPA_OK
    for x, i in ((k, 0), (v, 1)):
        want_codes, want_scales = _expect(x, codes[i], scales[i], table, lens, new, page)
        # rows that the call does not own keep their stale bytes; -0 and 0 differ in their code byte
        assert torch.equal(got[2 + i], want_scales)
        diff = got[i] != want_codes
        assert not diff.any(), f"{int(diff.sum())} codes differ"


def test_write_special_values():
    k, v, codes, scales, table, kv_len, cu = _cache([4], [4], 1, 128, 128, 16, "bf16")
    k[0], k[1], k[2], k[3] = 1.0, 1.0, 2.0 ** -100, 448.0
    k[0, 0, 5] = float("nan")
    k[1, 0, 7] = float("-inf")
    got = _write(k, v, codes, scales, table, kv_len, cu)
    p = int(table[0, 0])
    val = torch.from_numpy(oracle.dequantise_pool(got[0].view(torch.float8_e4m3fn), got[2]).numpy())[p, :4, 0]
    assert torch.isnan(val[0, 5]) and (val[0, :5] == 1).all() and (val[0, 6:] == 1).all()
    assert got[2][p, 0, 1] == 2.0 ** 120 and val[1, 7].float() == float("-inf") and (val[1, :7] == 0).all()
    assert got[2][p, 0, 2] == 2.0 ** -80 and (val[2] == 0).all()   # below half of the smallest code at 2^-80
    assert got[2][p, 0, 3] == 1.0 and (val[3] == 448).all()


def test_write_strided_rows_and_interleaved_pools():
    # k and v are halves of one packed [total, Hkv, 2 D] projection; K and V pages alternate in one pool
    lens, new, Hkv, D, page = [50, 20], [30, 20], 2, 128, 16
    k, v, codes, scales, table, kv_len, cu = _cache(lens, new, Hkv, D, D, page, "f16", seed=3)
    both = torch.cat([k, v], -1).to(DEV)
    pool = torch.stack(codes, 1).to(DEV).view(torch.float8_e4m3fn)  # [n_pages, 2, page, Hkv, D]
    wide = torch.full((2, table.shape[1] + 3), 7, dtype=torch.int32)
    wide[:, : table.shape[1]] = table
    sc = [s.to(DEV) for s in scales]
    fa.sdpa_cache_write_fp8(both[..., :D], both[..., D:], pool[:, 0], pool[:, 1], sc[0], sc[1],
                            wide.to(DEV)[:, : table.shape[1]], kv_len.to(DEV), cu.to(DEV))
    torch.cuda.synchronize()
    for x, i in ((k, 0), (v, 1)):
        want, ws = _expect(x, codes[i], scales[i], table, lens, new, page)
        assert torch.equal(pool[:, i].view(torch.uint8).cpu(), want) and torch.equal(sc[i].cpu(), ws)
    out = fa.sdpa_cache_read_fp8(pool[:, 0], pool[:, 1], sc[0], sc[1], wide.to(DEV)[:, : table.shape[1]],
                                 torch.tensor([0, 50, 70], dtype=torch.int32, device=DEV), 70, dtype=torch.float16)
    torch.cuda.synchronize()
    got = out[0][20:50].double().cpu()
    assert (got - k[:30].double()).abs().le(2.0 ** -4 * k[:30].double().abs() + 2.0 ** -10 * sc[0].cpu().max()).all()


def test_rows_without_a_slot_are_reported_and_skipped():
    # sequence 0: one new token more than rows (position -1); sequence 1: a page outside the pool;
    # sequence 2 is fine; the last packed row belongs to nobody
    lens, new, page = [3, 20, 5], [3, 2, 2], 16
    k, v, codes, scales, table, kv_len, cu = _cache(lens, new, 2, 64, 64, page, "bf16")
    extra = torch.ones((1, 2, 64), dtype=k.dtype)
    kv_len[0] = 2
    table[1, 1] = codes[0].shape[0]
    got = _write(torch.cat([k, extra]), torch.cat([v, extra]), codes, scales, table, kv_len, cu)
    assert fa.sdpa_check_device_status() == fa.SDPA_ERR_INVALID
    assert fa.sdpa_check_device_status() == fa.SDPA_OK
    q, s = oracle.quantise_e4m3_rows(k)
    want = codes[0].clone()
    for pos, row in ((0, 1), (1, 2)):
        want[int(table[0, 0]), pos] = q[row].view(torch.uint8)
    for pos, row in ((3, 5), (4, 6)):
        want[int(table[2, 0]), pos] = q[row].view(torch.uint8)
    assert torch.equal(got[0], want)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hkv,D,Dv,page", [(8, 128, 128, 64), (3, 64, 64, 16), (2, 192, 128, 128)])
def test_read_back(dtype, Hkv, D, Dv, page):
    lens = [1, 0, 16, 333, 64, 129]
    _, _, _, _, table, _, _ = _cache(lens, [0] * len(lens), Hkv, D, Dv, page, dtype, seed=9)
    n_pages = int(table.max()) + 4
    g = torch.Generator().manual_seed(2)
    # every finite code, scales that are no powers of two
    codes = [torch.randint(0, 127, (n_pages, page, Hkv, d), generator=g, dtype=torch.uint8) +
             128 * torch.randint(0, 2, (n_pages, page, Hkv, d), generator=g, dtype=torch.uint8) for d in (D, Dv)]
    scales = [torch.rand((n_pages, Hkv, page), generator=g) + 0.01 for _ in range(2)]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    total = int(cu[-1])
    outs = [torch.full((total + 2, Hkv, d), 7.0, dtype=DT[dtype], device=DEV) for d in (D, Dv)]
    f8 = [c.view(torch.float8_e4m3fn) for c in codes]
    fa.sdpa_cache_read_fp8(*(c.to(DEV) for c in f8), *(s.to(DEV) for s in scales), table.to(DEV), cu.to(DEV),
                           total + 2, k_out=outs[0], v_out=outs[1])
    torch.cuda.synchronize()
    assert fa.sdpa_check_device_status() == fa.SDPA_OK
    for i in range(2):
        val = oracle.dequantise_pool(f8[i], scales[i])
        want = torch.cat([oracle.gather_pages(val, table[b:b + 1], [L])[0, :L] for b, L in enumerate(lens)])
        got = outs[i][:total].cpu()
        # fp32 product (2^-24), then one rounding to 16 bits; code * scale <= 448 * 1.01 stays normal or is tiny
        err = (got.double() - want).abs()
        half = torch.finfo(DT[dtype]).eps / 2
        assert (err <= want.abs() * (half * (1 + 2.0 ** -11) + 2.0 ** -24) + 2.0 ** -25).all()
        assert (outs[i][total:] == 7.0).all()   # rows no sequence owns


def test_read_of_a_bad_page_is_zero_and_reported():
    codes = torch.full((2, 16, 1, 64), 0x38, dtype=torch.uint8).view(torch.float8_e4m3fn).to(DEV)
    ones = torch.ones((2, 1, 16), device=DEV)
    table = torch.tensor([[1, 9]], dtype=torch.int32, device=DEV)
    k, v = fa.sdpa_cache_read_fp8(codes, codes, ones, ones, table, torch.tensor([0, 40], dtype=torch.int32, device=DEV), 40)
    torch.cuda.synchronize()
    assert fa.sdpa_check_device_status() == fa.SDPA_ERR_INVALID   # page 9, and rows past the table
    assert (k[:16] == 1).all() and (k[16:] == 0).all() and (v[16:] == 0).all()


def test_many_sequences_and_one_token_each():
    # more sequences than one search level holds in a line, shuffled lengths, step of one token
    B, Hkv, D, page = 700, 2, 128, 16
    g = torch.Generator().manual_seed(1)
    lens = (torch.randint(1, 40, (B,), generator=g)).tolist()
    k, v, codes, scales, table, kv_len, cu = _cache(lens, [1] * B, Hkv, D, D, page, "bf16", seed=5)
    got = _write(k, v, codes, scales, table, kv_len, cu)
    want, ws = _expect(k, codes[0], scales[0], table, lens, [1] * B, page)
    assert torch.equal(got[0], want) and torch.equal(got[2], ws)


def test_large_values_beside_an_infinity_and_at_the_end_of_the_range():
    k, v, codes, scales, table, kv_len, cu = _cache([2], [2], 1, 64, 64, 16, "bf16")
    k[:], v[:] = 0.0, 0.0
    row = torch.tensor([float("-inf"), 3e38, -(2.0 ** 127), 2.0 ** 111, 1.5 * 2.0 ** 110, 2.0 ** 110, -1.0],
                       dtype=torch.float64).to(torch.bfloat16)
    k[0, 0, :7] = row
    # codes at 2^120: 225.7 -> 224, 128, the smallest (2^-9), 1.5 * 2^-10 -> 2^-9, the tie 2^-10 -> 0, 0
    want = [float("-inf"), 224 * 2.0 ** 120, -(2.0 ** 127), 2.0 ** 111, 2.0 ** 111, 0.0, 0.0]
    top = torch.tensor([247 * 2.0 ** 120, -248 * 2.0 ** 120, 255 * 2.0 ** 120], dtype=torch.float64).to(torch.bfloat16)
    assert top.double().tolist() == [247 * 2.0 ** 120, -248 * 2.0 ** 120, 255 * 2.0 ** 120]
    k[1, 0, :3] = top
    d = [c.to(DEV).view(torch.float8_e4m3fn) for c in codes] + [s.to(DEV) for s in scales]
    fa.sdpa_cache_write_fp8(k.to(DEV), v.to(DEV), *d, table.to(DEV), kv_len.to(DEV), cu.to(DEV))
    got, _ = fa.sdpa_cache_read_fp8(*d, table.to(DEV), cu.to(DEV), 2, dtype=torch.bfloat16)
    torch.cuda.synchronize()
    assert fa.sdpa_check_device_status() == fa.SDPA_OK
    assert d[2][int(table[0, 0]), 0, :2].tolist() == [2.0 ** 120] * 2
    assert got[0, 0, :7].double().cpu().tolist() == want
    assert got[1, 0, :3].double().cpu().tolist() == [240 * 2.0 ** 120, float("-inf"), float("inf")]
    assert (got[0, 0, 7:] == 0).all() and (got[1, 0, 3:] == 0).all()
