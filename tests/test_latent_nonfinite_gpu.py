"""GPU tests of latent attention where single queries are infinite or NaN, or their scores leave fp32's range.  Such a (token,
head) has NaN in O and LSE as soon as one of its scaled scores is NaN or +infinity; scores of -infinity are hidden keys.  The
output and the workspace hold finite values before each call, which must not come back."""
import pytest
import torch

import flash_attention_forward_gb300 as fa
from test_latent_gpu import DEV, cache, check_absorbed, check_expanded, offsets, packed

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
# what stands in dims 7 and 8 of the query, whose keys hold 1.0 and 1.0 there.  Scores of the clean queries have a standard
# deviation of 24 or 14 times the scale: after a piece's first block none passes its maximum by 2^8, so that O of a clean row
# is computed with the same running maximum whatever stands in the rows beside it
KINDS = {"inf": (INF, 0.0), "sign": (INF, -INF), "nan": (NAN, 0.0), "fp32": (2.0 ** 127, 2.0 ** 127), "scaled": (2.0 ** 127, 2.0 ** 126),
         "hidden": (-INF, 0.0)}
HIDDEN = {"hidden"}


def poison(q, rows, kind):
    q = q.clone()
    for t, h in rows:
        q[t, h] = 0.0 if kind in ("fp32", "scaled") else q[t, h]
        q[t, h, 7], q[t, h, 8] = KINDS[kind]
    return q


def clean(q, scale):
    """Queries for a scale of 1 (sixteenths: exact) or as they are."""
    q = q / 16 if scale == 1.0 else q.clone()
    q[..., 7:9] = 0.0
    return q


def check_rows(rows, kind, got, want, bitwise):
    (o, lse), (o0, lse0) = got, want
    keep = torch.ones(lse.shape, dtype=torch.bool, device=DEV)
    for t, h in rows:
        keep[h, t] = False
        if kind in HIDDEN:
            assert (o[t, h] == 0).all() and lse[h, t] == -INF, (t, h)
        else:
            assert torch.isnan(o[t, h]).all() and torch.isnan(lse[h, t]), (t, h, o[t, h], lse[h, t])
    if bitwise:
        assert torch.equal(o.transpose(0, 1)[keep], o0.transpose(0, 1)[keep]) and torch.equal(lse[keep], lse0[keep])


def absorbed_case(new, lens, Hq, kind, rows, dtype):
    scale = 1.0 if kind == "scaled" else 0.05
    q, pool, table, kv, cu = cache(new, lens, Hq, 64, dtype, seed=Hq + len(new))
    pool[..., 7:9] = torch.where(torch.isnan(pool[..., 7:9]), pool[..., 7:9], torch.ones_like(pool[..., 7:9]))
    q = clean(q, scale)
    max_kv = table.shape[1] * 64

    def call(q):
        ws = torch.zeros(fa.sdpa_fwd_latent_paged_workspace_size(len(new), Hq, q.shape[0], max(new), max_kv), dtype=torch.uint8, device=DEV)
        out = torch.full((q.shape[0], Hq, 512), 5.0, dtype=q.dtype, device=DEV)
        lse = torch.full((Hq, q.shape[0]), 5.0, device=DEV)
        fa.sdpa_fwd_latent_paged(q, pool, table, kv, cu, max(new), scale=scale, causal=True, out=out, lse=lse, workspace=ws)
        assert fa.sdpa_check_device_status() == fa.SDPA_OK
        return out, lse

    want = call(q)
    check_absorbed(q, pool, table, new, lens, *want, scale, True)
    check_rows(rows, kind, call(poison(q, rows, kind)), want, True)


# whole units, and cut ones; 16, 32 and 64 columns, two CTAs of heads; several tokens a tile
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("Hq,new,lens,rows", [(16, [1] * 6, [1, 128, 100, 64, 127, 90], [(0, 0), (1, 15), (4, 7)]),
                                              (16, [1, 1], [9000, 5000], [(0, 3), (1, 15)]), (32, [1, 1], [70, 9000], [(0, 31), (1, 0)]),
                                              (64, [1], [5000], [(0, 17), (0, 63)]), (128, [2, 1], [300, 3000], [(0, 64), (1, 127), (2, 63)]),
                                              (4, [20, 3], [2000, 100], [(0, 0), (13, 2), (22, 3)])])
def test_absorbed(kind, Hq, new, lens, rows):
    absorbed_case(new, lens, Hq, kind, rows, "bf16")


@pytest.mark.parametrize("kind", ["inf", "nan", "hidden"])   # fp16 holds no value whose scores overflow
def test_absorbed_f16(kind):
    absorbed_case([1, 3], [700, 60], 16, kind, [(0, 2), (3, 15)], "f16")


def expanded_case(new, lens, Hq, Hkv, kind, rows, dtype):
    scale = 1.0 if kind == "scaled" else 0.05
    q, k, r, v = packed(new, lens, Hq, Hkv, dtype, seed=Hq + len(new))
    k[..., 7:9] = 1.0
    q = clean(q, scale)
    cu_q, cu_k = offsets(new).to(DEV), offsets(lens).to(DEV)

    def call(q):
        size = fa.sdpa_fwd_latent_workspace_size(len(new), Hq, Hkv, q.shape[0], max(new), k.shape[0])
        out = torch.full((q.shape[0], Hq, 128), 5.0, dtype=q.dtype, device=DEV)
        lse = torch.full((Hq, q.shape[0]), 5.0, device=DEV)
        fa.sdpa_fwd_latent(q, k, r, v, cu_q, cu_k, max(new), scale=scale, causal=True, out=out, lse=lse,
                           workspace=torch.zeros(size, dtype=torch.uint8, device=DEV))
        assert fa.sdpa_check_device_status() == fa.SDPA_OK
        return out, lse

    want = call(q)
    check_expanded(q, k, r, v, new, lens, *want, scale, True)
    o, lse = call(poison(q, rows, kind))
    check_rows(rows, kind, (o, lse), want, False)
    # the others are rescaled together with the rows of their warp, so they are right within the tolerance
    for t, h in rows:
        o[t, h], lse[h, t] = want[0][t, h], want[1][h, t]
    check_expanded(q, k, r, v, new, lens, o, lse, scale, True)


# one tile a sequence (both accumulators, whole and cut), two tiles (whole and cut), a list
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("Hq,Hkv,new,lens,rows", [(4, 4, [3, 1, 60], [100, 1, 600], [(0, 0), (3, 3), (40, 1)]), (8, 1, [4, 1], [9000, 5000], [(0, 0), (4, 7)]),
                                                  (2, 2, [300, 5], [300, 700], [(0, 0), (200, 1), (299, 0), (304, 1)]), (6, 2, [500], [6000], [(0, 0), (499, 5)]),
                                                  (80, 80, [600, 1, 130, 300, 257, 900], [700, 1, 130, 900, 300, 900], [(0, 0), (600, 79), (1100, 40)])])
def test_expanded(kind, Hq, Hkv, new, lens, rows):
    expanded_case(new, lens, Hq, Hkv, kind, rows, "bf16")


@pytest.mark.parametrize("kind", ["inf", "nan", "hidden"])
def test_expanded_f16(kind):
    expanded_case([1, 3], [700, 60], 4, 4, kind, [(0, 2), (3, 3)], "f16")


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("new,lens,Hq,Hkv", [([1, 3], [700, 60], 8, 2), ([200, 5], [300, 9000], 4, 4), ([2], [20000], 4, 1)])
def test_chunks_over_pages(kind, new, lens, Hq, Hkv):
    # the same kernels over pages: one page a sequence
    scale, page = 1.0 if kind == "scaled" else 0.05, 1 << max(lens).bit_length()
    g = torch.Generator().manual_seed(Hq)
    q = clean(torch.randn((sum(new), Hq, 128), generator=g).bfloat16().to(DEV), scale)
    k, v = (torch.randn((len(new), page, Hkv, 128), generator=g).bfloat16().to(DEV) for _ in range(2))
    k[..., 7:9] = 1.0
    table = torch.arange(len(new), dtype=torch.int32, device=DEV)[:, None]
    kv, cu = torch.tensor(lens, dtype=torch.int32, device=DEV), offsets(new).to(DEV)
    rows = [(0, 0), (sum(new) - 1, Hq - 1)]
    want = fa.sdpa_fwd_paged(q, k, v, table, kv, cu, max(new), scale=scale, causal=True)
    assert torch.isfinite(want[0]).all() and torch.isfinite(want[1]).all()
    got = fa.sdpa_fwd_paged(poison(q, rows, kind), k, v, table, kv, cu, max(new), scale=scale, causal=True)
    assert fa.sdpa_check_device_status() == fa.SDPA_OK
    check_rows(rows, kind, got, want, False)
    keep = torch.ones(want[1].shape, dtype=torch.bool, device=DEV)
    for t, h in rows:
        keep[h, t] = False
    assert torch.isfinite(got[0].transpose(0, 1)[keep]).all() and torch.isfinite(got[1][keep]).all()
