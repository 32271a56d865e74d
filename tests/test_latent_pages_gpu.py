"""GPU tests of the absorbed latent attention over page tables with entries outside the pool, at every number of columns: with
64 the next block is fetched ahead by the same entries.  Such a page reads as rows of zeros."""
import pytest
import torch

import flash_attention_forward_gb300 as fa
from test_latent_gpu import DEV, attention, cache, check, rows_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq", [4, 32, 64, 128])
@pytest.mark.parametrize("page", [16, 64, 128, 256])
def test_entries_outside_the_pool(Hq, page):
    lens = [5 * 256 + 40, 3 * 256, 9]
    q, pool, table, kv, cu = cache([2, 1, 1], lens, Hq, page, "bf16", seed=Hq + page)
    zeros = torch.zeros((1, page, 576), dtype=q.dtype, device=DEV)
    wild = [-1, pool.shape[0], -(1 << 31), (1 << 31) - 1, -pool.shape[0], pool.shape[0] + 1]
    n_pages, whole = pool.shape[0], torch.cat([pool, zeros])
    ref_table = table.clone()
    at = 0
    for b, L in enumerate(lens):
        for i in range(b, L // page, 3):   # whole pages, the first and last blocks' among them
            table[b, i], ref_table[b, i] = wild[at % 6], n_pages
            at += 1
    assert at >= 3
    o, lse = fa.sdpa_fwd_latent_paged(q, pool, table, kv, cu, 2, scale=0.05, causal=True)
    assert fa.sdpa_check_device_status() == fa.SDPA_OK
    at = 0
    for b, (n, L) in enumerate(zip([2, 1, 1], lens)):
        x = rows_of(whole, ref_table, b, L)[:, None].expand(-1, Hq, -1)
        ref, ref_lse = attention(q[at:at + n], x, x[..., :512], 0.05, True)
        check(o[at:at + n], lse[:, at:at + n], ref, ref_lse, float(x.abs().max()))
        at += n
