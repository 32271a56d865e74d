"""GPU tests of the expanded latent attention over many short sequences, on both sides of the borders between a plan made by the
attention kernel, a line with cuts and a list; the workspace holds anything before the call.  Tolerances as in the tests of
fewer sequences."""
import numpy as np
import pytest
import torch

import flash_attention_forward_gb300 as fa
from test_latent_gpu import DEV, check_expanded, offsets, packed

pytestmark = pytest.mark.gpu


def lengths(B, most, prefix, seed):
    g = np.random.default_rng(seed)
    new = g.integers(0, most + 1, B)
    new[0] = most
    return new.tolist(), (new + g.integers(0, prefix + 1, B)).tolist()


# (new tokens, lengths), query heads, KV heads: 152 SMs take a list from 608 units on, where a sequence has more than one
# tile of 128 / (Hq / Hkv) tokens
@pytest.mark.parametrize("fill", [0, 0x11, 0xff])
@pytest.mark.parametrize("sizes,Hq,Hkv", [(lengths(300, 128, 0, 1), 16, 16), (lengths(300, 1, 60, 2), 16, 16), (lengths(257, 3, 40, 3), 128, 128),
                                          (lengths(256, 3, 40, 4), 128, 128), (([1, 3] * 600, [5, 3] * 600), 2, 2), (lengths(300, 32, 300, 5), 16, 4),
                                          (([1] * 303, [37] * 303), 2, 2), (([1] * 304, [37] * 304), 2, 2), (lengths(300, 129, 10, 6), 16, 16),
                                          (lengths(1100, 2, 3, 7), 8, 1)])
def test_many_short_sequences(sizes, Hq, Hkv, fill):
    new, lens = sizes
    q, k, r, v = packed(new, lens, Hq, Hkv, "bf16", seed=len(new))
    cu_q, cu_k = offsets(new).to(DEV), offsets(lens).to(DEV)
    ws = torch.full((fa.sdpa_fwd_latent_workspace_size(len(new), Hq, Hkv, sum(new), max(new), sum(lens)),), fill, dtype=torch.uint8, device=DEV)
    out = torch.full((sum(new), Hq, 128), float("nan"), dtype=q.dtype, device=DEV)
    lse = torch.full((Hq, sum(new)), float("nan"), dtype=torch.float32, device=DEV)
    fa.sdpa_fwd_latent(q, k, r, v, cu_q, cu_k, max(new), scale=0.07, causal=True, out=out, lse=lse, workspace=ws)
    assert fa.sdpa_check_device_status() == fa.SDPA_OK
    check_expanded(q, k, r, v, new, lens, out, lse, 0.07, True)
    # the workspace as that call left it, another batch, and the first one again
    fa.sdpa_fwd_latent(q, k, r, v, cu_q[-6:] - cu_q[-6], cu_k[-6:] - cu_k[-6], max(new), scale=0.07, causal=True, workspace=ws)
    again, lse2 = fa.sdpa_fwd_latent(q, k, r, v, cu_q, cu_k, max(new), scale=0.07, causal=True, workspace=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_captured_call_of_many_short_sequences():
    new, lens = lengths(300, 5, 90, 8)
    q, k, r, v = packed(new, lens, 8, 8, "f16", seed=8)
    cu_q, cu_k = offsets(new).to(DEV), offsets(lens).to(DEV)
    want = [t.clone() for t in fa.sdpa_fwd_latent(q, k, r, v, cu_q, cu_k, 5, causal=True)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = fa.sdpa_fwd_latent(q, k, r, v, cu_q, cu_k, 5, causal=True)
    for _ in range(2):
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert fa.sdpa_check_device_status() == fa.SDPA_OK


def test_two_lists_at_once_and_in_two_graphs():
    # the list's counter lies in each call's own workspace
    new, lens = [600, 1, 130, 300, 0, 257, 900, 40], [700, 1, 130, 900, 9, 100, 900, 300]
    q, k, r, v = packed(new, lens, 80, 80, "bf16", seed=9)
    cu_q, cu_k = offsets(new).to(DEV), offsets(lens).to(DEV)
    call = lambda s=None: fa.sdpa_fwd_latent(q, k, r, v, cu_q, cu_k, max(new), scale=0.07, causal=True, stream=s)
    want = [t.clone() for t in call()]
    check_expanded(q, k, r, v, new, lens, *want, 0.07, True)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [call(s) for s in (s1, s2) * 4]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, call()))
    for _ in range(3):
        for s, (g, out) in zip((s1, s2), graphs):
            with torch.cuda.stream(s):
                for t in out:
                    t.zero_()
                g.replay()
    torch.cuda.synchronize()
    for o, lse in got + [out for _, out in graphs]:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert fa.sdpa_check_device_status() == fa.SDPA_OK
