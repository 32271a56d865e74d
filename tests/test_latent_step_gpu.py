"""A serving loop over a latent cache: pages, positions, writes and attention of one step after the other, and the expanded
form as a second way to the same outputs."""
import pytest
import torch

import flash_attention_forward_gb300 as fa

pytestmark = pytest.mark.gpu

DEV = "cuda"
H, NOPE, ROT, LATENT, VDIM = 4, 128, 64, 512, 128
SCALE = (NOPE + ROT) ** -0.5


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Loop:
    """Sequences that grow and shrink: the cache of the library, and every row ever written, kept apart."""

    def __init__(self, B, page, n_pages, width, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.g, self.B, self.page = g, B, page
        self.table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
        self.kv_len, self.n_free = ints([0] * B), ints([n_pages])
        self.free = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
        self.pool = torch.full((n_pages, page, LATENT + ROT), float("nan"), dtype=torch.bfloat16, device=DEV)
        # small weights, so that the expanded keys and values are of the size of the latent vectors
        self.w_k = self.rand(H, NOPE, LATENT) * LATENT ** -0.5
        self.w_v = self.rand(H, VDIM, LATENT) * LATENT ** -0.5
        self.inv_freq = fa.sdpa_rope_frequencies(ROT, scaling="by_parts", factor=8.0, original_length=512)[0].to(DEV)
        self.rows = [torch.zeros(0, LATENT + ROT, dtype=torch.bfloat16, device=DEV) for _ in range(B)]

    def rand(self, *shape):
        return torch.randn(shape, generator=self.g, device=DEV)

    def step(self, change):
        new = [max(d, 0) for d in change]
        total = sum(new)
        self.kv_len, self.n_free, cu, positions, slots = fa.sdpa_cache_resize(
            self.table, self.kv_len, ints(change), self.free, self.n_free, self.page, max(total, 1))
        c, k_rope = self.rand(max(total, 1), LATENT).bfloat16(), self.rand(max(total, 1), ROT).bfloat16()
        q_nope, q_rope = self.rand(max(total, 1), H, NOPE).bfloat16(), self.rand(max(total, 1), H, ROT).bfloat16()
        q = torch.empty(max(total, 1), H, LATENT + ROT, dtype=torch.bfloat16, device=DEV)
        q[..., :LATENT] = torch.einsum("thn,hnl->thl", q_nope.float(), self.w_k).bfloat16()
        fa.sdpa_rope(q_rope, None, positions, self.inv_freq, q_out=q[..., LATENT:])
        fa.sdpa_latent_write(c, k_rope, self.pool, slots, positions, self.inv_freq)
        o = lse = None
        if total:
            o, lse = fa.sdpa_fwd_latent_paged(q, self.pool, self.table, self.kv_len, cu, max(new), scale=SCALE, causal=True)
        assert fa.sdpa_check_device_status() == fa.SDPA_OK
        # the same rows, without the library
        at = 0
        for b, d in enumerate(change):
            if d < 0:
                self.rows[b] = self.rows[b][:d]
                continue
            n0 = self.rows[b].shape[0]
            angle = torch.arange(n0, n0 + d, device=DEV).double()[:, None] * self.inv_freq.double()
            x, y = k_rope[at:at + d].double().split(ROT // 2, -1)
            turned = torch.cat([x * angle.cos() - y * angle.sin(), y * angle.cos() + x * angle.sin()], -1).bfloat16()
            self.rows[b] = torch.cat([self.rows[b], torch.cat([c[at:at + d], turned], -1)])
            at += d
        return new, cu, positions, q_nope, q, o, lse


@pytest.mark.parametrize("page", [16, 64])
def test_steps(page):
    m = Loop(4, page, 2000 // page, 900 // page + 1, seed=page)
    for change in ([300, 1, 0, 70], [1, 1, 129, 1], [3, -1, 4, -3], [-304, 2, 1, 200], [50, -3, -134, 1], [0, 0, 0, -1], [1, 1, 1, 1]):
        new, cu, positions, q_nope, q, o, lse = m.step(change)
        at = 0
        for b, n in enumerate(new):
            L = m.rows[b].shape[0]
            assert int(m.kv_len[b]) == L
            # every row of the cache, in its place
            t = torch.arange(L, device=DEV)
            cached = m.pool[m.table[b].long()[t // page], t % page]
            assert torch.equal(cached[:, :LATENT], m.rows[b][:, :LATENT])
            # a rotary value next to a border between two steps may fall on either side
            err = (cached[:, LATENT:].double() - m.rows[b][:, LATENT:].double()).abs()
            assert (err <= 2.0 ** -7 * m.rows[b][:, LATENT:].double().abs() + 1e-5).all()
            if n:
                x = cached.double()
                s = torch.einsum("nhd,ld->hnl", q[at:at + n].double(), x) * SCALE
                s = s.masked_fill(t > torch.arange(L - n, L, device=DEV)[:, None], -float("inf"))
                ref, ref_lse = torch.einsum("hnl,ld->nhd", s.softmax(-1), x[:, :LATENT]), s.logsumexp(-1)
                # as in the tests of the attention alone
                vmax = float(x[:, :LATENT].abs().max())
                assert ((o[at:at + n].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -13) * vmax).all()
                assert (lse[:, at:at + n].double() - ref_lse).abs().max() <= 2.0 ** -14
            at += n


def test_absorbed_and_expanded_forms_agree():
    # prompts: the absorbed form's latent outputs, taken through the values' expansion, against the expanded form
    m = Loop(3, 32, 60, 20, seed=1)
    new, cu, positions, q_nope, q, o, lse = m.step([200, 33, 129])
    rows = torch.cat(m.rows).float()
    k_nope = torch.einsum("tl,hnl->thn", rows[:, :LATENT], m.w_k).bfloat16()
    v = torch.einsum("tl,hvl->thv", rows[:, :LATENT], m.w_v).bfloat16()
    q2 = torch.cat([q_nope, q[..., LATENT:]], -1).contiguous()
    o2, lse2 = fa.sdpa_fwd_latent(q2, k_nope, rows[:, LATENT:].bfloat16().contiguous(), v, cu, cu, 200, scale=SCALE, causal=True)
    o1 = torch.einsum("thl,hvl->thv", o.float(), m.w_v)
    # Scores differ by the rounding of the absorbed queries and of the expanded keys, 2^-9 of each of 512 and 128 products of
    # N(0, 1) values (after the scale of the weights): standard deviations 2^-9 / sqrt(3) * 22 * SCALE and
    # 2^-9 / sqrt(3) * 11 * SCALE, together 0.002 natural units; eight of them, and as much again for the values and outputs
    # (2^-8 of values up to 5)
    assert (lse - lse2).abs().max() <= 8 * 0.002
    assert (o1 - o2.float()).abs().max() <= 2 * 8 * 0.002 * 5 + 2.0 ** -8 * 5 * 3


def test_two_calls_at_once_and_a_replayed_step():
    m = Loop(5, 16, 400, 70, seed=3)
    m.step([1000, 17, 500, 1, 64])
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    q = torch.randn(5, H, LATENT + ROT, generator=m.g, device=DEV).bfloat16()
    cu = torch.arange(6, dtype=torch.int32, device=DEV)
    want = fa.sdpa_fwd_latent_paged(q, m.pool, m.table, m.kv_len, cu, 1, scale=SCALE)
    torch.cuda.synchronize()
    got = [fa.sdpa_fwd_latent_paged(q, m.pool, m.table, m.kv_len, cu, 1, scale=SCALE, stream=s) for s in (s1, s2) * 4]
    torch.cuda.synchronize()
    for o, lse in got:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    # a decode step recorded once: pages, rotary positions, the write and the attention
    one, c, r, qr = ints([1] * 5), m.rand(5, LATENT).bfloat16(), m.rand(5, ROT).bfloat16(), m.rand(5, H, ROT).bfloat16()

    def step():
        _, _, cu, positions, slots = fa.sdpa_cache_resize(m.table, m.kv_len, one, m.free, m.n_free, 16, 5, kv_len_out=m.kv_len,
                                                          n_free_out=m.n_free)
        fa.sdpa_rope(qr, None, positions, m.inv_freq, q_out=q[..., LATENT:])
        fa.sdpa_latent_write(c, r, m.pool, slots, positions, m.inv_freq)
        return fa.sdpa_fwd_latent_paged(q, m.pool, m.table, m.kv_len, cu, 1, scale=SCALE, causal=True)

    step()
    torch.cuda.synchronize()
    start = [t.clone() for t in (m.table, m.kv_len, m.free, m.n_free, m.pool)]
    eager = [tuple(t.clone() for t in step()) for _ in range(20)]
    torch.cuda.synchronize()
    end = [t.clone() for t in (m.table, m.kv_len, m.free, m.n_free, m.pool)]
    for t, x in zip((m.table, m.kv_len, m.free, m.n_free, m.pool), start):
        t.copy_(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for want in eager:
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    for t, x in zip((m.table, m.kv_len, m.free, m.n_free), end):
        assert torch.equal(t, x)
    assert torch.equal(m.pool.view(torch.int16), end[4].view(torch.int16))
    assert fa.sdpa_check_device_status() == fa.SDPA_OK
