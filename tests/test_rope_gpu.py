"""GPU tests of rotary positions and of the latent cache's writer, against the definition in 64 bits.

Tolerance of a turned value y = factor (a cos - b sin): half a step of the type, eps / 2 * |y|; and in fp32
factor (|a| + |b|) times the error of cos and sin (the fraction of a turn rounded to 24 bits, pi 2^-24; sincospif's
2 steps, 2^-22; the product with factor, 2^-24) and of the three operations (2^-24 each): under 12 * 2^-24 in all.
Halves below fp16's normal range are off by up to 2^-25."""
import math

import pytest
import torch

import flash_attention_forward_gb300 as fa

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def turned(x, positions, inv_freq, interleaved, factor=1.0):
    """(y, |a| + |b|) in 64 bits, on the CPU."""
    x = x.double().cpu()
    half = inv_freq.numel()
    angle = positions.double().cpu()[:, None] * inv_freq.double().cpu()
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    ia = torch.arange(half) * 2 if interleaved else torch.arange(half)
    ib = ia + 1 if interleaved else ia + half
    y, size = x.clone(), torch.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = factor * (a * cos - b * sin), factor * (b * cos + a * sin)
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return y, size


def close(got, want, size, dt, factor=1.0, lost=0.0):
    """lost: error of the angle beside that of its fraction of a turn."""
    got = got.double().cpu()
    tol = size * lost + want.abs() * (torch.finfo(dt).eps / 2) * (1 + 2.0 ** -10) + abs(factor) * size * 12 * 2.0 ** -24
    if dt == torch.float16:
        tol = tol + 2.0 ** -25
    tol[size == 0] = 0.0   # copied dims, and pairs of zeros
    assert ((got - want).abs() <= tol).all(), float(((got - want).abs() - tol).max())


def case(total, Hq, Hk, D, dt, seed=0, far=100000):
    g = torch.Generator().manual_seed(seed)
    q, k = (torch.randn((total, h, D), generator=g).to(dt) for h in (Hq, Hk))
    return q.to(DEV), k.to(DEV), torch.randint(0, far, (total,), generator=g).to(torch.int32).to(DEV)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("total,Hq,Hk,D,rot", [(1, 32, 8, 128, 128), (64, 28, 4, 128, 32), (33, 1, 1, 64, 64), (257, 5, 3, 192, 64),
                                               (3, 128, 2, 192, 16), (5000, 7, 1, 64, 48), (2, 300, 16, 8 * 13, 96)])
def test_rope(dtype, interleaved, total, Hq, Hk, D, rot):
    q, k, pos = case(total, Hq, Hk, D, DT[dtype], seed=total + D)
    inv_freq = fa.sdpa_rope_frequencies(rot)[0].to(DEV)
    got = fa.sdpa_rope(q, k, pos, inv_freq, interleaved=interleaved, factor=1.25)
    for x, y in zip((q, k), got):
        want, size = turned(x, pos, inv_freq, interleaved, 1.25)
        close(y, want, size, DT[dtype], 1.25)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_negative_and_odd_angles(interleaved):
    q, _, _ = case(7, 3, 1, 64, torch.float16, seed=1)
    pos = torch.tensor([0, -1, 1 << 20, -(1 << 20) + 1, (1 << 31) - 1, -(1 << 31), 12345678], dtype=torch.int32, device=DEV)
    inv_freq = torch.tensor([1.0, 0.5, 0.0, 1e-30, 2.0 ** -140, -0.3, 1e-7, 6.2831855, 12345.678, 2.0 ** 24, 2e-3, 0.99999994,
                             -0.0, 3.14159274, 100.5, 1e-4] * 2, device=DEV)
    got, none = fa.sdpa_rope(q, None, pos, inv_freq, interleaved=interleaved)
    assert none is None
    # the angle's cosine in 64 bits loses 2^-53 of the angle itself, up to 2^31 * 2^24: so the turns are taken as
    # fractions of whole numbers here
    from fractions import Fraction
    two_pi = Fraction(0x6487ED5110B4611A62633145C06E0E68948127044533E63A010, 1 << 200)
    turns = [[(Fraction(p) * Fraction(f) / two_pi) % 1 for f in inv_freq.cpu().double().tolist()] for p in pos.tolist()]
    angle = torch.tensor([[float(t) * 2 * math.pi for t in r] for r in turns], dtype=torch.float64)
    want, size = turned(q, torch.ones(7), torch.ones(32), interleaved)
    x = q.double().cpu()
    ia = torch.arange(32) * 2 if interleaved else torch.arange(32)
    ib = ia + 1 if interleaved else ia + 32
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    want[..., ia], want[..., ib] = x[..., ia] * c - x[..., ib] * s, x[..., ib] * c + x[..., ia] * s
    # 1 / 2 pi is held to 2^-64 of itself, and a position's step to 2^-64 turns: with a frequency of 2^24 and a position of
    # 2^31 (2^52 turns) that is 2^-12 turns, with frequencies up to 1 it is below 2^-32
    whole = pos.double().cpu().abs()[:, None] * inv_freq.double().cpu().abs() / (2 * math.pi)
    lost = 2 * math.pi * 2.0 ** -64 * (whole + pos.double().cpu().abs()[:, None])
    both = torch.zeros(7, 1, 64, dtype=torch.float64)
    both[..., ia] = both[..., ib] = lost[:, None]
    close(got, want, size, torch.float16, lost=both)


def test_frequencies_out_of_range_give_nan_and_others_are_not_touched():
    q, _, pos = case(4, 2, 1, 64, torch.bfloat16, seed=2)
    inv_freq = torch.full((32,), 0.1, device=DEV)
    inv_freq[3], inv_freq[4], inv_freq[5] = float("nan"), float("inf"), 2.0 ** 25
    got, _ = fa.sdpa_rope(q, None, pos, inv_freq)
    bad = torch.isnan(got).any(0).any(0).cpu()
    assert bad.nonzero()[:, 0].tolist() == [3, 4, 5, 35, 36, 37]
    # an infinity or NaN of the input stays in its pair
    inv_freq.fill_(0.1)
    q[1, 0, 7], q[2, 1, 40] = float("nan"), float("inf")
    got, _ = fa.sdpa_rope(q, None, pos, inv_freq)
    odd = (~torch.isfinite(got)).nonzero().tolist()
    assert odd == [[1, 0, 7], [1, 0, 39], [2, 1, 8], [2, 1, 40]]


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_and_views_of_a_part_of_the_head(interleaved):
    total, Hq = 40, 6
    q, k, pos = case(total, Hq, 1, 576, torch.bfloat16, seed=3)
    q0, k0 = q.clone(), k.clone()
    inv_freq = fa.sdpa_rope_frequencies(64)[0].to(DEV)
    qv, kv = q[..., 512:], k[..., 512:]
    got = fa.sdpa_rope(qv, kv, pos, inv_freq, interleaved=interleaved, q_out=qv, k_out=kv)
    assert got[0] is qv
    for x, x0 in ((q, q0), (k, k0)):
        assert torch.equal(x[..., :512], x0[..., :512])
        close(x[..., 512:], *turned(x0[..., 512:], pos, inv_freq, interleaved), torch.bfloat16)
    # only q in place, the pass-through dims of k copied, canaries around the output
    q, k = q0.clone(), k0.clone()
    pad = torch.full((total + 2, 3, 576), 5.0, dtype=torch.bfloat16, device=DEV)
    fa.sdpa_rope(q, k, pos, inv_freq, interleaved=interleaved, q_out=q, k_out=pad[1:-1, 1:2])
    close(q, *turned(q0, pos, inv_freq, interleaved), torch.bfloat16)
    close(pad[1:-1, 1:2], *turned(k0, pos, inv_freq, interleaved), torch.bfloat16)
    pad[1:-1, 1:2] = 5.0
    assert (pad == 5.0).all()


def test_broadcast_inputs_and_shared_positions():
    # one rotary key read as that of four heads; the input of all tokens one row
    q, k, pos = case(9, 4, 1, 64, torch.float16, seed=5)
    inv_freq = fa.sdpa_rope_frequencies(64)[0].to(DEV)
    got_q, got_k = fa.sdpa_rope(q[:1].expand(9, -1, -1), k.expand(-1, 4, -1), pos, inv_freq)
    close(got_q, *turned(q[:1].expand(9, -1, -1), pos, inv_freq, False), torch.float16)
    close(got_k, *turned(k.expand(-1, 4, -1), pos, inv_freq, False), torch.float16)


def test_gradient():
    # y = R x is linear: its gradient R^T g is the call with -positions; against the formula and against differences
    x, g, pos = case(50, 4, 4, 64, torch.float16, seed=4)
    inv_freq = fa.sdpa_rope_frequencies(64)[0].to(DEV)
    back, _ = fa.sdpa_rope(g, None, -pos, inv_freq, factor=1.5)
    close(back, *turned(g, -pos, inv_freq, False, 1.5), torch.float16, 1.5)
    d = torch.randn(x.shape, generator=torch.Generator().manual_seed(9)).double()
    h = 0.125
    up, down = (turned((x.double().cpu() + s * h * d), pos, inv_freq, False, 1.5)[0] for s in (1, -1))
    diff = float((((up - down) / (2 * h)) * g.double().cpu()).sum())
    dot = float((back.double().cpu() * d).sum())
    # |back - R^T g| <= 2^-11 |back| + 18 2^-24 (|a| + |b|) + 2^-25 an entry, against |d|
    bound = float(((back.double().cpu().abs() * 2.0 ** -11 + 1e-5) * d.abs()).sum())
    assert abs(diff - dot) <= bound


def test_scaled_frequencies():
    plain, one = fa.sdpa_rope_frequencies(64)
    assert one == 1.0 and plain.dtype == torch.float32
    i = torch.arange(32, dtype=torch.float64)
    assert torch.equal(plain, (10000.0 ** (-i / 32)).float())
    lin, f = fa.sdpa_rope_frequencies(64, scaling="linear", factor=8.0)
    assert f == 1.0 and torch.allclose(lin * 8, plain, rtol=1e-6)
    base, f = fa.sdpa_rope_frequencies(64, scaling="base", factor=8.0)
    assert f == 1.0 and base[0] == 1.0 and abs(float(base[-1] * 8 / plain[-1]) - 1) < 1e-5
    parts, f = fa.sdpa_rope_frequencies(64, scaling="by_parts", factor=32.0, original_length=4096)
    assert abs(f - (0.1 * math.log(32.0) + 1)) < 1e-12
    turns = 4096 * plain.double() / (2 * math.pi)
    ratio = parts.double() / plain.double()
    assert (abs(ratio[turns > 40] - 1) < 1e-6).all() and (abs(ratio[turns < 0.7] * 32 - 1) < 1e-5).all()
    assert (ratio[1:] <= ratio[:-1] + 1e-9).all()
    for bad in (dict(scaling="none"), dict(scaling="by_parts", factor=2.0), dict(factor=0.5)):
        with pytest.raises(ValueError):
            fa.sdpa_rope_frequencies(64, **bad)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("total,page,n_pages", [(1, 16, 3), (9, 64, 2), (1000, 16, 100)])
def test_latent_write(dtype, interleaved, total, page, n_pages):
    dt = DT[dtype]
    g = torch.Generator().manual_seed(total)
    both = torch.randn((total, 576 + 8), generator=g).to(dt).to(DEV)   # one projection, read through views
    c, r = both[:, :512], both[:, 512:576]
    pos = torch.randint(0, 1 << 20, (total,), generator=g).to(torch.int32).to(DEV)
    slots = torch.randperm(page * n_pages, generator=g)[:total].to(DEV)
    slots[::4] = torch.where(torch.arange(total, device=DEV)[::4] % 8 == 0, slots[::4], -1 - slots[::4])
    wide = torch.full((n_pages, page + 1, 592), 3.0, dtype=dt, device=DEV)
    pool = wide[:, :page, :576]
    inv_freq = fa.sdpa_rope_frequencies(64)[0].to(DEV)
    fa.sdpa_latent_write(c, r, pool, slots, pos, inv_freq, interleaved=interleaved, factor=0.5)
    assert fa.sdpa_check_device_status() == fa.SDPA_OK
    want, size = turned(r[:, None], pos, inv_freq, interleaved, 0.5)
    live = slots >= 0
    at, row = slots[live] // page, slots[live] % page
    assert torch.equal(wide[at, row, :512], c[live])
    close(wide[at, row, 512:576][:, None], want[live.cpu()], size[live.cpu()], dt, 0.5)
    wide[at, row, :576] = 3.0
    assert (wide == 3.0).all()
    fa.sdpa_latent_write(c, r, pool, slots)
    assert torch.equal(wide[at, row, :576], both[live, :576])


def test_latent_write_reports_slots_behind_the_pool():
    c = torch.ones((4, 512), dtype=torch.float16, device=DEV)
    r = torch.ones((4, 64), dtype=torch.float16, device=DEV)
    pool = torch.zeros((4, 16, 576), dtype=torch.float16, device=DEV)[:2]
    slots = torch.tensor([3, 32, 1 << 40, -(1 << 40)], device=DEV)
    fa.sdpa_latent_write(c, r, pool, slots)
    assert fa.sdpa_check_device_status() == fa.SDPA_ERR_INVALID
    assert (pool[0, 3] == 1).all() and pool.float().sum() == 576 and fa.sdpa_check_device_status() == fa.SDPA_OK


def test_latent_write_of_one_row_to_many_slots():
    g = torch.Generator().manual_seed(2)
    c, r = torch.randn((1, 512), generator=g).half().to(DEV), torch.randn((1, 64), generator=g).half().to(DEV)
    pool = torch.zeros((3, 16, 576), dtype=torch.float16, device=DEV)
    slots = torch.arange(5, 45, device=DEV)
    fa.sdpa_latent_write(c.expand(40, -1), r.expand(40, -1), pool, slots)
    rows = pool.view(-1, 576)
    assert (rows[5:45] == torch.cat([c, r], 1)).all() and not rows[:5].any() and not rows[45:].any()


def test_latent_write_past_32_bits():
    n_pages = (1 << 32) // (576 * 2 * 256) + 20   # the last pages lie behind 2^32 bytes
    pool = torch.zeros((n_pages, 256, 576), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator().manual_seed(1)
    c, r = torch.randn((40, 512), generator=g).to(torch.bfloat16).to(DEV), torch.randn((40, 64), generator=g).to(torch.bfloat16).to(DEV)
    slots = (n_pages * 256 - 1 - 100 * torch.arange(40)).to(DEV)
    fa.sdpa_latent_write(c, r, pool, slots)
    assert torch.equal(pool.view(-1, 576)[slots], torch.cat([c, r], 1))
    assert int((pool.view(-1, 576)[:, 0] != 0).sum()) == 40


def test_streams_and_graphs():
    q, k, pos = case(30, 4, 2, 128, torch.bfloat16, seed=6)
    inv_freq = fa.sdpa_rope_frequencies(128)[0].to(DEV)
    want = [t.clone() for t in fa.sdpa_rope(q, k, pos, inv_freq)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fa.sdpa_rope(q, k, pos, inv_freq, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    pool = torch.zeros((2, 16, 576), dtype=torch.bfloat16, device=DEV)
    c, r = torch.randn((30, 512), device=DEV).bfloat16(), torch.randn((30, 64), device=DEV).bfloat16()
    slots = torch.arange(30, device=DEV)
    f64 = fa.sdpa_rope_frequencies(64)[0].to(DEV)
    fa.sdpa_latent_write(c, r, pool, slots, pos, f64)
    want_pool = pool.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = fa.sdpa_rope(q, k, pos, inv_freq)
        fa.sdpa_latent_write(c, r, pool, slots, pos, f64)
    for _ in range(2):
        pool.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got)) and torch.equal(pool, want_pool)
