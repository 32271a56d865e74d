"""Measured cases of the latent paged cache, the attention over it, rotary positions and page allocation.

Five operators, each through the package's public call and in a plain form of elementary torch
operations:

  resize       a step's change of every sequence's length: pages taken from and given back to a free list, the
               page table brought up to date, new tokens' positions and cache slots   sdpa_cache_resize
  rope         rotary positions on queries and keys, half or interleaved pairs        sdpa_rope
  write        new tokens' latent vectors and rotated shared keys stored into pages   sdpa_latent_write
  absorbed     attention of new tokens over the latent pages themselves: a row is key and, but for its rotary
               part, value of all heads                                              sdpa_fwd_latent_paged
  expanded     attention over keys and values expanded from the latent vectors, the rotary part of the keys one
               for all heads                                                         sdpa_fwd_latent

A latent cache is a pool [n_pages, page_size, 512 + 64] with a page table [B, max_pages]; row t of
sequence b is row t % page_size of page table[b, t / page_size], slot page * page_size + row of the pool.
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
LATENT, ROT = 512, 64
NOPE, VDIM = 128, 128


def listed():
    return [
        # the new token of each of 64 running sequences: once per step, before the layers
        resize("resize_step", 64, 64, (1, 1), (1024, 16384), False),
        # a scheduler's step over many sequences: prompts come in, sequences end, drafted tokens are dropped
        resize("resize_mixed", 1024, 16, (64, 8192), (1024, 16384), True),
        # a decode step's queries and keys, for every layer of every step
        rope("rope_step", 64, 32, 8, 128, 128, False, 16384, "bf16"),
        # a packed prompt batch far into long contexts, interleaved pairs, a quarter of the head rotated
        rope("rope_prompts", 32767, 28, 4, 128, 32, True, 1 << 20, "f16"),
        # a step's latent rows
        write("write_step", 64, 64, (1, 1), (1024, 16384), False, "bf16"),
        # the prompts of a batch of 16 requests, of the packed prefill workload's lengths
        write("write_prompts", 16, 64, (64, 8192), (64, 8192), True, "bf16"),
        # a few sequences, sixteen heads, small pages
        absorbed("absorbed_few", 3, 16, 16, (1, 1), (1000, 3001), "f16"),
        # the decode workload's batch with the sixteen heads of one of eight shards
        absorbed("absorbed_batch", 64, 16, 64, (1, 1), (1024, 16384), "bf16"),
        # all 128 heads on one GPU, two drafted tokens beside the sampled one
        absorbed("absorbed_drafts", 16, 128, 64, (1, 3), (1024, 16384), "bf16"),
        # a mixed batch of short prompt chunks and decoded tokens
        absorbed("absorbed_mixed", 8, 32, 16, (1, 200), (1000, 8192), "f16"),
        # the prompts of a small batch, odd lengths
        expanded("expanded_short", 7, 16, (33, 1000), (33, 2001), "f16"),
        # one long prompt, the heads of the FP8 workload
        expanded("expanded_long", 1, 128, (8192, 8192), (8192, 8192), "bf16"),
    ]


def named(name, **c):
    return {"name": name, **c} if name else c


# new, kv: inclusive ranges of the sequences' new tokens and of their cached rows (kv counts the new tokens
# too, and is raised to them where it is less; for resize it is the length before the call)
def resize(name, B, page, new, kv, mixed):
    return named(name, op="resize", B=B, page=page, new_lo=new[0], new_hi=new[1], kv_lo=kv[0], kv_hi=kv[1], mixed=mixed)


def rope(name, total, Hq, Hk, D, rot, interleaved, far, dtype):
    return named(name, op="rope", total=total, Hq=Hq, Hk=Hk, D=D, rot=rot, interleaved=interleaved, far=far, dtype=dtype)


def write(name, B, page, new, kv, interleaved, dtype):
    return named(name, op="write", B=B, page=page, new_lo=new[0], new_hi=new[1], kv_lo=kv[0], kv_hi=kv[1],
                 interleaved=interleaved, dtype=dtype)


def absorbed(name, B, H, page, new, kv, dtype, causal=True):
    return named(name, op="absorbed", B=B, H=H, page=page, new_lo=new[0], new_hi=new[1], kv_lo=kv[0], kv_hi=kv[1],
                 dtype=dtype, causal=causal)


def expanded(name, B, H, new, kv, dtype, causal=True):
    return named(name, op="expanded", B=B, H=H, new_lo=new[0], new_hi=new[1], kv_lo=kv[0], kv_hi=kv[1], dtype=dtype,
                 causal=causal)


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        m = most.setdefault(c["op"], [0.0, 0.0])
        m[0], m[1] = max(m[0], w["bytes"]), max(m[1], w["flops"])

    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        op = rng.choice(["resize", "rope", "write", "absorbed", "expanded"])
        B, page, dtype = log(1, 64), rng.choice([16, 32, 64, 128, 256]), rng.choice(["f16", "bf16"])
        new_hi = log(1, 8192)
        kv_hi = max(new_hi, log(16, 32768))
        new, kv = (rng.randint(1, new_hi), new_hi), (log(1, kv_hi), kv_hi)
        if op == "resize":
            c = resize(None, log(1, 2048), page, new, kv, rng.random() < 0.7)
        elif op == "rope":
            D = rng.choice([64, 128, 192])
            c = rope(None, log(1, 65536), log(1, 128), rng.choice([1, 2, 4, 8]), D, rng.choice([16, 32, 64, D]),
                     rng.random() < 0.5, log(64, 1 << 20), dtype)
        elif op == "write":
            c = write(None, B, page, new, kv, rng.random() < 0.5, dtype)
        elif op == "absorbed":
            if rng.random() < 0.6:
                new = (1, rng.choice([1, 1, 2, 5]))
            c = absorbed(None, B, rng.choice([4, 8, 16, 20, 32, 40, 64, 96, 128]), page, new, kv, dtype, rng.random() < 0.85)
        else:
            c = expanded(None, B, log(1, 128), new, kv, dtype, rng.random() < 0.85)
        w = work(c)
        if w["bytes"] <= most[op][0] and w["flops"] <= most[op][1]:
            return c


def lengths(case):
    """(new tokens, cached rows) of each sequence: spread over the ranges, in a mixed order."""
    B = case["B"]
    rng = random.Random(B)

    def spread(lo, hi):
        got = [hi if B == 1 else lo + (hi - lo) * i // (B - 1) for i in range(B)]
        rng.shuffle(got)
        return got

    new = spread(case["new_lo"], case["new_hi"])
    return new, [max(a, b) for a, b in zip(new, spread(case["kv_lo"], case["kv_hi"]))]


def changes(case):
    """(rows before, change) of each sequence: one token each, or a fifth with a new prompt, a tenth that end, a tenth
    that lose up to seven drafted tokens."""
    new, old = lengths(case)
    if not case["mixed"]:
        return old, new
    rng = random.Random(case["B"] + 1)
    change = []
    for b in range(case["B"]):
        x = rng.random()
        if x < 0.2:
            old[b] = 0
            change.append(new[b])
        elif x < 0.3:
            change.append(-old[b])
        elif x < 0.4:
            change.append(-min(old[b], rng.randint(1, 7)))
        else:
            change.append(1)
    return old, change


def pages_of(rows, page):
    return -(-rows // page)


def work(case):
    op = case["op"]
    if op == "resize":
        old, change = changes(case)
        moved = sum(abs(pages_of(o + d, case["page"]) - pages_of(o, case["page"])) for o, d in zip(old, change))
        # lengths and changes in, lengths and offsets out; a position and a slot a token; a page read and written
        return {"bytes": 16 * case["B"] + 12 * sum(max(d, 0) for d in change) + 8 * moved, "flops": 0}
    if op == "rope":
        return {"bytes": case["total"] * (4 * (case["Hq"] + case["Hk"]) * case["D"] + 4) + 2 * case["rot"], "flops": 0}
    new, kv = lengths(case)
    if op == "write":
        return {"bytes": sum(new) * (4 * (LATENT + ROT) + 12), "flops": 0}
    pairs = 0  # (query, key) pairs that see one another
    for n, L in zip(new, kv):
        pairs += n * L - n * (n - 1) // 2 if case["causal"] else n * L
    H = case["H"]
    if op == "absorbed":
        io = sum(new) * H * (2 * (LATENT + ROT) + 2 * LATENT + 4)
        return {"bytes": sum(kv) * 2 * (LATENT + ROT) + io, "flops": 2 * pairs * H * (2 * LATENT + ROT)}
    io = sum(new) * H * (2 * (NOPE + ROT) + 2 * VDIM + 4)
    return {"bytes": sum(kv) * 2 * (H * (NOPE + VDIM) + ROT) + io, "flops": 2 * pairs * H * (NOPE + ROT + VDIM)}


def frequencies(rot, stretched):
    """Radians a position of each pair; stretched: those of the slow pairs divided by 32, as for a context extended
    so far, with a ramp between pairs that turn 32 times and once within 4096 positions."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 10000.0 ** (-2 * i / rot)
    if stretched:
        keep = ((4096 * f / (2 * math.pi)).log() / math.log(32.0)).clamp(0, 1)
        f = f * (keep + (1 - keep) / 32)
    return f.float()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op = case["op"]

    def rand(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    def offsets(n):
        cu = [0]
        for x in n:
            cu.append(cu[-1] + x)
        return ints(cu)

    s = {"op": op, "case": case}
    if op == "resize":
        page = case["page"]
        old, change = changes(case)
        held = [pages_of(n, page) for n in old]
        need = sum(max(0, pages_of(o + d, page) - h) for o, d, h in zip(old, change, held))
        n_pages, width = sum(held) + need + 5, max(pages_of(max(o, o + d), page) for o, d in zip(old, change))
        perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
        s["table"] = torch.zeros((case["B"], width), dtype=torch.int32, device=dev)
        have = torch.arange(width, device=dev) < ints(held)[:, None]
        s["table"][have] = perm[:sum(held)]
        s["free_pages"] = torch.zeros(n_pages, dtype=torch.int32, device=dev)
        s["free_pages"][:n_pages - sum(held)] = perm[sum(held):]
        s["n_free"] = ints([n_pages - sum(held)])
        s["kv_len"], s["change"] = ints(old), ints(change)
        s["total"] = max(1, sum(max(d, 0) for d in change))
        return s
    dt = DTYPES[case["dtype"]]
    if op == "rope":
        n, D = case["total"], case["D"]
        s["q"], s["k"] = rand(n, case["Hq"], D).to(dt), rand(n, case["Hk"], D).to(dt)
        s["positions"] = torch.randint(0, case["far"], (n,), generator=g, device=dev, dtype=torch.int32)
        s["inv_freq"] = frequencies(case["rot"], case["far"] > 16384).to(dev)
        s["factor"] = 0.1 * math.log(32.0) + 1.0 if case["far"] > 16384 else 1.0
        return s
    new, kv = lengths(case)
    s["new"], s["kv"], s["dtype"] = new, kv, dt
    s["cu"], s["max_new"] = offsets(new), max(new)
    if op == "expanded":
        H = case["H"]
        s["q"] = rand(sum(new), H, NOPE + ROT).to(dt)
        # one product expands the latent vectors into keys and values, head by head
        both = rand(sum(kv), H, NOPE + VDIM).to(dt)
        s["k_nope"], s["v"] = both[..., :NOPE], both[..., NOPE:]
        s["k_rope"] = rand(sum(kv), ROT).to(dt)
        s["cu_k"], s["scale"] = offsets(kv), 1.0 / math.sqrt(NOPE + ROT)
        return s
    # the pages of the sequences lie anywhere in the pool; two pages stay free
    page = case["page"]
    held = [pages_of(n, page) for n in kv]
    n_pages, width = sum(held) + 2, max(held)
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros((case["B"], width), dtype=torch.int32, device=dev)
    table[torch.arange(width, device=dev) < ints(held)[:, None]] = perm[:sum(held)]
    s["table"], s["kv_len"] = table, ints(kv)
    if op == "write":
        n = sum(new)
        s["c"], s["k_rope"] = rand(n, LATENT).to(dt), rand(n, ROT).to(dt)
        s["pool"] = torch.zeros((n_pages, page, LATENT + ROT), dtype=dt, device=dev)
        b = torch.repeat_interleave(torch.arange(case["B"], device=dev), ints(new))
        pos = torch.arange(n, device=dev) - s["cu"].long()[b] + (s["kv_len"] - ints(new)).long()[b]
        s["positions"] = pos.to(torch.int32)
        s["slots"] = table[b, pos // page].long() * page + pos % page
        s["inv_freq"] = frequencies(ROT, False).to(dev)
        return s
    pool = torch.empty((n_pages, page, LATENT + ROT), dtype=dt, device=dev)
    step = max(1, (1 << 26) // (page * (LATENT + ROT)))
    for i in range(0, n_pages, step):
        pool[i:i + step] = rand(min(step, n_pages - i), page, LATENT + ROT).to(dt)
    s["pool"] = pool
    s["q"] = rand(sum(new), case["H"], LATENT + ROT).to(dt)
    s["scale"] = 1.0 / math.sqrt(LATENT + ROT)
    return s


def plain_resize(s):
    page, table, free = s["case"]["page"], s["table"], s["free_pages"]
    dev = table.device
    old, change, n_free = s["kv_len"].long(), s["change"].long(), s["n_free"].long()
    new = old + change
    po, pn = (old + page - 1) // page, (new + page - 1) // page
    back, more = (po - pn).clamp(min=0), (pn - po).clamp(min=0)
    seqs = torch.arange(len(old), device=dev)

    def spread(count, first):
        """(sequence, index) of every item, count[b] of each sequence from first[b] on."""
        b = torch.repeat_interleave(seqs, count)
        return b, torch.arange(len(b), device=dev) - (count.cumsum(0) - count)[b] + first[b]

    returned = table[spread(back, pn)]
    F, b_p = len(returned), spread(more, po)
    A = len(b_p[0])
    at = n_free + F - 1 - torch.arange(A, device=dev)
    taken = free[at.clamp(max=len(free) - 1)]
    if F:
        taken = torch.where(at >= n_free, returned[(at - n_free).clamp(min=0)], taken)
    table[b_p] = taken
    if F > A:
        free[n_free + torch.arange(F - A, device=dev)] = returned[:F - A]
    cu = torch.zeros(len(old) + 1, dtype=torch.int32, device=dev)
    cu[1:] = change.clamp(min=0).cumsum(0)
    b, pos = spread(change.clamp(min=0), old)
    positions = torch.zeros(s["total"], dtype=torch.int32, device=dev)
    slots = torch.full((s["total"],), -1, dtype=torch.int64, device=dev)
    positions[:len(b)] = pos.to(torch.int32)
    slots[:len(b)] = table[b, pos // page].long() * page + pos % page
    return [new.to(torch.int32), (n_free + F - A).to(torch.int32), cu, positions, slots, table, free]


def rotated(x, positions, inv_freq, interleaved, factor):
    """x [total, heads, D] in 32 bits with its first pairs turned."""
    angle = positions.double()[:, None] * inv_freq.double()
    cos, sin = (angle.cos() * factor).float()[:, None], (angle.sin() * factor).float()[:, None]
    half = inv_freq.shape[0]
    x = x.float()
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * cos - b * sin, b * cos + a * sin
    return y


def plain_attention(s):
    """Every sequence's new tokens against its rows, some queries at a time."""
    c, q = s["case"], s["q"]
    H = c["H"]
    Dv = LATENT if c["op"] == "absorbed" else VDIM
    o = torch.empty((q.shape[0], H, Dv), dtype=q.dtype, device=q.device)
    lse = torch.empty((H, q.shape[0]), device=q.device)
    at = at_k = 0
    for b, (n, L) in enumerate(zip(s["new"], s["kv"])):
        if c["op"] == "absorbed":
            rows = s["pool"][s["table"][b, :pages_of(L, c["page"])].long()].flatten(0, 1)[:L].float()
            k, v = rows.t()[None], rows[None, :, :LATENT]                     # [1, 576, L], [1, L, 512]
        else:
            shared = s["k_rope"][at_k:at_k + L].float()[:, None].expand(L, H, ROT)
            k = torch.cat([s["k_nope"][at_k:at_k + L].float(), shared], -1).permute(1, 2, 0)
            v = s["v"][at_k:at_k + L].float().transpose(0, 1)
            at_k += L
        step = max(1, (1 << 29) // (H * L))
        for i in range(0, n, step):
            m = min(step, n - i)
            x = q[at + i:at + i + m].float() * s["scale"]
            if c["op"] == "absorbed":
                x = torch.matmul(x.reshape(m * H, -1), k[0]).view(m, H, L).transpose(0, 1).contiguous()
            else:
                x = torch.matmul(x.transpose(0, 1), k)                        # [H, m, L]
            if c["causal"]:
                pos = torch.arange(L - n + i, L - n + i + m, device=q.device)
                x.masked_fill_(torch.arange(L, device=q.device) > pos[:, None], -math.inf)
            top = x.amax(-1, keepdim=True)
            x = x.sub_(top).exp_()
            total = x.sum(-1, keepdim=True)
            if c["op"] == "absorbed":
                y = torch.matmul(x.view(H * m, L), v[0]).view(H, m, Dv)
            else:
                y = torch.matmul(x, v)
            o[at + i:at + i + m] = (y / total).transpose(0, 1).to(q.dtype)
            lse[:, at + i:at + i + m] = (top + total.log())[..., 0]
        at += n
    return [o, lse]


def run(s):
    op, c = s["op"], s["case"]
    if not own:
        if op == "resize":
            return plain_resize(s)
        if op == "rope":
            return [rotated(s[n], s["positions"], s["inv_freq"], c["interleaved"], s["factor"]).to(s[n].dtype)
                    for n in ("q", "k")]
        if op == "write":
            turned = rotated(s["k_rope"][:, None], s["positions"], s["inv_freq"], c["interleaved"], 1.0)[:, 0]
            rows = s["pool"].view(-1, LATENT + ROT)
            rows[s["slots"]] = torch.cat([s["c"], turned.to(s["dtype"])], -1)
            return [s["pool"]]
        return plain_attention(s)
    import flash_attention_forward_gb300 as fa
    if op == "resize":
        got = fa.sdpa_cache_resize(s["table"], s["kv_len"], s["change"], s["free_pages"], s["n_free"], c["page"], s["total"])
        return [*got, s["table"], s["free_pages"]]
    if op == "rope":
        return fa.sdpa_rope(s["q"], s["k"], s["positions"], s["inv_freq"], interleaved=c["interleaved"], factor=s["factor"])
    if op == "write":
        fa.sdpa_latent_write(s["c"], s["k_rope"], s["pool"], s["slots"], s["positions"], s["inv_freq"],
                             interleaved=c["interleaved"])
        return [s["pool"]]
    if op == "absorbed":
        return fa.sdpa_fwd_latent_paged(s["q"], s["pool"], s["table"], s["kv_len"], s["cu"], s["max_new"],
                                        scale=s["scale"], causal=c["causal"])
    return fa.sdpa_fwd_latent(s["q"], s["k_nope"], s["k_rope"], s["v"], s["cu"], s["cu_k"], s["max_new"],
                              scale=s["scale"], causal=c["causal"])


def exact_resize(case, s):
    """The free list as a list: pages given back are pushed sequence by sequence, then new ones popped."""
    page = case["page"]
    table, old, change = s["table"].tolist(), s["kv_len"].tolist(), s["change"].tolist()
    stored, n_free = s["free_pages"].tolist(), s["n_free"].item()
    stack = stored[:n_free]
    for b, (o, d) in enumerate(zip(old, change)):
        stack += table[b][pages_of(o + d, page):pages_of(o, page)]
    for b, (o, d) in enumerate(zip(old, change)):
        for p in range(pages_of(o, page), pages_of(o + d, page)):
            table[b][p] = stack.pop()
    if len(stack) > n_free:
        stored[n_free:len(stack)] = stack[n_free:]
    cu, positions, slots = [0], [], []
    for b, (o, d) in enumerate(zip(old, change)):
        cu.append(cu[-1] + max(d, 0))
        for t in range(o, o + d):
            positions.append(t)
            slots.append(table[b][t // page] * page + t % page)
    if not positions:
        positions, slots = [0], [-1]
    got = [[o + d for o, d in zip(old, change)], [len(stack)], cu, positions, slots, table, stored]
    return [torch.tensor(x, dtype=torch.int64 if i == 4 else torch.int32, device="cuda") for i, x in enumerate(got)]


def exact(case, seed):
    """The same outputs from the definitions, in 64 bits."""
    if work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    op = case["op"]

    def turn(x, positions):
        """Pairs as complex numbers times e^(i angle)."""
        f = s["inv_freq"].double()
        w = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), positions.double()[:, None, None] * f)
        w = w * s.get("factor", 1.0)
        n, x = 2 * len(f), x.double()
        pairs = x[..., :n].unflatten(-1, (-1, 2)) if case["interleaved"] else x[..., :n].unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * w)
        z = z if case["interleaved"] else z.transpose(-1, -2)
        return torch.cat([z.flatten(-2), x[..., n:]], -1)

    if op == "resize":
        return exact_resize(case, s)
    if op == "rope":
        return [turn(s["q"], s["positions"]), turn(s["k"], s["positions"])]
    if op == "write":
        got = s["pool"].double()
        got.view(-1, LATENT + ROT)[s["slots"], :LATENT] = s["c"].double()
        got.view(-1, LATENT + ROT)[s["slots"], LATENT:] = turn(s["k_rope"][:, None], s["positions"])[:, 0]
        return [got]
    H, Dv = case["H"], LATENT if op == "absorbed" else VDIM
    o = torch.zeros((s["q"].shape[0], H, Dv), dtype=torch.float64, device="cuda")
    lse = torch.zeros((H, s["q"].shape[0]), dtype=torch.float64, device="cuda")
    at = at_k = 0
    for b, (n, L) in enumerate(zip(s["new"], s["kv"])):
        if op == "absorbed":
            t = torch.arange(L, device="cuda")
            flat = s["table"][b].long()[t // case["page"]] * case["page"] + t % case["page"]
            rows = s["pool"].reshape(-1, LATENT + ROT)[flat].double()
        for h in range(H):
            if op == "absorbed":
                k, v = rows, rows[:, :LATENT]
            else:
                k = torch.cat([s["k_nope"][at_k:at_k + L, h], s["k_rope"][at_k:at_k + L]], -1).double()
                v = s["v"][at_k:at_k + L, h].double()
            for i in range(0, n, 4096):
                m = min(4096, n - i)
                x = torch.einsum("md,ld->ml", s["q"][at + i:at + i + m, h].double(), k) * s["scale"]
                if case["causal"]:
                    x += torch.full_like(x, -math.inf).triu(L - n + i + 1)
                lse[h, at + i:at + i + m] = torch.logsumexp(x, -1)
                o[at + i:at + i + m, h] = torch.exp(x - lse[h, at + i:at + i + m, None]) @ v
        at += n
        at_k += L
    return [o, lse]
