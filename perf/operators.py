"""Measured cases of the quantised paged cache and the attention over paged caches.

Five operators, each through the package's public call and in a plain form of elementary torch
operations:

  write        new tokens' K and V quantised to e4m3 (one power-of-two scale per token and KV head)
               and stored into the pages of a cache                      sdpa_cache_write_fp8
  read         the cached rows of every sequence read back as packed 16-bit tensors
                                                                         sdpa_cache_read_fp8
  decode       one query token per sequence over the quantised pages     sdpa_decode_paged_fp8
  chunk        a chunk of new tokens per sequence over 16-bit pages      sdpa_fwd_paged
  chunk_fp8    the same over the quantised pages                         sdpa_fwd_paged_fp8

A cache is a pool [n_pages, page_size, Hkv, D] with a page table [B, max_pages]; row t of sequence
b is row t % page_size of page table[b, t / page_size].  kv_len[b] counts the rows of sequence b,
its new tokens (rows cu[b] .. cu[b + 1] of the packed tensors) being the last of them.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
MIN_EXP = -80  # smallest scale exponent: rows of zeros take it
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def case(name, op, B, Hq, Hkv, D, Dv, page, new, kv, dtype, causal=True):
    """new, kv: inclusive ranges of the sequences' new tokens and of their cached rows (kv counts the
    new tokens too, and is raised to them where it is less)."""
    c = {"op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "Dv": Dv, "page": page, "new_lo": new[0], "new_hi": new[1],
         "kv_lo": kv[0], "kv_hi": kv[1], "dtype": dtype, "causal": causal}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one decoded token for each of 32 running sequences goes into the cache: a call made for every layer
        # of every step, where latency is all
        case("write_step", "write", 32, 32, 8, 128, 128, 64, (1, 1), (1024, 16384), "bf16"),
        # the prompts of a batch of 16 requests, of the packed prefill workload's lengths
        case("write_prompts", "write", 16, 32, 8, 128, 128, 64, (64, 8192), (64, 8192), "bf16"),
        # a few short sequences read back, odd lengths, small pages, small heads
        case("read_short", "read", 3, 28, 4, 64, 64, 16, (1, 1), (1000, 3001), "f16"),
        # a batch's caches read back whole, to move or to re-use them
        case("read_long", "read", 16, 32, 8, 128, 128, 128, (1, 1), (1024, 16384), "bf16"),
        # a few sequences with the widest head group and the larger key dimension
        case("decode_few", "decode", 3, 64, 4, 192, 128, 16, (1, 1), (1000, 3001), "f16"),
        # the decode workload's batch: 64 sequences of 1024 to 16384 rows
        case("decode_batch", "decode", 64, 32, 8, 128, 128, 64, (1, 1), (1024, 16384), "bf16"),
        # a few drafted tokens per sequence checked against long caches: bound by reading the cache
        case("chunk_drafts", "chunk", 16, 32, 8, 128, 128, 64, (3, 8), (1024, 16384), "bf16"),
        # a mixed batch of prompt chunks, odd lengths, seven query heads per KV head
        case("chunk_mixed", "chunk", 8, 28, 4, 128, 128, 16, (1, 1000), (1000, 8192), "f16"),
        # one long prompt's chunk of 8192 tokens over 32768 rows
        case("chunk_long", "chunk", 1, 32, 8, 128, 128, 64, (8192, 8192), (32768, 32768), "bf16"),
        # drafted tokens over quantised pages
        case("chunk_fp8_drafts", "chunk_fp8", 16, 32, 8, 128, 128, 64, (3, 8), (1024, 16384), "bf16"),
        # prompt chunks of a mixed batch over quantised pages, seven query heads per KV head
        case("chunk_fp8_mixed", "chunk_fp8", 8, 28, 4, 128, 128, 16, (1, 1000), (1000, 8192), "f16"),
        # chunks of 2048 tokens of four long prompts over quantised pages
        case("chunk_fp8_long", "chunk_fp8", 4, 32, 8, 128, 128, 64, (2048, 2048), (16384, 16384), "bf16"),
    ]


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        m = most.setdefault(c["op"], [0.0, 0.0])
        m[0], m[1] = max(m[0], w["bytes"]), max(m[1], w["flops"])

    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        op = rng.choice(["write", "read", "decode", "chunk", "chunk_fp8"])
        dims = [(128, 128)] * 3 + [(192, 128)] + ([] if op == "decode" else [(64, 64)])
        D, Dv = rng.choice(dims)
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 7, 8, 16])
        new_hi = 1 if op in ("read", "decode") else log(1, 8192)
        kv_hi = max(new_hi, log(16, 32768))
        c = case(None, op, log(1, 64), Hq, Hkv, D, Dv, rng.choice([16, 32, 64, 128, 256]),
                 (rng.randint(1, new_hi), new_hi), (log(1, kv_hi), kv_hi), rng.choice(["f16", "bf16"]),
                 rng.random() < 0.85)
        w = work(c)
        if all(a <= b for a, b in zip((w["bytes"], w["flops"]), most[op])):
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


def work(case):
    new, kv = lengths(case)
    D, Dv, Hq, Hkv = case["D"], case["Dv"], case["Hq"], case["Hkv"]
    quantised = Hkv * (D + Dv + 8)   # one row of codes, with its two scales
    wide = Hkv * (D + Dv) * 2        # one 16-bit row
    if case["op"] == "write":
        return {"bytes": sum(new) * (wide + quantised), "flops": 0}
    if case["op"] == "read":
        return {"bytes": sum(kv) * (wide + quantised), "flops": 0}
    io = sum(new) * Hq * (2 * D + 2 * Dv + 4)  # q, o and the log-sum-exp
    pairs = 0  # (query, key) pairs that see one another
    for n, L in zip(new, kv):
        pairs += n * L - n * (n - 1) // 2 if case["causal"] else n * L
    row = wide if case["op"] == "chunk" else quantised
    return {"bytes": sum(kv) * row + io, "flops": 2 * pairs * Hq * (D + Dv)}


def quantise(x):
    """e4m3 codes of the rows of x and their scales: the least power of two that keeps a row within 448."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m <= 0.875, e - 9, e - 8)  # amax = m 2^e, 448 = 0.875 * 2^9
    e = torch.where(m == 0, torch.full_like(e, MIN_EXP), e).clamp(min=MIN_EXP)
    s = torch.ldexp(torch.ones_like(m), e)
    return (x / s[..., None]).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    B, Hq, Hkv, D, Dv, page = (case[n] for n in ("B", "Hq", "Hkv", "D", "Dv", "page"))
    dt = DTYPES[case["dtype"]]
    new, kv = lengths(case)

    def rand(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    def offsets(n):
        cu = [0]
        for x in n:
            cu.append(cu[-1] + x)
        return torch.tensor(cu, dtype=torch.int32, device=dev)

    # the pages of the sequences lie anywhere in the pool; two pages stay free
    pages = [-(-L // page) for L in kv]
    n_pages, max_pages = sum(pages) + 2, max(pages)
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros((B, max_pages), dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    s = {"op": case["op"], "case": case, "new": new, "kv": kv, "table": table, "dtype": dt,
         "kv_len": torch.tensor(kv, dtype=torch.int32, device=dev), "scale": 1.0 / math.sqrt(D),
         "max_new": max(new), "cu": offsets(new)}
    # keys with a few strong channels, values with a mean of their own in each channel
    gain, mean = torch.exp(0.5 * rand(Hkv, D)), 0.5 * rand(Hkv, Dv)
    if case["op"] == "write":
        n = sum(new)
        s["k"], s["v"] = (rand(n, Hkv, D) * gain).to(dt), (rand(n, Hkv, Dv) + mean).to(dt)
        s["k_pool"], s["v_pool"] = (torch.zeros((n_pages, page, Hkv, d), device=dev).to(torch.float8_e4m3fn)
                                    for d in (D, Dv))
        s["k_scale"], s["v_scale"] = (torch.zeros((n_pages, Hkv, page), device=dev) for _ in range(2))
        return s
    quantised = case["op"] != "chunk"
    pool_dt = torch.float8_e4m3fn if quantised else dt
    for name, d in (("k", D), ("v", Dv)):
        pool = torch.empty((n_pages, page, Hkv, d), dtype=pool_dt, device=dev)
        scale = torch.empty((n_pages, Hkv, page), device=dev)
        step = max(1, (1 << 26) // (page * Hkv * d))
        for i in range(0, n_pages, step):
            x = rand(min(step, n_pages - i), page, Hkv, d)
            x = (x * gain if name == "k" else x + mean).to(dt)
            if quantised:
                pool[i:i + step], sc = quantise(x)
                scale[i:i + step] = sc.transpose(1, 2)
            else:
                pool[i:i + step] = x
        s[name + "_pool"] = pool
        if quantised:
            s[name + "_scale"] = scale
    if case["op"] == "read":
        s["cu"], s["total"] = offsets(kv), sum(kv)
    else:
        q = rand(sum(new), Hq, D)
        s["q"] = (1.5 * q).to(dt)
    return s


def rows_of(s, name, b):
    """fp32 rows [kv_len, Hkv, D] of sequence b's cache."""
    page, L = s["case"]["page"], s["kv"][b]
    at = s["table"][b, :-(-L // page)].long()
    x = s[name + "_pool"][at].float()
    if name + "_scale" in s:
        x = x * s[name + "_scale"][at].transpose(1, 2)[..., None]
    return x.flatten(0, 1)[:L]


def plain_write(s):
    dev = s["table"].device
    n = torch.tensor(s["new"], device=dev)
    b = torch.repeat_interleave(torch.arange(len(s["new"]), device=dev), n)
    pos = torch.arange(len(b), device=dev) - s["cu"].long()[b] + (s["kv_len"].long() - n)[b]
    page, row = s["table"][b, pos // s["case"]["page"]].long(), pos % s["case"]["page"]
    for name in ("k", "v"):
        codes, scale = quantise(s[name])
        s[name + "_pool"][page, row] = codes
        s[name + "_scale"][page, :, row] = scale
    return [s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"]]


def plain_read(s):
    got = []
    for name in ("k", "v"):
        got.append(torch.cat([rows_of(s, name, b) for b in range(len(s["kv"]))]).to(s["dtype"]))
    return got


def plain_attention(s):
    """Every sequence's new tokens against its cached rows, some queries at a time."""
    c = s["case"]
    G, Hkv, Dv = c["Hq"] // c["Hkv"], c["Hkv"], c["Dv"]
    q = s["q"]
    o = torch.empty((q.shape[0], c["Hq"], Dv), dtype=q.dtype, device=q.device)
    lse = torch.empty((c["Hq"], q.shape[0]), device=q.device)
    at = 0
    for b, (n, L) in enumerate(zip(s["new"], s["kv"])):
        k = rows_of(s, "k", b).permute(1, 2, 0)                    # [Hkv, D, L]
        v = rows_of(s, "v", b).transpose(0, 1)                     # [Hkv, L, Dv]
        step = max(1, (1 << 29) // (c["Hq"] * L))
        for i in range(0, n, step):
            m = min(step, n - i)
            x = q[at + i:at + i + m].float().view(m, Hkv, G, -1).permute(1, 2, 0, 3).reshape(Hkv, G * m, -1)
            x = torch.matmul(x * s["scale"], k).view(Hkv, G, m, L)
            if c["causal"]:
                pos = torch.arange(L - n + i, L - n + i + m, device=q.device)
                x.masked_fill_(torch.arange(L, device=q.device) > pos[:, None], -math.inf)
            top = x.amax(-1, keepdim=True)
            x = x.sub_(top).exp_()
            total = x.sum(-1, keepdim=True)
            y = torch.matmul(x.view(Hkv, G * m, L), v).view(Hkv, G, m, Dv) / total
            o[at + i:at + i + m] = y.permute(2, 0, 1, 3).reshape(m, c["Hq"], Dv).to(q.dtype)
            lse[:, at + i:at + i + m] = (top + total.log()).reshape(c["Hq"], m)
        at += n
    return o, lse


def run(s):
    op = s["op"]
    if not own:
        if op == "write":
            return plain_write(s)
        if op == "read":
            return plain_read(s)
        o, lse = plain_attention(s)
        return [o, lse.t().contiguous() if op == "decode" else lse]
    import flash_attention_forward_gb300 as fa
    if op == "write":
        fa.sdpa_cache_write_fp8(s["k"], s["v"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["table"],
                                s["kv_len"], s["cu"])
        return [s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"]]
    if op == "read":
        return fa.sdpa_cache_read_fp8(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["table"], s["cu"],
                                      s["total"], dtype=s["dtype"])
    if op == "decode":
        return fa.sdpa_decode_paged_fp8(s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["table"],
                                        s["kv_len"], scale=s["scale"])
    if op == "chunk":
        return fa.sdpa_fwd_paged(s["q"], s["k_pool"], s["v_pool"], s["table"], s["kv_len"], s["cu"], s["max_new"],
                                 scale=s["scale"], causal=s["case"]["causal"])
    return fa.sdpa_fwd_paged_fp8(s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["table"],
                                 s["kv_len"], s["cu"], s["max_new"], scale=s["scale"], causal=s["case"]["causal"])


def exact(case, seed):
    """The same outputs from the definitions, in 64 bits, a sequence and a KV head at a time."""
    if work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    page, op = case["page"], case["op"]
    table = s["table"].tolist()

    def values(name, b, h):
        """Rows [kv_len, D] of head h of sequence b, gathered by flat row number."""
        t = torch.arange(s["kv"][b], device="cuda")
        flat = torch.tensor(table[b], device="cuda")[t // page] * page + t % page
        pool = s[name + "_pool"]
        x = pool[:, :, h].reshape(-1, pool.shape[-1])[flat].double()
        if name + "_scale" in s:
            x *= s[name + "_scale"][:, h].reshape(-1)[flat].double()[:, None]
        return x

    if op == "write":
        for name in ("k", "v"):
            x = s[name].double()
            top = x.abs().amax(-1)
            e = torch.where(top > 0, torch.ceil(torch.log2(top / E4M3_MAX)), torch.full_like(top, float(MIN_EXP)))
            # a logarithm next to a whole number may fall on either side of it
            e = torch.where(top > E4M3_MAX * torch.exp2(e), e + 1, e)
            e = torch.where(top <= E4M3_MAX * torch.exp2(e - 1), e - 1, e).clamp(min=MIN_EXP)
            y = x / torch.exp2(e)[..., None]
            # e4m3: 3 bits behind the leading one, steps of 2^-9 below 2^-6
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
            y = torch.round(y / step) * step
            at = 0
            for b, n in enumerate(s["new"]):
                t = torch.arange(s["kv"][b] - n, s["kv"][b], device="cuda")
                p, r = torch.tensor(table[b], device="cuda")[t // page], t % page
                s[name + "_pool"][p, r] = y[at:at + n].float().to(torch.float8_e4m3fn)
                s[name + "_scale"][p, :, r] = torch.exp2(e[at:at + n]).float()
                at += n
        return [s["k_pool"].float().double(), s["v_pool"].float().double(), s["k_scale"].double(), s["v_scale"].double()]
    if op == "read":
        return [torch.cat([torch.stack([values(n, b, h) for h in range(case["Hkv"])], 1) for b in range(case["B"])])
                for n in ("k", "v")]
    G = case["Hq"] // case["Hkv"]
    o = torch.zeros((s["q"].shape[0], case["Hq"], case["Dv"]), dtype=torch.float64, device="cuda")
    lse = torch.zeros((case["Hq"], s["q"].shape[0]), dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, L) in enumerate(zip(s["new"], s["kv"])):
        for h in range(case["Hkv"]):
            k, v = values("k", b, h), values("v", b, h)
            for j in range(h * G, (h + 1) * G):
                for i in range(0, n, 4096):
                    m = min(4096, n - i)
                    x = torch.einsum("md,ld->ml", s["q"][at + i:at + i + m, j].double(), k) * s["scale"]
                    if case["causal"]:
                        x += torch.full_like(x, -math.inf).triu(L - n + i + 1)
                    lse[j, at + i:at + i + m] = torch.logsumexp(x, -1)
                    o[at + i:at + i + m, j] = torch.exp(x - lse[j, at + i:at + i + m, None]) @ v
        at += n
    return [o, lse.t().contiguous() if op == "decode" else lse]
