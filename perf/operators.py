"""What is measured of the operators between two block-scaled linears of a
decoder layer: the RMS norm with an 8-bit output, rotary positions, the write
of new keys and values into an 8-bit paged cache, and the attention that reads
it.  Each has its plain form (elementary torch operations in 32 bits, angles in
64) and, where `own` is true, the library's call; `exact` computes the same
from the definitions in 64 bits.

A case's "op" names the operator:
  norm    q, s = quantise(rms_norm(bf16(x + res)) * w), res' = bf16(x + res)
  rope    the first `rot` dimensions of each head turned by position * frequency
  append  n new tokens of each sequence into the cache
  attn    queries of each sequence against its cached keys and values
"""
import math

import torch

own = False

QMAX = {"int8": 127.0, "fp8": 448.0}
FP8 = torch.float8_e4m3fn


# ---- cases --------------------------------------------------------------------

def listed():
    return [
        # one decode step of 8 sequences: the norm in front of a linear, latency only
        {"name": "norm fp8 8 rows", "op": "norm", "kind": "fp8", "rows": 8, "cols": 4096, "group": 128},
        # a prefill of 4096 tokens in front of an INT8 linear
        {"name": "norm int8 4096 rows", "op": "norm", "kind": "int8", "rows": 4096, "cols": 4096, "group": 128},
        # an odd number of rows as wide as the MLP, in front of an MXFP8 linear
        {"name": "norm mx 2047 rows wide", "op": "norm", "kind": "mx", "rows": 2047, "cols": 14336, "group": 32},
        # one decode step of 64 sequences at far positions: q and k heads of a fused QKV output
        {"name": "rope decode 64", "op": "rope", "tokens": 64, "heads": 40, "dim": 128, "rot": 128,
         "layout": "half", "factor": 1.0, "base": 500000.0, "far": 100000},
        # a long prompt, neighbouring pairs, half of each head, scaled for a long context
        {"name": "rope prefill 8191 partial", "op": "rope", "tokens": 8191, "heads": 40, "dim": 128, "rot": 64,
         "layout": "pairs", "factor": 8.0, "base": 10000.0, "far": 0},
        # one token for each of 64 sequences, most of them into a block that has tokens already
        {"name": "append decode int8 64", "op": "append", "kind": "int8", "batch": 64, "new": 1, "cached": 2048,
         "ragged": True, "kv_heads": 8, "dim": 128, "page": 64, "block": 16},
        # the prompts of four sequences, ragged
        {"name": "append prefill fp8 8192", "op": "append", "kind": "fp8", "batch": 4, "new": 2731, "cached": 77,
         "ragged": True, "kv_heads": 8, "dim": 128, "page": 64, "block": 64},
        # one sequence decoding: latency, few rows, work to be split along the cache
        {"name": "attn decode int8 1x4096", "op": "attn", "kind": "int8", "batch": 1, "new": 1, "cached": 4095,
         "ragged": False, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "block": 16, "window": 0},
        # a full decode batch over ragged caches
        {"name": "attn decode fp8 64x8192", "op": "attn", "kind": "fp8", "batch": 64, "new": 1, "cached": 8191,
         "ragged": True, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "block": 64, "window": 0},
        # a very long context decoding, small heads
        {"name": "attn decode int8 2x131071", "op": "attn", "kind": "int8", "batch": 2, "new": 1, "cached": 131070,
         "ragged": True, "heads": 32, "kv_heads": 8, "dim": 64, "page": 32, "block": 32, "window": 0},
        # chunked prefill: pieces of three prompts over what is cached, sliding window
        {"name": "attn chunk fp8 3x512", "op": "attn", "kind": "fp8", "batch": 3, "new": 513, "cached": 6000,
         "ragged": True, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "block": 16, "window": 4096},
        # a whole prompt
        {"name": "attn prefill int8 8192", "op": "attn", "kind": "int8", "batch": 1, "new": 8192, "cached": 0,
         "ragged": False, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "block": 64, "window": 0},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "rope", "append", "attn", "attn"])
    if op == "norm":
        kind = rng.choice(["int8", "fp8", "mx"])
        cols = 128 * _log(rng, 4, 112) + (0 if kind == "mx" else rng.choice([0, 0, 8, 57]))
        group = 32 if kind == "mx" else rng.choice([128, 128, 64, cols])
        return {"op": op, "kind": kind, "rows": _log(rng, 1, 29360128 // cols), "cols": cols, "group": group}
    dim = rng.choice([64, 128])
    if op == "rope":
        return {"op": op, "tokens": _log(rng, 1, 8191), "heads": rng.randint(1, 40), "dim": dim,
                "rot": rng.choice([dim, dim // 2, dim // 4]), "layout": rng.choice(["half", "pairs"]),
                "factor": rng.choice([1.0, 4.0, 8.0]), "base": rng.choice([10000.0, 500000.0]),
                "far": rng.choice([0, 1000, 100000, 1000000])}
    kind, kv_heads = rng.choice(["int8", "fp8"]), rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    c = {"op": op, "kind": kind, "kv_heads": kv_heads, "dim": dim, "page": page,
         "block": rng.choice([b for b in (1, 8, 16, 32, 64) if page % b == 0]), "ragged": rng.random() < 0.7}
    if op == "append":
        c["batch"] = _log(rng, 1, 64)
        c["new"] = 1 if rng.random() < 0.4 else _log(rng, 1, max(1, 10000 // c["batch"]))
        c["cached"] = _log(rng, 1, 4096) - 1
        return c
    c["heads"] = kv_heads * rng.choice([g for g in (1, 2, 4, 5, 8) if g * kv_heads <= 40])
    c["window"] = 0 if rng.random() < 0.7 else _log(rng, 1, 4096)
    if rng.random() < 0.6:
        c["batch"], c["new"] = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 4])
        c["cached"] = _log(rng, 1, min(131072, 500000 // c["batch"])) - 1
    else:
        c["batch"] = _log(rng, 1, 8)
        c["new"] = _log(rng, 5, 6000 // c["batch"])
        c["cached"] = _log(rng, 1, 8000 // c["batch"]) - 1
    return c


def _lens(case):
    """(new tokens, tokens cached before) of each sequence: whole numbers that the case alone fixes."""
    b, n, c = case["batch"], case["new"], case["cached"]
    if not case["ragged"]:
        return [n] * b, [c] * b
    part = [((i * 40503 + 12829) % 65536) / 65536.0 for i in range(b)]
    new = [max(1, n - int(p * n * 0.6)) for p in part]
    old = [c - int(((p * 7.0) % 1.0) * c * 0.75) for p in part]
    new[0], old[0] = n, c
    return new, old


# ---- inputs --------------------------------------------------------------------

def _codes(shape, kind, gen):
    """Codes as a quantiser leaves them: the values bell-shaped, the largest near the type's end."""
    x = torch.empty(shape, dtype=torch.float16, device="cuda").normal_(generator=gen)
    if kind == "int8":
        return x.mul_(36.0).round_().clamp_(-127, 127).to(torch.int8).view(torch.uint8)
    return x.mul_(120.0).clamp_(-448, 448).to(FP8).view(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    st = {"case": case}
    if case["op"] == "norm":
        m, k = case["rows"], case["cols"]
        hot = torch.where(torch.rand(k, generator=gen, device="cuda") < 0.01, 20.0, 1.0)  # channels far larger than the rest
        st["x"] = normal(m, k).bfloat16()
        st["res"] = (normal(m, k) * 3.0 * hot).bfloat16()
        st["w"] = (1.0 + 0.2 * normal(k)).bfloat16()
        st["sf"] = torch.zeros(-(-m // 128) * (k // 128) * 512, dtype=torch.uint8, device="cuda") if case["kind"] == "mx" else None
        return st
    if case["op"] == "rope":
        t, h, d = case["tokens"], case["heads"], case["dim"]
        st["x"] = normal(t, h * d + 2 * d)[:, : h * d].bfloat16().view(t, h, d)
        order = torch.randperm(t, generator=gen, device="cuda").to(torch.int32)
        st["pos"] = torch.randint(0, case["far"], (t,), generator=gen, device="cuda", dtype=torch.int32) if case["far"] else order
        half = case["rot"] // 2
        i = torch.arange(half, dtype=torch.float64, device="cuda")
        st["freqs"] = case["base"] ** (-i / half) / case["factor"] / (2.0 * math.pi)  # turns for each position
        st["mscale"] = 1.0 + 0.1 * math.log(case["factor"])
        return st
    new, old = _lens(case)
    b, hk, d, page, block = case["batch"], case["kv_heads"], case["dim"], case["page"], case["block"]
    total = [n + c for n, c in zip(new, old)]
    pages = [-(-n // page) for n in total]
    count = sum(pages) + 3
    order = torch.randperm(count, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(b, max(pages), dtype=torch.int32, device="cuda")
    at = 0
    for i in range(b):
        table[i, : pages[i]] = order[at : at + pages[i]]
        at += pages[i]
    st["table"] = table
    st["offsets"] = torch.tensor([sum(new[:i]) for i in range(b + 1)], dtype=torch.int32, device="cuda")
    st["lens"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    st["kc"], st["vc"] = (_codes((count, hk, page, d), case["kind"], gen) for _ in range(2))
    st["ks"], st["vs"] = (
        (3.0 + torch.rand(count, hk, page // block, generator=gen, device="cuda")) / QMAX[case["kind"]] for _ in range(2))
    rows = sum(new)
    if case["op"] == "append":
        st["k"], st["v"] = (normal(rows, hk * d).bfloat16().view(rows, hk, d) for _ in range(2))
        st["units"] = sum((c + n - 1) // block - c // block + 1 for n, c in zip(new, old))
    else:
        st["q"] = normal(rows, case["heads"] * d).bfloat16().view(rows, case["heads"], d)
        st["max_new"], st["max_len"] = max(new), max(total)
    return st


# ---- one pass -------------------------------------------------------------------

def run(st):
    return {"norm": _norm, "rope": _rope, "append": _append, "attn": _attn}[st["case"]["op"]](st)


def _norm(st):
    case = st["case"]
    kind, k, group = case["kind"], case["cols"], case["group"]
    m = case["rows"]
    if own:
        import block_scaled_w8a8_b200 as bq
        if kind == "mx":
            q, sf, res = bq.mx_rmsnorm_quant(st["x"], st["w"], eps=1e-6, residual=st["res"], sf=st["sf"])
            return q.view(FP8), sf.view(torch.float8_e8m0fnu), res
        q, s, res = bq.rmsnorm_quant(st["x"], st["w"], eps=1e-6, residual=st["res"], group_k=group,
                                     dtype=bq.INT8 if kind == "int8" else bq.FP8_E4M3)
        if kind == "fp8":
            return q.view(FP8), s, res
        return _values(q.view(torch.int8), s, group), s, res
    res = (st["x"].float() + st["res"].float()).bfloat16()
    r = res.float()
    y = r * torch.rsqrt((r * r).mean(1, keepdim=True) + 1e-6) * st["w"].float()
    if kind == "mx":
        a = y.view(m, k // 32, 32)
        amax = a.abs().amax(2)
        e = (torch.frexp(amax)[1] - 1 - 8).clamp(-127, 127)          # floor(log2 amax) - 8
        q = torch.ldexp(a, -e[..., None]).clamp(-448, 448).to(FP8)
        byte = torch.where(amax > 0, e + 127, 0).to(torch.uint8)
        full = st["sf"].view(-(-m // 128), k // 128, 32, 4, 4).permute(0, 3, 2, 1, 4)   # row block, 32s, row, K block, group
        rows = torch.zeros(full.shape[0] * 128, k // 32, dtype=torch.uint8, device=y.device)
        rows[:m] = byte
        full.copy_(rows.view(full.shape))
        return q.view(m, k), st["sf"].view(torch.float8_e8m0fnu), res
    kb = -(-k // group)
    a = torch.nn.functional.pad(y, (0, kb * group - k)).view(m, kb, group)
    s = _over_q(a.abs().amax(2), kind)
    c = torch.where(s[..., None] > 0, a / s[..., None], 0.0)
    c = c.round().clamp(-128, 127).to(torch.int8) if kind == "int8" else c.clamp(-448, 448).to(FP8)
    q = c.view(torch.uint8).view(m, kb * group)[:, :k].contiguous()
    s = s.t().contiguous()
    return (q.view(FP8) if kind == "fp8" else _values(q.view(torch.int8), s, group)), s, res


def _over_q(amax, kind):
    """amax / Q, one division (by a tensor: torch multiplies by the reciprocal of a number)."""
    return amax / torch.full_like(amax, QMAX[kind])


def _values(c, s, group):
    """What INT8 codes [M, K] with scales [Kb, M] stand for, as bf16."""
    m, k = c.shape
    out = torch.empty(m, k, dtype=torch.bfloat16, device=c.device)
    if k % group == 0:
        torch.mul(c.view(m, k // group, group), s.t()[..., None], out=out.view(m, k // group, group))
    else:
        torch.mul(c, s.t().repeat_interleave(group, dim=1, output_size=s.shape[0] * group)[:, :k], out=out)
    return out


def _rope(st):
    case = st["case"]
    if own:
        import block_scaled_w8a8_b200 as bq
        return bq.rope(st["x"], st["pos"], st["freqs"], mscale=st["mscale"],
                       layout=bq.ROPE_HALF if case["layout"] == "half" else bq.ROPE_INTERLEAVED)
    x = st["x"].float()
    half = case["rot"] // 2
    turns = st["pos"].double()[:, None] * st["freqs"][None]
    angle = (turns - turns.floor()) * (2.0 * math.pi)
    cos, sin = (f(angle).float()[:, None] * st["mscale"] for f in (torch.cos, torch.sin))
    if case["layout"] == "half":
        a, b = x[..., :half], x[..., half : 2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0 : 2 * half : 2], x[..., 1 : 2 * half : 2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(2)
    return torch.cat([turned, x[..., 2 * half :]], -1).bfloat16()


def _append(st):
    case = st["case"]
    kind, page, block = case["kind"], case["page"], case["block"]
    if own:
        import block_scaled_w8a8_b200 as bq
        cache = bq.KvCache(st["kc"], st["vc"], st["ks"], st["vs"], bq.INT8 if kind == "int8" else bq.FP8_E4M3)
        bq.kv_append(cache, st["k"], st["v"], st["offsets"], st["lens"], st["table"])
    else:
        dev, b = st["k"].device, case["batch"]
        new = (st["offsets"][1:] - st["offsets"][:-1]).long()
        old = st["lens"].long() - new
        count = torch.div(old + new - 1, block, rounding_mode="floor") - torch.div(old, block, rounding_mode="floor") + 1
        seq = torch.repeat_interleave(torch.arange(b, device=dev), count, output_size=st["units"])     # of each touched block
        nth = torch.arange(st["units"], device=dev) - (count.cumsum(0) - count)[seq]
        pos = (torch.div(old, block, rounding_mode="floor")[seq] + nth)[:, None] * block + torch.arange(block, device=dev)
        was, is_new = pos < old[seq, None], (pos >= old[seq, None]) & (pos < (old + new)[seq, None])
        where = st["table"][seq, torch.div(pos[:, 0], page, rounding_mode="floor")].long()
        slot, sub = pos % page, torch.div(pos[:, 0] % page, block, rounding_mode="floor")
        row = (st["offsets"][seq, None].long() + pos - old[seq, None]).clamp(0, st["k"].shape[0] - 1)
        for x, codes, scales in ((st["k"], st["kc"], st["ks"]), (st["v"], st["vc"], st["vs"])):
            fresh = torch.where(is_new[..., None, None], x[row].float(), 0.0).transpose(1, 2)         # [U, H, block, D]
            heads = torch.arange(x.shape[1], device=dev)
            before = codes[where[:, None, None], heads[None, :, None], slot[:, None]]
            s0 = torch.where(was.any(1)[:, None], scales[where, :, sub], 0.0)
            s1 = torch.maximum(s0, _over_q(fresh.abs().amax((2, 3)), kind))[..., None, None]
            stood = before.view(torch.int8 if kind == "int8" else FP8).float() * s0[..., None, None]
            c = torch.where(s1 > 0, torch.where(is_new[:, None, :, None], fresh, stood) / s1, 0.0)
            c = c.round().clamp(-128, 127).to(torch.int8) if kind == "int8" else c.clamp(-448, 448).to(FP8)
            put = is_new[:, None, :, None] | (was[:, None, :, None] & (s1 > s0[..., None, None]))
            codes[where[:, None, None], heads[None, :, None], slot[:, None]] = torch.where(put, c.view(torch.uint8), before)
            scales[where, :, sub] = s1[..., 0, 0]
    if kind == "int8":  # the codes are whole numbers and have to be equal
        return st["kc"].view(torch.int8), st["vc"].view(torch.int8), st["ks"], st["vs"]
    return st["kc"].view(FP8), st["vc"].view(FP8), st["ks"], st["vs"]


def _attn(st):
    case = st["case"]
    kind, page, block = case["kind"], case["page"], case["block"]
    if own:
        import block_scaled_w8a8_b200 as bq
        cache = bq.KvCache(st["kc"], st["vc"], st["ks"], st["vs"], bq.INT8 if kind == "int8" else bq.FP8_E4M3)
        return bq.kv_attention(st["q"], cache, st["offsets"], st["lens"], st["table"], st["max_new"], st["max_len"],
                               window=case["window"])
    dev, b, hk, d, g = st["q"].device, case["batch"], case["kv_heads"], case["dim"], case["heads"] // case["kv_heads"]
    n, length = st["max_new"], st["table"].shape[1] * page
    new = (st["offsets"][1:] - st["offsets"][:-1]).long()
    old = st["lens"].long() - new
    i = torch.arange(n, device=dev)
    row = (st["offsets"][:-1, None].long() + i).clamp(max=st["q"].shape[0] - 1)                       # [B, n]
    q = st["q"][row].float().view(b, n, hk, g, d).permute(0, 2, 3, 1, 4).reshape(b, hk, g * n, d)
    table = st["table"].long()

    def spread(codes, scales):
        x = codes.view(torch.int8 if kind == "int8" else FP8)[table].float()                          # [B, pages, H, page, D]
        x = x.view(*x.shape[:3], page // block, block, d).mul_(scales[table][..., None, None])
        return x.view(b, -1, hk, page, d).transpose(1, 2).reshape(b, hk, length, d)

    s = (q @ spread(st["kc"], st["ks"]).transpose(2, 3)).view(b, hk, g, n, length).mul_(1.0 / math.sqrt(d))
    j, pos = torch.arange(length, device=dev), (old[:, None] + i)[:, None, None, :, None]
    seen = (j <= pos) & (j < st["lens"].long()[:, None, None, None, None])
    if case["window"]:
        seen = seen & (j > pos - case["window"])
    s = s.masked_fill_(~seen, -math.inf)
    s = torch.exp(s.sub_(s.amax(-1, keepdim=True).clamp(min=-3e38)))
    total = s.sum(-1, keepdim=True)
    o = s.view(b, hk, g * n, length) @ spread(st["vc"], st["vs"])
    o = o.view(b, hk, g, n, d) / torch.where(total > 0, total, 1.0)
    seq = torch.repeat_interleave(torch.arange(b, device=dev), new, output_size=st["q"].shape[0])
    at = torch.arange(st["q"].shape[0], device=dev) - st["offsets"][seq].long()
    return o[seq, :, :, at].reshape(-1, case["heads"], d).bfloat16()


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    if case["op"] == "norm":
        m, k = case["rows"], case["cols"]
        scales = m * k // 32 if case["kind"] == "mx" else 4 * m * -(-k // case["group"])
        return {"bytes": 7 * m * k + 2 * k + scales, "flops": 6 * m * k}
    if case["op"] == "rope":
        e = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": 4 * e + 4 * case["tokens"] + 4 * case["rot"], "flops": 3 * case["tokens"] * case["heads"] * case["rot"]}
    new, old = _lens(case)
    hk, d, block = case["kv_heads"], case["dim"], case["block"]
    if case["op"] == "append":
        row = hk * d
        held = sum((c % block) for c in old)                 # tokens of a block that a new scale may touch again
        units = sum((c + n - 1) // block - c // block + 1 for n, c in zip(new, old))
        return {"bytes": 2 * (3 * sum(new) * row + held * row + 8 * units * hk), "flops": 6 * sum(new) * row}
    w, moved, pairs = case["window"], 0, 0
    for n, c in zip(new, old):
        first = max(0, c - w + 1) if w else 0
        moved += c + n - first
        if w:
            full = min(n, max(0, c + n - w + 1)) if c + n >= w else 0
            less = n - full                                  # rows at c .. c + less - 1 see all before them
            pairs += full * w + less * c + less * (less + 1) // 2
        else:
            pairs += n * c + n * (n + 1) // 2
    h = case["heads"]
    return {"bytes": 2 * moved * hk * (d + 4.0 / block) + 4 * sum(new) * h * d, "flops": 4 * pairs * h * d}


# ---- the definitions in 64 bits -----------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    f8 = torch.float64
    if case["op"] == "norm":
        m, k, kind = case["rows"], case["cols"], case["kind"]
        res = (st["x"].to(f8) + st["res"].to(f8)).to(torch.bfloat16)
        r = res.to(f8)
        y = r / torch.sqrt(r.square().sum(1, keepdim=True) / k + 1e-6) * st["w"].to(f8)
        group, scales, codes = case["group"], [], []
        for k0 in range(0, k, group):
            a = y[:, k0 : k0 + group]
            top = a.abs().max(1).values
            if kind == "mx":
                e = (torch.floor(torch.log2(top)) - 8).clamp(-127, 127)
                codes.append((a * torch.exp2(-e)[:, None]).clamp(-448, 448).to(FP8).to(f8))
                scales.append(torch.exp2(e))
            else:
                s = top / QMAX[kind]
                c = a / s[:, None]
                scales.append(s)
                codes.append(c.to(FP8).to(f8) if kind == "fp8" else torch.round(c) * s[:, None])
        codes = torch.cat(codes, 1)
        if kind != "mx":
            return codes, torch.stack(scales), res.to(f8)
        out = torch.full((st["sf"].numel(),), 2.0 ** -127, dtype=f8, device=codes.device)
        i, g = torch.arange(m, device=codes.device)[:, None], torch.arange(k // 32, device=codes.device)[None]
        out[((i // 128) * (k // 128) + g // 4) * 512 + 16 * (i % 32) + 4 * (i % 128 // 32) + g % 4] = torch.stack(scales, 1)
        return codes, out, res.to(f8)
    if case["op"] == "rope":
        x, half = st["x"].to(f8), case["rot"] // 2
        angle = torch.remainder(st["pos"].to(f8)[:, None] * st["freqs"], 1.0) * (2.0 * math.pi)
        out = x.clone()
        for i in range(half):
            a, b = (i, i + half) if case["layout"] == "half" else (2 * i, 2 * i + 1)
            c, s = (f(angle[:, i])[:, None] * st["mscale"] for f in (torch.cos, torch.sin))
            out[..., a] = x[..., a] * c - x[..., b] * s
            out[..., b] = x[..., a] * s + x[..., b] * c
        return out
    new, old = _lens(case)
    page, block, d, hk = case["page"], case["block"], case["dim"], case["kv_heads"]
    view = torch.int8 if case["kind"] == "int8" else FP8
    table = st["table"].tolist()
    if case["op"] == "append":
        units = sum((c + n - 1) // block - c // block + 1 for n, c in zip(new, old))
        if units > 4000:
            return None
        got = []
        for x, codes, scales in ((st["k"], st["kc"], st["ks"]), (st["v"], st["vc"], st["vs"])):
            val, sc, row = codes.view(view).to(f8), scales.to(f8), 0
            for b in range(case["batch"]):
                p, end = old[b], old[b] + new[b]
                while p < end:
                    stop = min(end, (p // block + 1) * block)
                    at, a, z = table[b][p // page], p % page, (stop - 1) % page + 1
                    begin, sub = a // block * block, a // block
                    rows = x[row : row + stop - p].to(f8).transpose(0, 1)
                    s0 = sc[at, :, sub].clone() if a > begin else torch.zeros_like(sc[at, :, sub])
                    s1 = torch.maximum(s0, rows.abs().amax((1, 2)) / QMAX[case["kind"]])
                    back = (val[at, :, begin:a] * s0[:, None, None]) / s1[:, None, None]
                    both = torch.cat([torch.where((s1 > s0)[:, None, None], back, val[at, :, begin:a]), rows / s1[:, None, None]], 1)
                    val[at, :, begin:z] = torch.round(both) if case["kind"] == "int8" else both.to(FP8).to(f8)
                    sc[at, :, sub] = s1
                    row, p = row + stop - p, stop
            got.append((val, sc))
        return (None, None, got[0][1], got[1][1]) if case["kind"] == "int8" else (got[0][0], got[1][0], got[0][1], got[1][1])
    h, g = case["heads"], case["heads"] // hk
    out = torch.zeros(sum(new), h, d, dtype=f8, device=st["q"].device)
    row = 0
    for b in range(case["batch"]):
        n, c = new[b], old[b]
        ids = st["table"][b, : -(-(n + c) // page)].long()
        pos, j = torch.arange(c, c + n, device=ids.device)[:, None], torch.arange(n + c, device=ids.device)[None]
        seen = (j <= pos) & ((j > pos - case["window"]) if case["window"] else (j >= 0))
        for t in range(hk):
            k, v = ((codes[ids, t].view(view).to(f8) * scales[ids, t].to(f8).repeat_interleave(block, 1)[..., None]).reshape(-1, d)[: n + c]
                    for codes, scales in ((st["kc"], st["ks"]), (st["vc"], st["vs"])))
            for e in range(t * g, (t + 1) * g):
                s = (st["q"][row : row + n, e].to(f8) @ k.t()) / math.sqrt(d)
                out[row : row + n, e] = torch.softmax(s.masked_fill(~seen, -math.inf), 1) @ v
        row += n
    return out
