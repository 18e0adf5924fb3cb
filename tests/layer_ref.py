"""Plain 64-bit implementations of the operators between two linears (torch,
any device), written from their definitions, and the bounds their tests use.

Rounding to type t is off by at most half a step, u(t) = finfo(t).eps / 2
relative to the value: fp32 2^-24, bf16 2^-8, fp16 2^-11, e4m3 2^-4 (and half a
subnormal step, 2^-10, near zero)."""
import math

import torch

F8 = torch.float64
FP8 = torch.float8_e4m3fn
U32, UBF16, UFP16 = 2.0 ** -24, 2.0 ** -8, 2.0 ** -11
QMAX = {0: 127.0, 1: 448.0}


def decode(codes, dtype):
    """Codes (uint8) -> float64 values."""
    return codes.view(torch.int8 if dtype == 0 else FP8).to(torch.float32).to(F8)


def encode(x32, s32, dtype):
    """Codes of fp32 x with fp32 scale s > 0 (broadcast): one IEEE division,
    round to nearest even, saturation; s == 0 gives 0."""
    c = torch.where(s32 > 0, x32 / torch.where(s32 > 0, s32, 1.0), 0.0)
    if dtype == 0:
        return c.round().clamp(-128, 127).to(torch.int8).view(torch.uint8)
    return c.clamp(-448, 448).to(FP8).view(torch.uint8)


# ---- norm ---------------------------------------------------------------------

def rmsnorm(x, w, eps, res=None, w_off=0.0):
    """(r as bf16, y in 64 bits)."""
    r = x if res is None else (x.float() + res.float()).bfloat16()
    d = r.to(F8)
    y = d / torch.sqrt(d.square().mean(1, keepdim=True) + eps) * (w.to(F8) + w_off)
    return r, y


def norm_rel(K):
    """Relative error of the kernel's fp32 y: at most ceil(K/32) + 40 roundings of
    partial sums (all terms positive) halved by the root, and ten more of the
    division, root and products."""
    return (0.5 * (K / 32 + 40) + 10) * U32


def check_codes(q, s, y, group, dtype, rel):
    """q [M, K], s [Kb, M] against y in 64 bits: s is amax / Q and each code
    lies within half a step of y / s, up to the fp32 error of y."""
    M, K = y.shape
    c = decode(q, dtype)
    for g in range(-(-K // group)):
        a, cg = y[:, g * group:(g + 1) * group], c[:, g * group:(g + 1) * group]
        s64 = a.abs().amax(1) / QMAX[dtype]
        err = (s[g].to(F8) - s64).abs()
        assert (err <= s64 * (rel + 2 * U32) + 2.0 ** -149).all(), f"scale of group {g}"
        n = a / torch.where(s64 > 0, s64, 1.0)[:, None]
        step = torch.full_like(n, 0.5) if dtype == 0 else \
            torch.maximum(n.abs() * 2.0 ** -4, torch.full_like(n, 2.0 ** -10))
        tol = step + n.abs() * (2 * rel + 8 * U32)
        bad = (cg - n).abs() > tol
        assert not bad.any(), (f"group {g}: {int(bad.sum())} codes off, first "
                               f"{cg[bad][0].item()} for {n[bad][0].item()}")


# ---- rotary positions ------------------------------------------------------------

def rope(x, pos, turns, layout, mscale):
    out, half = x.to(F8).clone(), turns.shape[0]
    t = pos.to(F8)[:, None] * turns[None]
    ang = (t - torch.floor(t)) * (2 * math.pi)
    c, s = torch.cos(ang)[:, None] * mscale, torch.sin(ang)[:, None] * mscale
    ia = torch.arange(half, device=x.device) * (1 if layout == 0 else 2)
    ib = ia + (half if layout == 0 else 1)
    a, b = out[..., ia].clone(), out[..., ib].clone()
    out[..., ia] = a * c - b * s
    out[..., ib] = b * c + a * s
    mag = torch.zeros_like(out)
    mag[..., ia] = (a.abs() + b.abs()) * mscale
    mag[..., ib] = mag[..., ia]
    return out, mag


# ---- cache -----------------------------------------------------------------------

def append(codes, scales, x, off, lens, table, dtype):
    """The cache's codes [P, H, page, D] and scales after one call, block by block."""
    codes, scales = codes.clone(), scales.clone()
    P, H, page, D = codes.shape
    bt = page // scales.shape[2]
    off, lens, table = off.tolist(), lens.tolist(), table.tolist()
    for b in range(len(lens)):
        n = off[b + 1] - off[b]
        first, p, row = lens[b] - n, lens[b] - n, off[b]
        while p < lens[b]:
            stop = min(lens[b], (p // bt + 1) * bt)
            pg, a = table[b][p // page], p % page
            t0, sub = a // bt * bt, a // bt
            new = x[row:row + stop - p].float().transpose(0, 1)           # [H, n, D]
            s_old = scales[pg, :, sub] if a > t0 else torch.zeros_like(scales[pg, :, sub])
            amax = new.abs().amax((1, 2))
            # by a tensor: torch multiplies by the reciprocal of a number
            s_new = torch.maximum(s_old, amax / torch.full_like(amax, QMAX[dtype]))
            old = decode(codes[pg, :, t0:a], dtype).float() * s_old[:, None, None]
            again = encode(old, s_new[:, None, None], dtype)
            grew = (s_new > s_old)[:, None, None]
            codes[pg, :, t0:a] = torch.where(grew, again, codes[pg, :, t0:a])
            codes[pg, :, a:a + stop - p] = encode(new, s_new[:, None, None], dtype)
            scales[pg, :, sub] = s_new
            row, p = row + stop - p, stop
        assert p == max(lens[b], first)
    return codes, scales


# ---- attention ---------------------------------------------------------------------

def attention(q, codes_k, codes_v, ks, vs, off, lens, table, dtype, scale=None, causal=True,
              window=0):
    """(out, lse, tol, lse_tol) in 64 bits for the rows of the sequences; tol and
    lse_tol bound the error of a kernel's bf16 output and fp32 lse.

    Bound: a score's error is at most e = (2 D + 16) u32 * scale * sum |q k|
    (D products and sums, the scales) + 2^-20 (exp2 and its argument, whose
    size is below 2^4 where p matters); it changes each weight by 2 e relative,
    numerator and denominator together.  A kernel may round the weights to fp16
    (2^-11 relative, 2^-25 absolute below its normal range, relative to the
    largest weight times its value scale) and sums them in fp32.  The lse has
    the scores' error, that of the fp32 sum, and of a logarithm and one sum."""
    T, H, D = q.shape
    page, Hk = codes_k.shape[2], codes_k.shape[1]
    bt = page // ks.shape[2]
    scale = 1 / math.sqrt(D) if scale is None else scale
    out = torch.zeros(T, H, D, dtype=F8, device=q.device)
    lse = torch.full((T, H), -math.inf, dtype=F8, device=q.device)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    o, ls = off.tolist(), lens.tolist()
    for b in range(len(ls)):
        n, L = o[b + 1] - o[b], ls[b]
        if n == 0 or L == 0:
            continue
        ids = table[b, :-(-L // page)].long()
        pos = torch.arange(L - n, L, device=q.device)[:, None]
        j = torch.arange(L, device=q.device)[None]
        seen = torch.ones(n, L, dtype=torch.bool, device=q.device)
        if causal:
            seen = seen & (j <= pos)
        if window:
            seen = seen & (j > pos - window)
        for h in range(Hk):
            def rows(c, s):
                v = decode(c[ids, h], dtype) * s[ids, h].to(F8).repeat_interleave(bt, 1)[..., None]
                return v.reshape(-1, D)[:L]
            k, v = rows(codes_k, ks), rows(codes_v, vs)
            for e in range(h * (H // Hk), (h + 1) * (H // Hk)):
                qq = q[o[b]:o[b + 1], e].to(F8)
                z = (qq @ k.t() * scale).masked_fill(~seen, -math.inf)
                err = ((2 * D + 16) * U32 * abs(scale) * (qq.abs() @ k.abs().t()))
                err = err.masked_fill(~seen, 0).amax(1, keepdim=True) + 2.0 ** -20
                any_ = seen.any(1, keepdim=True)
                p = torch.where(any_, torch.softmax(z, 1), 0.0)
                p = torch.where(seen, p, 0.0)
                r = p @ v
                out[o[b]:o[b + 1], e] = r
                lse[o[b]:o[b + 1], e] = torch.where(any_[:, 0], torch.logsumexp(z, 1), -math.inf)
                ltol[o[b]:o[b + 1], e] = err[:, 0] + L * U32 + 4 * U32 * z.masked_fill(
                    ~seen, 0).abs().amax(1) + 8 * U32
                vmax = (v.abs().amax() if L else 0.0)
                tol[o[b]:o[b + 1], e] = (UBF16 * r.abs() + (2 * err + 2 * UFP16 + L * U32)
                                         * (p @ v.abs()) + L * 2.0 ** -25 * vmax)
    return out, lse, tol, ltol
