"""The operators between two linears at the edges of their ranges: a long tail under
a dominating key, scales far apart, zeros with a sign, values that are not numbers,
more rows than a launch has CTAs."""
import math

import pytest
import torch

import block_scaled_w8a8_b200 as bq
import layer_ref as ref
from test_layer_ops import L, gen, make_batch, randn, random_cache    # noqa: F401 (L: a fixture)

gpu = pytest.mark.gpu
F8 = torch.float64


# ---- attention --------------------------------------------------------------------

def attention_and_bounds(q, c, off, lens, table, scale):
    """(out, lse, their bounds) of causal attention in 64 bits, row by row.

    A weight w_j = softmax_j * vs_j may be rounded to fp16: by 2^-11 of itself, or by
    2^-33 of the row's largest below fp16's normal range, where a kernel's largest weight is 2^8 or
    more.  A score's error e is that of layer_ref.attention, with 2^-23 of the largest
    exponent (scores, scales and references in log2 units) for exp2 and its argument;
    sums are fp32.  Value scales below 2^-80 may count as 2^-80."""
    D, H, Hk = q.shape[2], q.shape[1], c.k.shape[1]
    page, bt = c.k.shape[2], c.k.shape[2] // c.ks.shape[2]
    out, lse = torch.zeros(*q.shape, dtype=F8, device="cuda"), torch.zeros(q.shape[:2], dtype=F8, device="cuda")
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    o, ls = off.tolist(), lens.tolist()
    for b in range(len(ls)):
        n, len_ = o[b + 1] - o[b], ls[b]
        ids = table[b, :-(-len_ // page)].long()
        seen = (torch.arange(len_, device="cuda")[None] <=
                torch.arange(len_ - n, len_, device="cuda")[:, None])
        for h in range(H):
            hk = h // (H // Hk)

            def rows(codes, s):
                return (ref.decode(codes[ids, hk], c.dtype).reshape(-1, D)[:len_],
                        s[ids, hk].to(F8).repeat_interleave(bt, 1).reshape(-1)[:len_])
            (k, ks), (v, vs) = rows(c.k, c.ks), rows(c.v, c.vs)
            qq, at = q[o[b]:o[b + 1], h].to(F8), slice(o[b], o[b + 1])
            z = (qq @ (k * ks[:, None]).t() * scale).masked_fill(~seen, -math.inf)
            zmax = z.masked_fill(~seen, 0).abs().amax(1, keepdim=True) / math.log(2)
            lg = vs.clamp(min=2.0 ** -80).log2().abs().max()
            e = ((2 * D + 16) * ref.U32 * abs(scale) * (qq.abs() @ (k.abs() * ks[:, None]).t())).masked_fill(
                ~seen, 0).amax(1, keepdim=True) + (2 * zmax + 2 * lg + 64) * 2.0 ** -23
            p = torch.softmax(z, 1)
            w, small = p * vs, p * torch.where(vs < 2.0 ** -80, 2.0 ** -80, 0.0)
            out[at, h] = w @ v
            lse[at, h] = torch.logsumexp(z, 1)
            tol[at, h] = (ref.UBF16 * out[at, h].abs() + (2 * e + ref.UFP16 + 2 * len_ * ref.U32) *
                          (w @ v.abs()) + small @ v.abs() +
                          2.0 ** -33 * w.amax(1, keepdim=True) * (seen.to(F8) @ v.abs()))
            ltol[at, h] = (e + 8 * ref.U32 * (zmax + lg + 64))[:, 0] + 2 * len_ * ref.U32
    return out, lse, tol, ltol


def check(q, c, off, lens, table, scale):
    want, lse_w, tol, ltol = attention_and_bounds(q, c, off, lens, table, scale)
    lse = torch.zeros(q.shape[:2], device="cuda")
    got = bq.kv_attention(q, c, off, lens, table, int((off[1:] - off[:-1]).max()), int(lens.max()), scale,
                          lse=lse)
    bq.check_device_status()
    d, dl = (got.to(F8) - want).abs(), (lse.to(F8) - lse_w).abs()
    assert (d <= tol).all(), (f"{int((d > tol).sum())} of {d.numel()} off, the worst by "
                              f"{(d / tol).nan_to_num(math.inf).max().item()} of the bound")
    assert (dl <= ltol).all(), f"lse off by {(dl / ltol).max().item()} of its bound"


# new tokens, lengths, Hq, Hk, D, page, bt: each kernel, and each way it groups scales
KERNELS = [([1, 1], [5000, 700], 2, 1, 128, 64, 16), ([1, 2], [3000, 1200], 4, 2, 128, 32, 8),
           ([1, 1], [5000, 700], 4, 1, 64, 64, 32), ([2, 1], [4000, 700], 4, 1, 64, 64, 16),
           ([1, 1], [5000, 700], 4, 1, 64, 32, 4), ([40], [3000], 2, 1, 128, 64, 64),
           ([40, 30], [2500, 900], 2, 1, 128, 64, 16), ([30], [2500], 4, 2, 128, 32, 8),
           ([60], [2500], 2, 1, 64, 128, 64), ([60], [2500], 2, 1, 64, 32, 32), ([60], [2500], 2, 1, 64, 16, 2),
           ([1, 1], [3000, 700], 2, 1, 96, 32, 16)]
IDS = ["n%s-l%s-h%d.%d-d%d-p%d.%d" % ("+".join(map(str, c[0])), "+".join(map(str, c[1])), *c[2:]) for c in KERNELS]


@gpu
@pytest.mark.parametrize("dtype", [bq.INT8, bq.FP8_E4M3])
@pytest.mark.parametrize("gap", [20.4, 23.42, 24.0])
@pytest.mark.parametrize("case", KERNELS, ids=IDS)
def test_a_tail_under_dominating_keys_keeps_its_sum(L, case, gap, dtype):    # noqa: F811
    """Every sixteenth key has a score `gap` binary places above all others and a value of
    zero, so that the output is made of the others' weights alone."""
    new, lens, Hq, Hk, D, page, bt = case
    g = gen(D + bt)
    off, ln, table, count = make_batch(g, new, lens, page)
    c = bq.kv_cache(count, Hk, page, D, bt, dtype)
    top = torch.arange(page, device="cuda") % 16 == 0
    c.k[:, :, top, 0] = 1 if dtype == bq.INT8 else 0x38                      # 1.0; all others 0
    v = torch.randint(64, 127, c.v.shape, generator=g, device="cuda", dtype=torch.uint8)
    c.v.copy_(torch.where(top[:, None], 0, v))
    c.ks.fill_(1.0)
    c.vs.fill_(1 / 127)
    q = randn(g, sum(new), Hq, D).bfloat16()
    q[..., 0] = 1
    check(q, c, off, ln, table, gap * math.log(2))
