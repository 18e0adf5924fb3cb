"""The operators between two linears at the edges of their ranges: a long tail under
a dominating key, scales far apart, zeros with a sign, values that are not numbers,
more rows than a launch has CTAs."""
import ctypes
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
    sums are fp32, in which a key may be lost whose term is below 2^-41 of it."""
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
            lg = vs.clamp(min=2.0 ** -70).log2().abs().max()
            e = ((2 * D + 16) * ref.U32 * abs(scale) * (qq.abs() @ (k.abs() * ks[:, None]).t())).masked_fill(
                ~seen, 0).amax(1, keepdim=True) + (2 * zmax + 2 * lg + 64) * 2.0 ** -23
            p = torch.softmax(z, 1)
            w = p * vs
            out[at, h] = w @ v
            lse[at, h] = torch.logsumexp(z, 1)
            tol[at, h] = (ref.UBF16 * out[at, h].abs() + (2 * e + ref.UFP16 + 2 * len_ * ref.U32) *
                          (w @ v.abs()) +
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


def draw_scales(g, s, how):
    """Value scales [pages, heads, blocks] for one of the ways that they can differ."""
    u = torch.rand(s.shape, generator=g, device="cuda")
    some = torch.rand(s.shape, generator=g, device="cuda") < 0.4
    if how == "zeros":                      # blocks of zeros between ordinary ones
        return torch.where(some, 0.0, 0.01 + u)
    if how == "zeros beside huge":
        return torch.where(some, 0.0, (1 + u) * 2.0 ** 29)
    if how == "outliers":                   # a few blocks far above the others
        return torch.where(u < 0.1, 2.0 ** 20, 0.01)
    if how == "spread":                     # all that the sum is promised for
        return torch.exp2(100 * u - 70)
    if how == "tiny":
        return torch.exp2(-60 - 10 * u)
    assert how == "none"                    # every value is zero
    return torch.zeros_like(u)


@gpu
@pytest.mark.parametrize("dtype", [bq.INT8, bq.FP8_E4M3])
@pytest.mark.parametrize("how", ["zeros", "zeros beside huge", "outliers", "spread", "tiny", "none"])
@pytest.mark.parametrize("case", KERNELS, ids=IDS)
def test_attention_with_scales_far_apart(L, case, how, dtype):               # noqa: F811
    """Blocks of zero keys and of zero values, which are written with a scale of zero, and
    value scales over many powers of two: out and lse."""
    new, lens, Hq, Hk, D, page, bt = case
    g = gen(3 * D + bt)
    off, ln, table, count = make_batch(g, new, lens, page)
    c = random_cache(g, count, Hk, page, D, bt, dtype)
    c.vs.copy_(draw_scales(g, c.vs, how))
    c.ks.mul_(torch.rand(c.ks.shape, generator=g, device="cuda") > 0.3)
    for b, n in enumerate(lens):            # the first and the last block of each sequence
        for t in (0, n - 1):
            c.vs[int(table[b, t // page]), :, t % page // bt] = 0 if how != "tiny" else 2.0 ** -65
    for codes, s in ((c.k, c.ks), (c.v, c.vs)):
        codes.mul_((s != 0).repeat_interleave(bt, 2)[..., None])
    q = randn(g, sum(new), Hq, D).bfloat16()
    check(q, c, off, ln, table, 1 / math.sqrt(D))


@gpu
@pytest.mark.parametrize("dtype", [bq.INT8, bq.FP8_E4M3])
@pytest.mark.parametrize("order", ["huge last", "huge first"])
@pytest.mark.parametrize("case", KERNELS, ids=IDS)
def test_keys_of_zero_value_stay_in_the_sum_beside_huge_ones(L, case, order, dtype):    # noqa: F811
    """Half of the sequence has values of zero, the other half scales of 2^30: references
    that lie 2^100 apart in one kernel, and in the parts that are joined."""
    new, lens, Hq, Hk, D, page, bt = case
    g = gen(5 * D + bt)
    off, ln, table, count = make_batch(g, new, lens, page)
    c = random_cache(g, count, Hk, page, D, bt, dtype)
    c.vs.zero_()
    for b, n in enumerate(lens):
        for t in range(0, n, bt):
            if (t < n // 2) == (order == "huge first"):
                c.vs[int(table[b, t // page]), :, t % page // bt] = 2.0 ** 30
    c.v.mul_((c.vs != 0).repeat_interleave(bt, 2)[..., None])
    q = randn(g, sum(new), Hq, D).bfloat16()
    check(q, c, off, ln, table, 1 / math.sqrt(D))


# ---- cache -------------------------------------------------------------------------

def one_append(k, v, H, D, page, bt, dtype):
    """The cache after one call with all of k, v as a sequence, and what the definition says."""
    T = k.shape[0]
    pages = -(-T // page)
    i32 = dict(dtype=torch.int32, device="cuda")
    off, lens = torch.tensor([0, T], **i32), torch.tensor([T], **i32)
    table = torch.arange(pages, **i32).view(1, pages)
    c = bq.kv_cache(pages, H, page, D, bt, dtype)
    want = [ref.append(a, s, x, off, lens, table, dtype) for a, s, x in ((c.k, c.ks, k), (c.v, c.vs, v))]
    bq.kv_append(c, k, v, off, lens, table)
    bq.check_device_status()
    return c, want


@gpu
@pytest.mark.parametrize("dtype", [bq.INT8, bq.FP8_E4M3])
@pytest.mark.parametrize("H,D,page,bt", [(2, 128, 32, 16), (1, 64, 16, 1), (2, 8, 8, 4), (1, 5, 8, 4),
                                         (1, 256, 128, 128)])
def test_append_keeps_the_sign_of_zero(L, H, D, page, bt, dtype):            # noqa: F811
    """-0, and negative values whose code is a zero, byte for byte."""
    g = gen(D + bt)
    k, v = (randn(g, 3 * page - 1, H, D).bfloat16() for _ in range(2))
    for x in (k, v):
        kind = torch.randint(0, 4, x.shape, generator=g, device="cuda")
        x.copy_(torch.where(kind == 0, -0.0, torch.where(kind == 1, x * 2.0 ** -24, x)))
        x[1].fill_(-0.0)
    c, want = one_append(k, v, H, D, page, bt, dtype)
    for got, scales, (codes, s) in ((c.k, c.ks, want[0]), (c.v, c.vs, want[1])):
        assert torch.equal(got, codes) and torch.equal(scales, s)
    if dtype == bq.FP8_E4M3:
        assert (c.k == 0x80).any() and (c.k == 0).any()


@gpu
@pytest.mark.parametrize("dtype", [bq.INT8, bq.FP8_E4M3])
@pytest.mark.parametrize("H,D,page,bt", [(2, 128, 32, 16), (1, 64, 16, 1), (3, 8, 32, 32), (1, 256, 128, 128)])
def test_append_with_values_that_are_not_numbers(L, H, D, page, bt, dtype):  # noqa: F811
    """A block with a NaN has a NaN scale, at any alignment; all others are what they are
    without it, and the next sequence to use the block finds nothing of it."""
    g = gen(7 * D + bt)
    T = 4 * page - 3
    k, v = (randn(g, T, H, D).bfloat16() for _ in range(2))
    k[0, 0, D // 2] = 3.0
    k[0, 0, 1], v[page + 1, H - 1, D - 1], v[2 * page, 0] = math.nan, -math.nan, math.nan
    _, want = one_append(k.nan_to_num(0.0), v.nan_to_num(0.0), H, D, page, bt, dtype)
    pages = want[0][0].shape[0]

    def shifted(x):                         # an address that no vector load takes
        return torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].view(x.shape).copy_(x)

    def per_block(x):
        full = torch.zeros(pages * page, H, D, dtype=x.dtype, device="cuda")
        full[:T] = x
        return full.view(pages, page // bt, bt, H, D).permute(0, 3, 1, 2, 4).flatten(3).any(3)

    code = 0 if dtype == bq.INT8 else 0x7F
    live = per_block(torch.ones_like(k, dtype=torch.bool))
    for kk, vv in ((k, v), (shifted(k), shifted(v))):
        c, _ = one_append(kk, vv, H, D, page, bt, dtype)
        for x, got, s, (codes, scales) in ((k, c.k, c.ks, want[0]), (v, c.v, c.vs, want[1])):
            bad = per_block(x.isnan())
            assert bad.any() and not bad[live].all()
            assert s[bad].isnan().all() and torch.equal(s[~bad], scales[~bad])
            wide = bad.repeat_interleave(bt, 2)
            assert torch.equal(got[~wide], codes[~wide])
            written = torch.zeros(pages * page, dtype=torch.bool, device="cuda")
            written[:T] = True
            assert (got[wide & written.view(pages, 1, page)] == code).all()
        # a token more does not make the block a number again; its first one does
        i32 = dict(dtype=torch.int32, device="cuda")
        table = torch.arange(pages, **i32).view(1, pages)
        one = torch.ones(1, H, D, dtype=torch.bfloat16, device="cuda")
        if bt > 1:
            bq.kv_append(c, one, one, torch.tensor([0, 1], **i32), torch.tensor([2], **i32), table)
            assert c.ks[0, 0, 0].isnan() and c.vs[0, 0, 0] == c.vs[0, 0, 0]
        bq.kv_append(c, one, one, torch.tensor([0, 1], **i32), torch.tensor([1], **i32), table)
        assert (c.ks[0, :, 0] == 1 / torch.full((1,), ref.QMAX[dtype], device="cuda")).all()
    bq.check_device_status()


@gpu
@pytest.mark.parametrize("dtype", [bq.INT8, bq.FP8_E4M3])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("case", KERNELS, ids=IDS)
def test_attention_shows_values_that_are_not_numbers(L, case, which, dtype):  # noqa: F811
    """A block with a NaN scale makes the rows that see it NaN, and no other sequence."""
    new, lens, Hq, Hk, D, page, bt = case
    new, lens = new[:1] + [3], lens[:1] + [900]
    g = gen(11 * D + bt)
    off, ln, table, count = make_batch(g, new, lens, page)
    c = random_cache(g, count, Hk, page, D, bt, dtype)
    q = randn(g, sum(new), Hq, D).bfloat16()
    clean = bq.kv_attention(q, c, off, ln, table, max(new), max(lens))
    for t in (5, lens[0] // 2, lens[0] - new[0]):          # all rows of the first sequence see them
        s = (c.ks if which == "k" else c.vs)[int(table[0, t // page]), Hk - 1, t % page // bt:][:1]
        kept = s.clone()
        s.fill_(math.nan)
        lse = torch.zeros(sum(new), Hq, device="cuda")
        got = bq.kv_attention(q, c, off, ln, table, max(new), max(lens), lse=lse)
        s.copy_(kept)
        heads = torch.arange(Hq, device="cuda") // (Hq // Hk) == Hk - 1
        assert got[:new[0], heads].isnan().all()
        assert which == "v" or lse[:new[0], heads].isnan().all()
        assert torch.equal(got[:, ~heads], clean[:, ~heads])
        assert torch.equal(got[new[0]:], clean[new[0]:])
    bq.check_device_status()


# ---- norm --------------------------------------------------------------------------

def shifted(x):
    """A copy at an address, and with a row stride, that no vector load takes."""
    M, K = x.shape
    return torch.zeros(M, K + 3, dtype=x.dtype, device="cuda")[:, 1:1 + K].copy_(x)


@gpu
@pytest.mark.parametrize("dtype", [bq.INT8, bq.FP8_E4M3])
@pytest.mark.parametrize("K,group", [(1024, 128), (512, 512), (256, 8)])
def test_norm_with_values_that_are_not_numbers(L, K, group, dtype):          # noqa: F811
    """A NaN makes its row NaN, an infinity its group (the other values are divided by
    infinity), a NaN weight its column's group: in the scales, at any alignment."""
    g = gen(K + group)
    x, w = randn(g, 6, K).bfloat16(), (1 + 0.2 * randn(g, K)).bfloat16()
    clean_q, clean_s = bq.rmsnorm_quant(x, w, group_k=group, dtype=dtype)
    x[1, K - 3], x[2, 5], x[4, K // 2] = math.nan, math.inf, -math.nan
    wn = w.clone()
    wn[K // 2 + 1] = math.nan
    code = 0 if dtype == bq.INT8 else 0x7F
    at = K // 2 // group                    # the group of column K // 2, and of the next one
    for view in (x, shifted(x)):
        q, s = bq.rmsnorm_quant(view, w, group_k=group, dtype=dtype)
        for m in (1, 4):
            assert s[:, m].isnan().all() and (q[m] == code).all()
        assert s[0, 2].isnan() and (s[1:, 2] == 0).all() and (q[2, group:] == 0).all()
        c, n = bq.rmsnorm_quant(view, wn, group_k=group, dtype=dtype)
        for m in (0, 3, 5):
            if view is x:
                assert torch.equal(q[m], clean_q[m]) and torch.equal(s[:, m], clean_s[:, m])
            assert n[at, m].isnan() and not n[:at, m].isnan().any() and not n[at + 1:, m].isnan().any()
            keep = torch.arange(K, device="cuda") // group != at
            assert torch.equal(c[m, keep], q[m, keep])
            assert (c[m, ~keep] == code).all()


@gpu
def test_mx_norm_with_values_that_are_not_numbers(L):                        # noqa: F811
    import gpu_util
    K, g = 256, gen(41)
    x, w = randn(g, 5, K).bfloat16(), (1 + 0.2 * randn(g, K)).bfloat16()
    x[1, 7] = math.nan
    w[40] = math.nan
    got = []
    for view in (x, shifted(x)):
        q, sf = bq.mx_rmsnorm_quant(view, w)
        e = gpu_util.mx_sf_rows(sf, 5, K)
        assert (q[1] == 0x7F).all() and (e[1] == 0).all()
        assert (q[:, 40] & 0x7F == 0x7F).all()
        rest = torch.arange(K, device="cuda") != 40
        assert not (q[[0, 2, 3, 4]][:, rest] & 0x7F == 0x7F).any()
        got.append((q, torch.from_numpy(e)))
    assert all(torch.equal(a, b) for a, b in zip(*got))


@gpu
@pytest.mark.parametrize("dtype", [bq.INT8, bq.FP8_E4M3])
@pytest.mark.parametrize("w_off", [0.0, 1.0])
@pytest.mark.parametrize("M,K,group", [(40, 4096, 128), (9, 512, 512), (7, 200, 8), (3, 20480, 256)])
def test_norm_codes_do_not_depend_on_alignment(L, M, K, group, w_off, dtype):    # noqa: F811
    """The same rows for the vector kernel and the other one: codes bit for bit, ties
    included; scales up to the order of a row's sum (K terms) and its root."""
    g = gen(K + group)
    x = (randn(g, M, K) * 8).round().bfloat16()          # few distinct values: many exact halves
    w = (1 + 0.25 * randn(g, K).round()).bfloat16() - w_off
    x[M // 2] = 0
    x[0, :group] *= 2.0 ** -40
    q, s, h = bq.rmsnorm_quant(x, w, 1e-5, None, group, dtype, w_off, want_h=True)
    q2, s2, h2 = bq.rmsnorm_quant(shifted(x), w, 1e-5, None, group, dtype, w_off, want_h=True)
    assert torch.equal(q, q2)
    rel = 2 * ref.norm_rel(K)
    assert ((s.double() - s2.double()).abs() <= rel * s.double()).all()
    assert ((h.double() - h2.double()).abs() <= (2 * ref.UBF16 + rel) * h.double().abs()).all()


# ---- host calls ----------------------------------------------------------------------

@gpu
def test_arguments_without_a_truth_value_are_refused(L):                     # noqa: F811
    both = torch.tensor([True, False])
    x, w = torch.ones(2, 128, dtype=torch.bfloat16, device="cuda"), torch.ones(128, dtype=torch.bfloat16,
                                                                               device="cuda")
    with pytest.raises(RuntimeError):
        bq.rmsnorm_quant(x, w, want_h=both)
    i32 = dict(dtype=torch.int32, device="cuda")
    c = bq.kv_cache(1, 1, 16, 64)
    out = torch.full((1, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    q = torch.ones_like(out)
    args = (q, c, torch.tensor([0, 1], **i32), torch.ones(1, **i32), torch.zeros(1, 1, **i32), 1, 16)
    with pytest.raises(RuntimeError):
        bq.kv_attention(*args, causal=both, out=out)
    assert (out == 7).all()
    assert (bq.kv_attention(*args, causal=both[:1], out=out) == 0).all()


# ---- more rows than a launch has CTAs, workspaces ---------------------------------------

@gpu
@pytest.mark.parametrize("M,K,group,dtype,off", [
    (1000, 20480, 256, bq.INT8, 0), (1000, 4096, 4096, bq.INT8, 0), (1000, 4096, 4096, bq.FP8_E4M3, 0),
    (2500, 200, 100, bq.INT8, 0), (2500, 200, 100, bq.FP8_E4M3, 0), (2500, 256, 128, bq.INT8, 1),
    (700, 14336, 128, bq.FP8_E4M3, 0)])
def test_norm_of_more_rows_than_ctas(L, M, K, group, dtype, off):            # noqa: F811
    """Every kernel goes through its loop over rows several times, in place of the residual."""
    g = gen(M + K + group)
    x, w = randn(g, M, K).bfloat16(), (1 + 0.2 * randn(g, K)).bfloat16()
    x *= torch.exp2(torch.arange(M, device="cuda") % 7 - 3)[:, None]         # rows of different size
    res = randn(g, M, K + 8).bfloat16()[:, off:off + K]
    r, y = ref.rmsnorm(x, w, 1e-5, res)
    q, s, ro = bq.rmsnorm_quant(x, w, 1e-5, res, group, dtype, res_out=res)
    assert ro is res and torch.equal(res, r)
    ref.check_codes(q, s, y, group, dtype, ref.norm_rel(K))


@gpu
def test_mx_norm_of_more_rows_than_ctas(L):                                  # noqa: F811
    import gpu_util
    M, K, g = 2000, 4096, gen(43)
    x, w = randn(g, M, K).bfloat16(), (1 + 0.2 * randn(g, K)).bfloat16()
    x *= torch.exp2(torch.arange(M, device="cuda") % 7 - 3)[:, None]
    res = randn(g, M, K).bfloat16()
    r, y = ref.rmsnorm(x, w, 1e-6, res)
    q, sf, ro = bq.mx_rmsnorm_quant(x, w, 1e-6, res, res_out=res)
    assert ro is res and torch.equal(res, r)
    rel = ref.norm_rel(K)
    e = torch.from_numpy(gpu_util.mx_sf_rows(sf, M, K)).cuda().double()
    a = y.view(M, K // 32, 32)
    low, high = (torch.floor(torch.log2(a.abs().amax(2) * f)) + 119 for f in (1 - 2 * rel, 1 + 2 * rel))
    assert ((e >= low) & (e <= high)).all()
    n = (a / torch.exp2(e - 127)[..., None]).clamp(-448, 448)
    tol = torch.maximum(n.abs() * 2.0 ** -4, torch.full_like(n, 2.0 ** -10)) + n.abs() * 2 * rel
    assert ((ref.decode(q, 1).view(a.shape) - n).abs() <= tol).all()


@pytest.mark.parametrize("B,T,Hq,Hkv,D,max_q,max_kv", [
    (1, 1, 32, 8, 128, 1, 1 << 17), (2, 2, 4, 4, 64, 1, 1 << 17), (1, 64, 4, 4, 128, 64, 6000),
    (1, 1, 8, 8, 96, 1, 4000)])
def test_split_keys_have_a_workspace(L, B, T, Hq, Hkv, D, max_q, max_kv):    # noqa: F811
    """Long keys of few rows are split, so the workspace holds at least two parts of each
    row behind the 64 KiB left alone; it grows with the keys and refuses less."""
    n = bq.kv_attention_workspace_size(B, T, Hq, Hkv, D, max_q, max_kv, 64, 16)
    assert n >= 65536 + 2 * T * Hq * (D + 2) * 4
    assert bq.kv_attention_workspace_size(B, T, Hq, Hkv, D, max_q, 16, 64, 16) <= n
    fake = ctypes.c_void_p
    cols = -(-max_kv // 64)
    args = [fake(0x1000), Hq * D, D, fake(0x1000), fake(0x1000), fake(0x1000), cols, cols, B, T, Hq, Hkv, D,
            max_q, max_kv, *[fake(0x1000)] * 4, 16, 64, 16, 0, 0.1, 1, 0, fake(0x9000), Hq * D, D, None]
    for ws, size, status in [(None, 0, bq.ERR_WORKSPACE), (fake(0x10000), n - 1, bq.ERR_WORKSPACE),
                             (fake(0x10004), n, bq.ERR_ALIGNMENT)]:
        assert L.bq_kv_attention(*args, ws, size, None) == status


def test_attention_refuses_a_page_table_that_is_not_there(L):                # noqa: F811
    """Also for a cache without pages: lengths are on the device, so the table is read."""
    p = ctypes.c_void_p
    for n_pages, arrays in ((0, None), (16, p(0x1000))):
        args = [p(0x1000), 512, 128, p(0x1000), p(0x1000), None, 8, 8, 2, 4, 4, 2, 128, 2, 512, *[arrays] * 4,
                n_pages, 64, 16, 0, 0.1, 1, 0, p(0x9000), 512, 128, None, p(0x10000), 1 << 40, None]
        assert L.bq_kv_attention(*args) == bq.ERR_INVALID_ARG


def test_attention_refuses_sizes_that_its_kernels_cannot_number(L):          # noqa: F811
    """Rows of a key head are numbered in 32 bits, and a workspace's size must not wrap round."""
    n = ctypes.c_size_t(0)

    def size(B, T, Hq, Hkv, D, max_q, max_kv):
        return L.bq_kv_attention_workspace_size(B, T, Hq, Hkv, D, max_q, max_kv, 64, 16, ctypes.byref(n))
    assert size(1, 1 << 28, 8, 1, 64, 1 << 28, 128) == bq.ERR_UNSUPPORTED
    assert size(1, 1 << 28, 8, 1, 64, 1 << 27, 128) == bq.OK
    assert size(1, 4, 8, 1, 64, (1 << 31) - 1, 128) == bq.OK         # a bound far above the call's rows
    assert size(1, (1 << 31) - 2, 65535, 65535 // 3, 255, 1, (1 << 31) - 1) == bq.ERR_UNSUPPORTED
    p = ctypes.c_void_p
    args = [p(0x1000), 512, 64, p(0x1000), p(0x1000), p(0x1000), 8, 8, 1, 1 << 28, 8, 1, 64, 1 << 28, 512,
            *[p(0x1000)] * 4, 16, 64, 16, 0, 0.1, 1, 0, p(0x9000), 512, 64, None, p(0x10000), 1 << 62, None]
    assert L.bq_kv_attention(*args) == bq.ERR_UNSUPPORTED


@gpu
@pytest.mark.parametrize("D", [128, 64, 40])
def test_attention_with_a_row_bound_far_above_the_rows(L, D):                # noqa: F811
    g = gen(D)
    off, ln, table, count = make_batch(g, [3], [300], 32)
    c = random_cache(g, count, 1, 32, D, 16, bq.INT8)
    q = randn(g, 3, 8, D).bfloat16()
    want, _, tol, _ = ref.attention(q, c.k, c.v, c.ks, c.vs, off, ln, table, bq.INT8)
    got = bq.kv_attention(q, c, off, ln, table, 2 ** 31 - 1, 300)
    bq.check_device_status()
    assert ((got.double() - want).abs() <= tol).all()


@gpu
@pytest.mark.parametrize("dtype", [bq.INT8, bq.FP8_E4M3])
@pytest.mark.parametrize("M,K,group", [(300, 4096, 128), (64, 2048, 2048), (40, 14336, 64), (20, 1000, 8)])
def test_norm_codes_are_those_of_exact_quotients(L, M, K, group, dtype):     # noqa: F811
    """code = t Q / max |t| to nearest, ties to even, with t = r w: a product of two bf16 is
    exact in fp32, a quotient that is no tie lies farther from one than fp32's half step
    (both have 16 bits: at least 2^-20 of itself), and a tie is exact in 64 bits."""
    g = gen(M + K + group)
    x = (randn(g, M, K) * torch.exp2(torch.arange(M, device="cuda") % 9 - 4.0)[:, None]).bfloat16()
    w = (1 + 0.2 * randn(g, K)).bfloat16()
    x[:, ::3] = (x[:, ::3].float() * 4).round().bfloat16()       # many quotients in the middle of two codes
    t = x.to(F8) * w.to(F8)
    amax = t.view(M, -1, group).abs().amax(2, keepdim=True)
    n = torch.where(amax > 0, t.view(M, -1, group) * ref.QMAX[dtype] / torch.where(amax > 0, amax, 1.0), 0.0)
    if dtype == bq.INT8:
        assert ((n - n.floor()) == 0.5).sum() > 10
        want = n.round().to(torch.int8).view(torch.uint8)
    else:
        want = n.float().to(ref.FP8).view(torch.uint8)
    want = want.view(M, K)
    for view in (x, shifted(x)):
        q, _ = bq.rmsnorm_quant(view, w, group_k=group, dtype=dtype)
        assert torch.equal(q, want), f"{int((q != want).sum())} of {q.numel()} codes"
