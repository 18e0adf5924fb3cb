"""The operators between two linears -- norm with an 8-bit output, rotary
positions, the paged 8-bit cache and its attention -- against plain 64-bit
implementations, and their refusals."""
import ctypes
import math

import pytest
import torch

import block_scaled_w8a8_b200 as bq
import layer_ref as ref

gpu = pytest.mark.gpu
P = ctypes.c_void_p
FAKE = P(0x1000)


@pytest.fixture(scope="module")
def L():
    from block_scaled_w8a8_b200 import build
    build.build()
    return bq.lib()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


# ---- refusals (host) --------------------------------------------------------------

def norm_args(**kw):
    a = dict(x=FAKE, ldx=256, res=None, ldr=0, w=FAKE, off=0.0, eps=1e-6, M=4, K=256, group=128,
             dtype=0, q=FAKE, ldq=256, s=FAKE, ro=None, ldro=0, h=None, ldh=0, st=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw, status", [
    (dict(dtype=2), bq.ERR_INVALID_ARG), (dict(group=0), bq.ERR_INVALID_ARG),
    (dict(M=-1), bq.ERR_INVALID_ARG), (dict(ldx=255), bq.ERR_INVALID_ARG),
    (dict(ldq=255), bq.ERR_INVALID_ARG), (dict(res=FAKE, ldr=255), bq.ERR_INVALID_ARG),
    (dict(ro=FAKE, ldro=255), bq.ERR_INVALID_ARG), (dict(h=FAKE, ldh=0), bq.ERR_INVALID_ARG),
    (dict(eps=-1.0), bq.ERR_INVALID_ARG), (dict(eps=math.nan), bq.ERR_INVALID_ARG),
    (dict(off=math.inf), bq.ERR_INVALID_ARG), (dict(w=None), bq.ERR_INVALID_ARG),
    (dict(s=None), bq.ERR_INVALID_ARG), (dict(q=None), bq.ERR_INVALID_ARG),
    (dict(ro=FAKE, ldro=300), bq.ERR_INVALID_ARG),                       # x in place, other stride
    (dict(K=98305, ldx=98305, ldq=98305), bq.ERR_UNSUPPORTED),
    (dict(M=0, x=None, w=None, q=None, s=None), bq.OK),
    (dict(K=0, x=None, w=None, q=None, s=None), bq.OK)])
def test_norm_refusals(L, kw, status):
    assert L.bq_rmsnorm_quant(*norm_args(**kw)) == status


def test_mx_norm_refusals(L):
    a = [FAKE, 256, None, 0, FAKE, 0.0, 1e-6, 4, 256, FAKE, 256, FAKE, None, 0, None, 0, None]
    for i, v, status in [(8, 200, bq.ERR_UNSUPPORTED), (10, 255, bq.ERR_INVALID_ARG),
                         (10, 257, bq.ERR_ALIGNMENT), (11, None, bq.ERR_INVALID_ARG),
                         (4, None, bq.ERR_INVALID_ARG), (7, 0, bq.OK)]:
        b = list(a)
        b[i] = v
        assert L.bq_mx_rmsnorm_quant(*b) == status, (i, v)


def test_rope_refusals(L):
    def call(**kw):
        a = dict(x=FAKE, ldt=256, ldh=128, pos=FAKE, turns=FAKE, T=4, H=2, D=128, rot=128,
                 layout=0, ms=1.0, out=P(0x9000), ldot=256, ldoh=128, st=None)
        a.update(kw)
        return L.bq_rope(*a.values())
    for kw in [dict(layout=2), dict(T=-1), dict(D=0), dict(rot=3), dict(rot=130), dict(rot=-2),
               dict(ldt=-1), dict(ldot=200), dict(ldoh=64), dict(x=None), dict(out=None),
               dict(pos=None), dict(turns=None), dict(out=FAKE, ldot=512)]:
        assert call(**kw) == bq.ERR_INVALID_ARG, kw
    assert call(T=0, x=None, out=None, pos=None, turns=None) == bq.OK
    assert call(H=0, x=None, out=None, pos=None, turns=None) == bq.OK


def test_rope_frequencies(L):
    def turns(*a, **k):
        return bq.rope_frequencies(*a, device="cpu", **k)
    t, ms = turns(8, 10000.0)
    want = torch.tensor([10000.0 ** (-2 * i / 8) / (2 * math.pi) for i in range(4)],
                        dtype=torch.float64)
    assert ms == 1.0 and torch.allclose(t, want, rtol=1e-14, atol=0)
    t2, ms = turns(8, 10000.0, bq.ROPE_LINEAR, 4.0)
    assert ms == 1.0 and torch.allclose(t2, want / 4, rtol=1e-14, atol=0)
    # NTK: the last frequency is that of linear interpolation, the first is kept
    t3, ms = turns(8, 10000.0, bq.ROPE_NTK, 4.0)
    assert ms == 1.0 and abs(t3[3] / (want[3] / 4) - 1) < 1e-12 and abs(t3[0] / want[0] - 1) < 1e-14
    # YaRN: fast turns are kept, slow ones interpolated, those between mixed
    t4, ms = turns(128, 10000.0, bq.ROPE_YARN, 8.0, 4096, 32.0, 1.0)
    full = turns(128, 10000.0)[0]
    r = 4096 * full
    assert abs(ms - (1 + 0.1 * math.log(8.0))) < 1e-6
    assert torch.equal(t4[r >= 32], full[r >= 32])
    assert torch.allclose(t4[r <= 1], full[r <= 1] / 8, rtol=1e-14, atol=0)
    mid = (r > 1) & (r < 32)
    g = (r[mid] - 1) / 31
    assert mid.any()
    assert torch.allclose(t4[mid], (1 - g) * full[mid] / 8 + g * full[mid], rtol=1e-13, atol=0)
    for a in [(0,), (7,), (8, 1.0), (8, math.nan), (8, 1e4, 4), (8, 1e4, bq.ROPE_LINEAR, 0.5),
              (2, 1e4, bq.ROPE_NTK, 2.0), (8, 1e4, bq.ROPE_YARN, 2.0, 0),
              (8, 1e4, bq.ROPE_YARN, 2.0, 64, 1.0, 1.0)]:
        with pytest.raises(bq.BqError) as e:
            turns(*a)
        assert e.value.status == bq.ERR_INVALID_ARG


def append_args(**kw):
    a = dict(k=FAKE, ldk=256, hk=128, v=FAKE, ldv=256, hv=128, off=FAKE, lens=FAKE, table=FAKE,
             ld=8, cols=8, B=2, T=4, H=2, D=128, P=16, page=64, bt=16, dtype=0, kc=FAKE, vc=FAKE,
             ks=FAKE, vs=FAKE, st=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw, status", [
    (dict(dtype=3), bq.ERR_INVALID_ARG), (dict(B=-1), bq.ERR_INVALID_ARG),
    (dict(H=0), bq.ERR_INVALID_ARG), (dict(D=0), bq.ERR_INVALID_ARG),
    (dict(page=0), bq.ERR_INVALID_ARG), (dict(bt=0), bq.ERR_INVALID_ARG),
    (dict(bt=24), bq.ERR_INVALID_ARG), (dict(ld=7), bq.ERR_INVALID_ARG),
    (dict(ldk=-1), bq.ERR_INVALID_ARG), (dict(k=None), bq.ERR_INVALID_ARG),
    (dict(vs=None), bq.ERR_INVALID_ARG), (dict(table=None), bq.ERR_INVALID_ARG),
    (dict(H=70000), bq.ERR_UNSUPPORTED), (dict(T=1 << 31), bq.ERR_UNSUPPORTED),
    (dict(P=1 << 32), bq.ERR_UNSUPPORTED), (dict(cols=1 << 26, ld=1 << 26), bq.ERR_UNSUPPORTED),
    (dict(cols=(1 << 24) + 1, ld=1 << 25), bq.ERR_UNSUPPORTED),
    (dict(T=0, k=None), bq.OK), (dict(B=0, off=None), bq.OK)])
def test_append_refusals(L, kw, status):
    assert L.bq_kv_append(*append_args(**kw)) == status


def attn_args(**kw):
    a = dict(q=FAKE, ldq=512, hq=128, off=FAKE, lens=FAKE, table=FAKE, ld=8, cols=8, B=2, T=4,
             Hq=4, H=2, D=128, mq=2, ml=512, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, P=16, page=64,
             bt=16, dtype=0, scale=0.1, causal=1, window=0, out=P(0x9000), ldo=512, ho=128,
             lse=None, ws=P(0x10000), wsb=1 << 40, st=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw, status", [
    (dict(dtype=-1), bq.ERR_INVALID_ARG), (dict(Hq=3), bq.ERR_INVALID_ARG),
    (dict(Hq=1), bq.ERR_INVALID_ARG), (dict(mq=-1), bq.ERR_INVALID_ARG),
    (dict(D=257), bq.ERR_UNSUPPORTED), (dict(scale=math.nan), bq.ERR_INVALID_ARG),
    (dict(window=-1), bq.ERR_INVALID_ARG), (dict(window=4, causal=0), bq.ERR_INVALID_ARG),
    (dict(ldo=100), bq.ERR_INVALID_ARG), (dict(ho=64), bq.ERR_INVALID_ARG),
    (dict(ldo=256, ho=128), bq.ERR_INVALID_ARG), (dict(q=None), bq.ERR_INVALID_ARG),
    (dict(out=None), bq.ERR_INVALID_ARG), (dict(kc=None), bq.ERR_INVALID_ARG),
    (dict(bt=5), bq.ERR_INVALID_ARG), (dict(T=0, q=None, out=None), bq.OK),
    (dict(B=0, off=None), bq.OK)])
def test_attention_refusals(L, kw, status):
    assert L.bq_kv_attention(*attn_args(**kw)) == status


def test_attention_workspace_is_checked(L):
    n = bq.kv_attention_workspace_size(1, 1, 32, 8, 128, 1, 1 << 17, 64, 16)
    if n:
        a = attn_args(B=1, T=1, Hq=32, H=8, ldq=4096, ldo=4096, ml=1 << 17, cols=2048, ld=2048,
                      mq=1)
        for ws, size, status in [(None, 0, bq.ERR_WORKSPACE), (P(0x10000), n - 1, bq.ERR_WORKSPACE),
                                 (P(0x10004), n, bq.ERR_ALIGNMENT)]:
            a[-3], a[-2] = ws, size
            assert L.bq_kv_attention(*a) == status
    assert L.bq_kv_attention_workspace_size(1, 1, 4, 2, 128, 1, 64, 64, 24, None) == \
        bq.ERR_INVALID_ARG


def test_binding_refuses_host_tensors_and_wrong_shapes(L):
    x = torch.zeros(2, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bq.rmsnorm_quant(x, torch.zeros(8, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        bq.rope(x.view(2, 1, 8), torch.zeros(2, dtype=torch.int32), torch.zeros(4).double())
    with pytest.raises(ValueError):
        bq.kv_cache(2, 1, 16, 8, block_t=5, device="cpu")


@gpu
def test_binding_refuses_wrong_device_arrays(L):
    x = torch.zeros(2, 8, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(8, dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    for bad in [lambda: bq.rmsnorm_quant(x, w[:7]), lambda: bq.rmsnorm_quant(x.float(), w),
                lambda: bq.rmsnorm_quant(x, w, residual=x[:1]),
                lambda: bq.rmsnorm_quant(x.t(), w[:2]),
                lambda: bq.rmsnorm_quant(x, w, residual=x.cpu()),
                lambda: bq.rmsnorm_quant(x, w, s=torch.zeros(1, 3, device="cuda")),
                lambda: bq.rmsnorm_quant(x[:1].expand(2, 8), w),
                lambda: bq.mx_rmsnorm_quant(torch.zeros(2, 128, dtype=torch.bfloat16,
                                                        device="cuda"),
                                            torch.zeros(128, dtype=torch.bfloat16, device="cuda"),
                                            sf=torch.zeros(8, dtype=torch.uint8, device="cuda")),
                lambda: bq.rope(x.view(2, 1, 8), torch.zeros(3, **i32),
                                torch.zeros(4, dtype=torch.float64, device="cuda")),
                lambda: bq.rope(x.view(2, 1, 8), torch.zeros(2, **i32),
                                torch.zeros(4, device="cuda"))]:
        with pytest.raises(ValueError):
            bad()
    c = bq.kv_cache(2, 1, 16, 8, block_t=4)
    off, lens, tab = torch.zeros(2, **i32), torch.zeros(1, **i32), torch.zeros(1, 2, **i32)
    k = x.view(2, 1, 8)
    for bad in [lambda: bq.kv_append(c, k, k[:1], off, lens, tab),
                lambda: bq.kv_append(c, k.expand(2, 2, 8), k, off, lens, tab),
                lambda: bq.kv_append(c, k, k, off[:1], lens, tab),
                lambda: bq.kv_append(c, k, k, off, lens, tab[0]),
                lambda: bq.kv_append(c, k, k, off.long(), lens, tab),
                lambda: bq.kv_append(c._replace(k=c.k[:, :, :8]), k, k, off, lens, tab),
                lambda: bq.kv_append(c._replace(vs=c.vs[:, :, :2]), k, k, off, lens, tab),
                lambda: bq.kv_attention(k.float(), c, off, lens, tab, 1, 1),
                lambda: bq.kv_attention(k, c, off, lens, tab, 1, 1,
                                        out=torch.zeros(2, 1, 4, dtype=torch.bfloat16,
                                                        device="cuda")),
                lambda: bq.kv_attention(k, c, off, lens, tab, 1, 1,
                                        lse=torch.zeros(1, 2, device="cuda"))]:
        with pytest.raises(ValueError):
            bad()


# ---- norm ---------------------------------------------------------------------------

NORM = [(1, 1, 128), (3, 7, 4), (2, 33, 5), (5, 128, 128), (4, 200, 128), (7, 256, 256),
        (3, 256, 8), (130, 384, 128), (2, 1000, 16), (9, 4096, 128), (300, 4096, 128),
        (3, 4096, 4096), (2, 4104, 8192), (5, 8200, 128), (2, 14336, 64), (2, 20480, 256),
        (2, 40000, 128), (1, 98304, 128), (1, 98301, 98301)]


@gpu
@pytest.mark.parametrize("dtype", [bq.INT8, bq.FP8_E4M3])
@pytest.mark.parametrize("M,K,group", NORM)
def test_norm_against_64_bits(L, M, K, group, dtype):
    g = gen(M * 1000 + K + group + dtype)
    x, res = randn(g, M, K).bfloat16(), (3 * randn(g, M, K)).bfloat16()
    x[M // 2].zero_()
    w = (1 + 0.2 * randn(g, K)).bfloat16()
    r, y = ref.rmsnorm(x, w, 1e-5, res)
    q, s, ro, h = bq.rmsnorm_quant(x, w, 1e-5, res, group, dtype, want_h=True)
    assert torch.equal(ro, r)
    rel = ref.norm_rel(K)
    ref.check_codes(q, s, y, group, dtype, rel)
    assert ((h.double() - y).abs() <= y.abs() * (ref.UBF16 + 2 * rel)).all()
    # no residual, weights kept as their difference from 1, nothing else asked for
    _, y = ref.rmsnorm(x, w, 1e-5, None, 1.0)
    q, s = bq.rmsnorm_quant(x, w, 1e-5, group_k=group, dtype=dtype, weight_offset=1.0)
    ref.check_codes(q, s, y, group, dtype, rel)


@gpu
@pytest.mark.parametrize("dtype", [bq.INT8, bq.FP8_E4M3])
@pytest.mark.parametrize("K,pad,first", [(512, 8, 0), (512, 3, 0), (512, 8, 1), (500, 12, 4)])
def test_norm_strides_alignment_and_in_place(L, K, pad, first, dtype):
    M, g = 6, gen(K + pad + first)
    def strided(t, fill):
        big = torch.full((M, K + pad + first), fill, dtype=t.dtype, device="cuda")
        v = big[:, first:first + K]
        v.copy_(t)
        return big, v
    x, res = randn(g, M, K).bfloat16(), randn(g, M, K).bfloat16()
    w = randn(g, K).bfloat16()
    r, y = ref.rmsnorm(x, w, 1e-6, res)
    xb, xv = strided(x, 5.0)
    rb, rv = strided(res, 5.0)
    qb, qv = strided(torch.zeros(M, K, dtype=torch.uint8, device="cuda"), 77)
    hb, hv = strided(torch.zeros_like(x), 5.0)
    q, s, ro, h = bq.rmsnorm_quant(xv, w, 1e-6, rv, 128, dtype, q=qv, res_out=rv, h=hv)
    assert ro is rv and torch.equal(rv, r) and torch.equal(xv, x)
    ref.check_codes(q.contiguous(), s, y, 128, dtype, ref.norm_rel(K))
    for big, fill in ((xb, 5.0), (rb, 5.0), (qb, 77), (hb, 5.0)):
        assert (big[:, :first] == fill).all() and (big[:, first + K:] == fill).all()
    # the sum in place of x
    x2 = x.clone()
    bq.rmsnorm_quant(x2, w, 1e-6, res, res_out=x2)
    assert torch.equal(x2, r)


@gpu
@pytest.mark.parametrize("M,K", [(1, 128), (5, 256), (127, 384), (130, 4096), (33, 14336),
                                 (2, 40064)])
def test_mx_norm_against_64_bits(L, M, K):
    import gpu_util
    g = gen(M + K)
    x, res = randn(g, M, K).bfloat16(), randn(g, M, K).bfloat16()
    res[:, 32:64], x[:, 32:64] = 0, 0
    w = (1 + 0.2 * randn(g, K)).bfloat16()
    r, y = ref.rmsnorm(x, w, 1e-6, res)
    q, sf, ro, h = bq.mx_rmsnorm_quant(x, w, 1e-6, res, want_h=True)
    assert torch.equal(ro, r)
    rel = ref.norm_rel(K)
    e = torch.from_numpy(gpu_util.mx_sf_rows(sf, M, K)).cuda().double()
    a = y.view(M, K // 32, 32)
    amax = a.abs().amax(2)
    low, high = (torch.floor(torch.log2(amax * f)) + 119 for f in (1 - 2 * rel, 1 + 2 * rel))
    zero = amax == 0
    assert (e[zero] == 0).all() and zero.any()
    assert ((e >= low) & (e <= high))[~zero].all()
    n = a / torch.exp2(e - 127)[..., None]
    n = n.clamp(-448, 448)
    c = ref.decode(q, 1).view(a.shape)
    tol = torch.maximum(n.abs() * 2.0 ** -4, torch.full_like(n, 2.0 ** -10)) + n.abs() * 2 * rel
    assert ((c - n).abs() <= tol).all()
    assert ((h.double() - y).abs() <= y.abs() * (ref.UBF16 + 2 * rel)).all()


@gpu
def test_norm_empty(L):
    w = torch.ones(16, dtype=torch.bfloat16, device="cuda")
    q, s = bq.rmsnorm_quant(torch.empty(0, 16, dtype=torch.bfloat16, device="cuda"), w)
    assert q.shape == (0, 16) and s.shape == (1, 0)


# ---- rotary positions ------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("layout", [bq.ROPE_HALF, bq.ROPE_INTERLEAVED])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 2, 2), (3, 2, 5, 4), (7, 3, 64, 64), (33, 5, 128, 64),
                                       (64, 40, 128, 128), (300, 8, 128, 32), (5, 2, 96, 24),
                                       (4, 3, 256, 256), (9, 2, 80, 0), (2000, 6, 64, 16)])
def test_rope_against_64_bits(L, T, H, D, rot, layout):
    g = gen(T + H + D + rot)
    wide = randn(g, T, H * D + 2 * D).bfloat16()
    pos = torch.randint(-1000, 2 ** 31 - 1, (T,), generator=g, device="cuda", dtype=torch.int32)
    pos[: T // 2] = torch.arange(T // 2, device="cuda", dtype=torch.int32)
    if rot:
        turns, ms = bq.rope_frequencies(rot, 500000.0, bq.ROPE_YARN, 8.0, 8192)
    else:
        turns, ms = torch.empty(0, dtype=torch.float64, device="cuda"), 1.0
    for x in (wide[:, D:D + H * D].view(T, H, D) if D % 2 == 0 else
              wide[:, :H * D].reshape(T, H, D),
              wide[:, 1:1 + H * D].unflatten(1, (H, D)),
              randn(g, H, T, D).bfloat16().transpose(0, 1)):
        want, mag = ref.rope(x, pos, turns, layout, ms)
        # u(bf16) of the result, and fp32 sine, cosine and angle (2 pi 2^-25) on |a| + |b|
        tol = want.abs() * ref.UBF16 + mag * 2.0 ** -20 + 2.0 ** -134
        before = wide.clone()
        got = bq.rope(x, pos, turns, layout, ms)
        assert torch.equal(wide, before)
        assert ((got.double() - want).abs() <= tol).all()
        assert torch.equal(got[..., rot:], x[..., rot:])
        y = x.clone()
        assert bq.rope(y, pos, turns, layout, ms, out=y) is y and torch.equal(y, got)
        # only the heads given are written
        part = torch.full((T, H + 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
        bq.rope(x, pos, turns, layout, ms, out=part[:, 1:1 + H])
        assert torch.equal(part[:, 1:1 + H], got)
        assert (part[:, 0] == 7).all() and (part[:, H + 1:] == 7).all()


@gpu
def test_rope_undone_by_the_negated_position(L):
    g = gen(3)
    x = randn(g, 50, 4, 64).bfloat16()
    pos = torch.randint(0, 10 ** 6, (50,), generator=g, device="cuda", dtype=torch.int32)
    turns, _ = bq.rope_frequencies(64)
    back = bq.rope(bq.rope(x, pos, turns), -pos, turns)
    mag = x.double().abs().amax(-1, keepdim=True)
    # two roundings to bf16 of values of at most sqrt(2) max |x|, the first turned again
    assert ((back.double() - x.double()).abs() <= 4 * ref.UBF16 * mag).all()


# ---- cache -------------------------------------------------------------------------------

def make_batch(g, new, lens, page, spare=2):
    """offsets, lens, a shuffled page table, and how many pages there are."""
    off = [0]
    for n in new:
        off.append(off[-1] + n)
    need = [-(-n // page) for n in lens]
    count = sum(need) + spare
    order = torch.randperm(count, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(need + [1]) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    i32 = dict(dtype=torch.int32, device="cuda")
    return torch.tensor(off, **i32), torch.tensor(lens, **i32), table, count


def random_cache(g, count, H, page, D, bt, dtype, garbage=False):
    """A cache of random codes; with `garbage`, every byte value in every slot."""
    c = bq.kv_cache(count, H, page, D, bt, dtype)
    for t in (c.k, c.v):
        x = randn(g, *t.shape) * (36 if dtype == 0 else 120)
        t.copy_(x.round().clamp(-127, 127).to(torch.int8).view(torch.uint8) if dtype == 0 else
                x.clamp(-448, 448).to(ref.FP8).view(torch.uint8))
        if garbage:
            t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    for t in (c.ks, c.vs):
        t.copy_((0.5 + torch.rand(t.shape, generator=g, device="cuda")) * 3 / ref.QMAX[dtype])
        if garbage:
            t.fill_(math.nan)
    return c


@gpu
@pytest.mark.parametrize("dtype", [bq.INT8, bq.FP8_E4M3])
@pytest.mark.parametrize("H,D,page,bt", [(1, 5, 6, 3), (2, 16, 8, 1), (3, 64, 16, 16),
                                         (2, 128, 64, 16), (1, 128, 128, 128), (2, 256, 32, 8),
                                         (8, 64, 64, 2), (1, 96, 256, 256), (1, 8, 512, 512)])
def test_append_bit_exact(L, H, D, page, bt, dtype):
    g = gen(H + D + page + bt)
    # (new, length after): a fresh block, a block continued, one that ends inside, none, many
    calls = [([3, 0, 1, 2 * page + 1, 0], [3, 0, 1, 2 * page + 1, 0]),
             ([1, 1, 1, 1, 1], [4, 1, 2, 2 * page + 2, 1]),
             ([page, 0, 2, 5, bt], [4 + page, 1, 4, 2 * page + 7, 1 + bt])]
    off, lens, table, count = make_batch(g, *calls[-1], page)
    c = random_cache(g, count, H, page, D, bt, dtype, garbage=True)
    for step, (new, ln) in enumerate(calls):
        T = sum(new)
        wide = (randn(g, T + 3, 2 * H * D + 6) * 2.0 ** step).bfloat16()
        k = wide[:, 3:3 + H * D].unflatten(1, (H, D))
        v = randn(g, H, T + 3, D).bfloat16().transpose(0, 1)
        k[0, 0].zero_()
        off, lens = (torch.tensor(t, dtype=torch.int32, device="cuda")
                     for t in ([sum(new[:i]) for i in range(len(new) + 1)], ln))
        want = [ref.append(*a, off, lens, table, dtype)
                for a in ((c.k, c.ks, k), (c.v, c.vs, v))]
        for again in range(2):                       # the second time changes nothing
            bq.kv_append(c, k, v, off, lens, table)
            for (codes, scales), got, gs in zip(want, (c.k, c.v), (c.ks, c.vs)):
                assert torch.equal(got, codes)
                assert torch.equal(gs.view(torch.int32), scales.view(torch.int32))
    bq.check_device_status()


@gpu
@pytest.mark.parametrize("dtype", [bq.INT8, bq.FP8_E4M3])
def test_append_codes_of_many_values_bit_exact(L, dtype):
    """The cache write forms its quotients without divisions: every bf16 value
    against scales of all magnitudes, and scales that lie next to a power of two."""
    g = gen(23 + dtype)
    H, D, page = 1, 128, 64
    every = torch.arange(0, 0x7F80, device="cuda", dtype=torch.int32).to(torch.int16)
    every = torch.cat([every, every | -0x8000]).view(torch.bfloat16)     # all finite values
    for step in range(40):
        e = 2.0 ** (step * 6 - 120)
        top = (every.abs().float() <= e).nonzero()[:, 0]
        # values near the block's largest, where codes are not all zero, in random order
        near = top[every[top].abs().float() > e * 2.0 ** -14]
        x = every[near[torch.randint(0, near.numel(), (64 * D * 4,), generator=g, device="cuda")]]
        x = x.view(256, H, D)
        i32 = dict(dtype=torch.int32, device="cuda")
        off, lens = torch.tensor([0, 256], **i32), torch.tensor([256], **i32)
        table = torch.arange(4, **i32).view(1, 4)
        c = bq.kv_cache(4, H, page, D, page, dtype)
        want = ref.append(c.k, c.ks, x, off, lens, table, dtype)
        bq.kv_append(c, x, x, off, lens, table)
        assert torch.equal(c.ks, want[1]) and torch.equal(c.k, want[0]), step
        assert torch.equal(c.v, c.k)


@gpu
def test_append_skips_and_records_what_it_cannot_use(L):
    g = gen(5)
    i32 = dict(dtype=torch.int32, device="cuda")
    k = randn(g, 4, 1, 16).bfloat16()
    for off, lens, table in [([0, 2, 4], [2, 3], [[0, 1], [9, 9]]), ([0, 2, 4], [2, 3], [[0, 1], [-1, 0]]),
                             ([0, 2, 4], [2, 1], [[0, 1], [2, 3]]), ([0, 2, 4], [2, 99], [[0, 1], [2, 3]]),
                             ([0, 2, 9], [2, 7], [[0, 1], [2, 3]]), ([0, 2, 1], [2, 3], [[0, 1], [2, 3]])]:
        c = random_cache(g, 4, 1, 4, 16, 2, bq.INT8)
        before = c.k.clone()
        bq.kv_append(c, k, k, torch.tensor(off, **i32), torch.tensor(lens, **i32),
                     torch.tensor(table, **i32))
        with pytest.raises(bq.BqError) as e:
            bq.check_device_status()
        assert e.value.status == bq.ERR_INVALID_ARG
        assert torch.equal(c.k[1:], before[1:])          # only sequence 0's page is written
        assert torch.equal(c.k[0, 0, :2], ref.append(before, c.ks.clone(), k,
                           torch.tensor([0, 2]), torch.tensor([2]), torch.tensor([[0]]), 0)[0][0, 0, :2])
    bq.check_device_status()


# ---- attention ------------------------------------------------------------------------------

def check_attention(g, new, lens, Hq, Hk, D, page, bt, dtype, scale=None, causal=True, window=0,
                    tail=3, sharp=1.0, max_q=None, max_kv=None, ws=None):
    off, ln, table, count = make_batch(g, new, lens, page)
    c = random_cache(g, count, Hk, page, D, bt, dtype)
    # whatever stands behind the last token, and in pages of nobody, is not looked at
    junk = random_cache(g, count, Hk, page, D, bt, dtype, garbage=True)
    live = torch.zeros(count, page, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        for p in range(-(-n // page)):
            live[int(table[b, p]), : min(page, n - p * page)] = True
    for a, z in ((c.k, junk.k), (c.v, junk.v)):
        a.copy_(torch.where(live[:, None, :, None], a, z))
    blk = live.view(count, page // bt, bt).any(2)
    for a, z in ((c.ks, junk.ks), (c.vs, junk.vs)):
        a.copy_(torch.where(blk[:, None], a, z))
    T = sum(new) + tail
    q = (sharp * randn(g, T, Hq * D + 8)).bfloat16()[:, :Hq * D].unflatten(1, (Hq, D))
    want, lse_w, tol, ltol = ref.attention(q, c.k, c.v, c.ks, c.vs, off, ln, table, dtype, scale, causal,
                                     window)
    out = torch.full((T, Hq, D + 2), 7.0, dtype=torch.bfloat16, device="cuda")[..., :D]
    lse = torch.full((T, Hq), 7.0, device="cuda")
    bq.kv_attention(q, c, off, ln, table, max(new + [0]) if max_q is None else max_q,
                    max(lens + [0]) if max_kv is None else max_kv, scale, causal, window, out, lse,
                    ws)
    bq.check_device_status()
    n = sum(new)
    assert (out[n:] == 7).all() and (lse[n:] == 7).all()
    d = (out[:n].double() - want[:n]).abs()
    assert torch.isfinite(out[:n]).all()
    worst = (d - tol[:n]).max().item() if n else 0.0
    assert (d <= tol[:n]).all(), f"{int((d > tol[:n]).sum())} of {d.numel()} off, by up to {worst}"
    empty = torch.isinf(lse_w[:n])
    assert (out[:n][empty] == 0).all() and (lse[:n][empty] == -math.inf).all()
    dl = (lse[:n].double() - lse_w[:n])[~empty].abs()
    assert (dl <= ltol[:n][~empty]).all()
    return out, lse


ATTN = [  # new, lens, Hq, Hk, D, page, bt, causal, window
    ([1], [1], 1, 1, 64, 16, 16, True, 0),
    ([1], [7], 2, 1, 5, 4, 2, True, 0),
    ([1, 1, 1], [3, 0, 40], 4, 2, 128, 16, 8, True, 0),           # a row with no key at all
    ([1, 1], [200, 1000], 32, 8, 128, 64, 16, True, 0),
    ([1, 1], [129, 4097], 8, 8, 64, 32, 32, True, 0),
    ([1, 1, 1], [300, 31, 64], 8, 1, 128, 64, 1, True, 0),
    ([1, 1], [515, 77], 16, 1, 64, 128, 64, True, 100),
    ([1], [260], 20, 1, 128, 16, 4, True, 0),                      # more than 16 rows
    ([2, 4, 0, 3], [66, 4, 12, 700], 8, 2, 128, 64, 64, True, 0),
    ([1, 2], [100, 90], 4, 4, 256, 16, 16, True, 0),
    ([1, 5], [100, 90], 6, 2, 96, 16, 16, True, 33),
    ([4, 4], [2, 4], 4, 2, 64, 16, 16, True, 0),                   # rows before the first key
    ([5, 9], [70, 33], 8, 2, 128, 32, 8, False, 0),                # every key for every row
    ([64], [64], 4, 1, 128, 64, 64, True, 0),
    ([130, 1, 200], [130, 65, 333], 4, 2, 128, 64, 16, True, 0),
    ([257], [1000], 8, 4, 128, 16, 16, True, 0),
    ([300, 77], [300, 500], 5, 1, 64, 32, 16, True, 0),
    ([513, 100], [900, 100], 8, 2, 128, 64, 32, True, 128),
    ([150, 40], [400, 41], 4, 2, 64, 64, 64, True, 1),             # a window of itself
    ([190], [450], 6, 2, 128, 128, 1, False, 0),
    ([140, 20], [140, 300], 4, 4, 256, 32, 32, True, 64),
    ([1, 2], [3000, 900], 6, 2, 96, 24, 8, True, 0),               # split keys, any size of head
    ([3, 1], [130, 2500], 5, 1, 33, 10, 5, True, 1000),
    ([2], [4000], 4, 4, 128, 8, 4, True, 0),                       # pages that end inside a tile
    ([60, 9], [30, 9], 4, 1, 256, 16, 16, True, 2 ** 31 - 1),      # rows before the first key
    ([6, 9], [3, 9], 2, 1, 64, 16, 16, True, 2 ** 31 - 1),
    ([200, 9], [130, 9], 4, 2, 128, 64, 16, True, 2 ** 31 - 1),
    ([1, 2], [6000, 300], 4, 2, 128, 64, 16, True, 2000),          # a window of split keys
    ([3], [5001], 2, 2, 64, 32, 32, True, 1),
    ([300, 40], [5000, 1000], 4, 2, 128, 64, 16, True, 1500),
    ([2], [3001], 2, 1, 80, 16, 8, True, 1200),
]


@gpu
@pytest.mark.parametrize("dtype", [bq.INT8, bq.FP8_E4M3])
@pytest.mark.parametrize("case", ATTN, ids=lambda c: "n%s-l%s-h%d.%d-d%d-p%d.%d-%s-w%d" % (
    "+".join(map(str, c[0])), "+".join(map(str, c[1])), *c[2:]))
def test_attention_against_64_bits(L, case, dtype):
    new, lens, Hq, Hk, D, page, bt, causal, window = case
    check_attention(gen(sum(lens) + D), new, lens, Hq, Hk, D, page, bt, dtype, causal=causal,
                    window=window)


@gpu
@pytest.mark.parametrize("dtype", [bq.INT8, bq.FP8_E4M3])
@pytest.mark.parametrize("new,lens,Hq,Hk,D", [([1, 1], [700, 65], 8, 2, 128),
                                              ([200, 9], [300, 64], 8, 2, 128)])
def test_attention_scales_and_bounds(L, new, lens, Hq, Hk, D, dtype):
    # sharp and flat scores, a negative scale, bounds far above the lengths
    for i, (scale, sharp) in enumerate([(None, 12.0), (0.0, 1.0), (-0.05, 1.0), (1e-3, 300.0)]):
        check_attention(gen(i), new, lens, Hq, Hk, D, 64, 16, dtype, scale=scale, sharp=sharp,
                        max_q=1000, max_kv=9000)


@gpu
@pytest.mark.parametrize("new,lens", [([1, 1], [50, 20]), ([150, 1], [160, 20])])
def test_attention_skips_and_records_what_it_cannot_use(L, new, lens):
    g = gen(9)
    off, ln, table, count = make_batch(g, new, lens, 16)
    c = random_cache(g, count, 2, 16, 128, 16, bq.INT8)
    T = sum(new)
    q = randn(g, T, 4, 128).bfloat16()
    good = bq.kv_attention(q, c, off, ln, table, max(new), max(lens))
    bq.check_device_status()
    seq0 = slice(0, new[0])

    def call(o=off, n=ln, t=table, mq=max(new), ml=max(lens)):
        out = torch.full_like(q, 7.0)
        bq.kv_attention(q, c, o, n, t, mq, ml, out=out)
        with pytest.raises(bq.BqError) as e:
            bq.check_device_status()
        assert e.value.status == bq.ERR_INVALID_ARG
        return out

    for out in (call(n=torch.tensor([lens[0], 10 ** 6], dtype=torch.int32, device="cuda")),
                call(o=torch.tensor([0, new[0], 10 ** 6], dtype=torch.int32, device="cuda")),
                call(n=torch.tensor([lens[0], -3], dtype=torch.int32, device="cuda"))):
        assert torch.equal(out[seq0], good[seq0]) and (out[new[0]:] == 7).all()
    out = call(ml=max(lens) - 1)                      # sequence 0 is longer than promised
    assert (out[seq0] == 7).all() and torch.equal(out[new[0]:], good[new[0]:])
    # a page outside the cache: its keys are left out
    bad = table.clone()
    bad[1, 0] = count
    out = call(t=bad)
    assert torch.equal(out[seq0], good[seq0]) and torch.isfinite(out).all()
    bq.check_device_status()


@gpu
def test_attention_on_a_side_stream_and_in_a_graph(L):
    """Captured once, replayed with other lengths, offsets and queries; two
    graphs whose workspaces live side by side."""
    g = gen(11)
    page, Hk, D = 32, 2, 128
    for Hq, new, lens in ((8, [1, 1, 1], [900, 33, 400]), (8, [90, 1, 40], [900, 33, 400])):
        off, ln, table, count = make_batch(g, new, lens, page)
        c = random_cache(g, count, Hk, page, D, 16, bq.FP8_E4M3)
        q = randn(g, sum(new), Hq, D).bfloat16()
        want = bq.kv_attention(q, c, off, ln, table, max(new), 1000)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = bq.kv_attention(q, c, off, ln, table, max(new), 1000)
        side.synchronize()
        assert torch.equal(got, want)
        graphs = []
        for _ in range(2):
            out = torch.zeros_like(q)
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                bq.kv_attention(q, c, off, ln, table, max(new), 1000, out=out)
            graphs.append((gr, out))
        for lens2 in (lens, [len_ - 5 for len_ in lens]):
            ln.copy_(torch.tensor(lens2, dtype=torch.int32))
            q.copy_(randn(g, *q.shape).bfloat16())
            want = bq.kv_attention(q, c, off, ln, table, max(new), 1000)
            for gr, out in graphs:
                gr.replay()
            for gr, out in graphs:
                assert torch.equal(out, want)


@gpu
@pytest.mark.parametrize("new,Hq,Hk,D,page,bt", [
    ([1, 3], 4, 2, 128, 16, 16), ([1, 1], 8, 2, 64, 32, 32), ([2, 1], 4, 2, 96, 24, 8),
    ([90, 40], 4, 2, 128, 16, 16), ([70, 140], 2, 1, 64, 64, 64)])
def test_attention_behind_a_window_needs_no_pages(L, new, Hq, Hk, D, page, bt):
    """Pages that no row sees any more may be gone, and their scales NaN."""
    g = gen(D + page)
    lens, window = [1000, 530], 70
    off, ln, table, count = make_batch(g, new, lens, page)
    c = random_cache(g, count, Hk, page, D, bt, bq.INT8)
    q = randn(g, sum(new), Hq, D).bfloat16()
    want = bq.kv_attention(q, c, off, ln, table, max(new), 1000, window=window)
    lse = torch.zeros(sum(new), Hq, device="cuda")
    for b, (n, len_) in enumerate(zip(new, lens)):
        gone = max(0, len_ - n - window + 1) // page
        for t in (c.ks, c.vs):
            t[table[b, :gone].long()] = math.nan
        table[b, :gone] = -1
    got = bq.kv_attention(q, c, off, ln, table, max(new), 1000, window=window, lse=lse)
    bq.check_device_status()
    assert torch.equal(got, want) and torch.isfinite(lse).all()


@gpu
@pytest.mark.parametrize("new,Hq,Hk,D", [([1, 2], 8, 4, 128), ([80, 1], 8, 4, 128),
                                         ([1, 2], 8, 4, 96), ([40, 1], 4, 2, 64)])
def test_attention_takes_codes_at_any_address(L, new, Hq, Hk, D):
    g = gen(3 * D)
    off, ln, table, count = make_batch(g, new, [700, 65], 32)
    c = random_cache(g, count, Hk, 32, D, 16, bq.FP8_E4M3)
    q = randn(g, sum(new), Hq, D).bfloat16()
    want, _, tol, _ = ref.attention(q, c.k, c.v, c.ks, c.vs, off, ln, table, bq.FP8_E4M3)
    for shift in (1, 4, 8):
        k, v = (torch.empty(t.numel() + 16, dtype=torch.uint8, device="cuda")[shift:shift + t.numel()]
                .view(t.shape).copy_(t) for t in (c.k, c.v))
        got = bq.kv_attention(q, c._replace(k=k, v=v), off, ln, table, max(new), 700)
        assert ((got.double() - want).abs() <= tol).all()
    bq.check_device_status()


@gpu
@pytest.mark.parametrize("D,new", [(128, 1), (128, 90), (96, 1)])
def test_cache_past_32_bits(L, D, new):
    """Pages whose codes lie more than 2^32 bytes into the arrays."""
    g = gen(D)
    Hk, page, bt = 8, 64, 16
    count = (1 << 32) // (Hk * page * D) + 40
    small = bq.kv_cache(12, Hk, page, D, bt, bq.INT8)
    big = bq.kv_cache(count, Hk, page, D, bt, bq.INT8)
    i32 = dict(dtype=torch.int32, device="cuda")
    lens = [300, new + 3]
    near = torch.randperm(12, generator=g, device="cuda").to(torch.int32)[:12].view(2, 6)
    far = near + (count - 12)
    old = torch.tensor([n - new for n in lens])
    for upto, n in ((old, old.tolist()), (torch.tensor(lens), [new, new])):
        off = torch.tensor([0, n[0], sum(n)], **i32)
        ln = upto.to(**i32)
        k, v = (randn(g, sum(n), Hk, D).bfloat16() for _ in range(2))
        bq.kv_append(small, k, v, off, ln, near)
        bq.kv_append(big, k, v, off, ln, far)
    for a, b in zip(small[:4], big[:4]):
        assert torch.equal(a, b[count - 12:]) and int((b[:count - 12] != 0).sum()) == 0
    q = randn(g, 2 * new, 2 * Hk, D).bfloat16()
    assert torch.equal(bq.kv_attention(q, small, off, ln, near, new, 400),
                       bq.kv_attention(q, big, off, ln, far, new, 400))
    bq.check_device_status()


@gpu
def test_a_batch_of_many_sequences(L):
    """More sequences than a warp counts side by side, some of them with nothing new."""
    g = gen(23)
    B, H, D, page, bt = 1500, 1, 64, 16, 8
    new = [(i * 7) % 3 for i in range(B)]
    lens = [n + (i * 5) % 29 for i, n in enumerate(new)]
    off, ln, table, count = make_batch(g, new, lens, page)
    c = random_cache(g, count, H, page, D, bt, bq.INT8)
    k, v = (randn(g, sum(new) + 2, H, D).bfloat16() for _ in range(2))
    want = [ref.append(a, s, t, off, ln, table, bq.INT8) for a, s, t in ((c.k, c.ks, k), (c.v, c.vs, v))]
    bq.kv_append(c, k, v, off, ln, table)
    assert torch.equal(c.k, want[0][0]) and torch.equal(c.v, want[1][0])
    assert torch.equal(c.ks, want[0][1]) and torch.equal(c.vs, want[1][1])
    q = randn(g, sum(new), 2, D).bfloat16()
    out = bq.kv_attention(q, c, off, ln, table, 2, 40)
    want, _, tol, _ = ref.attention(q, c.k, c.v, c.ks, c.vs, off, ln, table, bq.INT8)
    assert ((out.double() - want).abs() <= tol).all()
    bq.check_device_status()


@gpu
def test_norm_rope_and_append_in_a_graph(L):
    """Captured once, replayed with other inputs, against the same calls made eagerly."""
    g = gen(29)
    H, D, T = 2, 128, 9
    x, res = randn(g, T, 512).bfloat16(), randn(g, T, 512).bfloat16()
    w = (1 + 0.1 * randn(g, 512)).bfloat16()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    turns, ms = bq.rope_frequencies(D)
    off, ln, table, count = make_batch(g, [4, 5], [30, 20], 16)
    start = random_cache(g, count, H, 16, D, 8, bq.FP8_E4M3)
    c = bq.kv_cache(count, H, 16, D, 8, bq.FP8_E4M3)
    k, v = (randn(g, T, H, D).bfloat16() for _ in range(2))

    def step(out):
        q8, s, r = bq.rmsnorm_quant(x, w, residual=res, dtype=bq.FP8_E4M3)
        m8, m = bq.mx_rmsnorm_quant(x, w)[:2]
        bq.rope(k, pos, turns, mscale=ms, out=out)
        bq.kv_append(c, out, v, off, ln, table)
        return q8, s, r, m8, m

    turned = torch.empty_like(k)
    step(turned)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step(turned)
    for i in range(2):
        for t in (x, res, k, v):
            t.copy_(randn(g, *t.shape).bfloat16())
        pos.add_(100 * i)
        ln.sub_(i)
        for a, b in zip(c[:4], start[:4]):
            a.copy_(b)
        graph.replay()
        got = [t.clone() for t in (*kept, turned, *c[:4])]
        for a, b in zip(c[:4], start[:4]):
            a.copy_(b)
        eager = torch.empty_like(k)
        want = (*step(eager), eager, *c[:4])
        # the atoms of rows that are not there hold what they held
        for n, (a, b) in enumerate(zip(got, want)):
            if n != 4:
                assert torch.equal(a, b), n
    bq.check_device_status()


@gpu
def test_two_calls_at_once(L):
    """Calls on two streams, each with a workspace of its own."""
    g = gen(31)
    page, Hk, D = 32, 2, 128
    for new, lens in (([1, 1], [5000, 70]), ([300, 1], [2000, 90])):
        off, ln, table, count = make_batch(g, new, lens, page)
        c = random_cache(g, count, Hk, page, D, 16, bq.INT8)
        qs = [randn(g, sum(new), 8, D).bfloat16() for _ in range(2)]
        want = [bq.kv_attention(q, c, off, ln, table, max(new), 5000) for q in qs]
        streams = [torch.cuda.Stream() for _ in qs]
        for _ in range(5):
            got = []
            for st, q in zip(streams, qs):
                st.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(st):
                    got.append(bq.kv_attention(q, c, off, ln, table, max(new), 5000))
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
def test_attention_repeats_its_bits(L):
    g = gen(13)
    for new, lens in (([1] * 4, [5000, 17, 900, 64]), ([70, 300], [2000, 300])):
        off, ln, table, count = make_batch(g, new, lens, 64)
        c = random_cache(g, count, 2, 64, 128, 16, bq.INT8)
        q = randn(g, sum(new), 8, 128).bfloat16()
        first = bq.kv_attention(q, c, off, ln, table, max(new), max(lens))
        for _ in range(3):
            assert torch.equal(first, bq.kv_attention(q, c, off, ln, table, max(new), max(lens)))


@gpu
@pytest.mark.parametrize("dtype", [bq.INT8, bq.FP8_E4M3])
def test_layer_of_them_together(L, dtype):
    """norm -> QKV linear -> rotary -> cache -> attention -> O linear -> norm,
    a prompt and then single tokens, each step against 64 bits on its own inputs."""
    g = gen(17)
    H, Hq, Hk, D, page, bt = 512, 4, 2, 128, 32, 8
    wq, sq = bq.quant_weight(0.05 * randn(g, (Hq + 2 * Hk) * D, H), dtype=dtype)
    wo, so = bq.quant_weight(0.05 * randn(g, H, Hq * D), dtype=dtype)
    w1 = (1 + 0.1 * randn(g, H)).bfloat16()
    turns, ms = bq.rope_frequencies(D, 10000.0, bq.ROPE_YARN, 4.0, 4096)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.randperm(8, generator=g, device="cuda").to(torch.int32).view(2, 4)
    cache = bq.kv_cache(8, Hk, page, D, bt, dtype)
    old = [0, 0]
    for new in ([70, 45], [1, 1], [1, 1]):
        T, lens = sum(new), [a + b for a, b in zip(old, new)]
        off, ln = torch.tensor([0, new[0], T], **i32), torch.tensor(lens, **i32)
        pos = torch.cat([torch.arange(a, a + b, **i32) for a, b in zip(old, new)])
        x, res = randn(g, T, H).bfloat16(), randn(g, T, H).bfloat16()
        q8, s, res = bq.rmsnorm_quant(x, w1, residual=res, dtype=dtype, res_out=res)
        _, y = ref.rmsnorm(res, w1, 1e-6)
        ref.check_codes(q8, s, y, 128, dtype, ref.norm_rel(H))
        qkv = bq.gemm(q8, s, wq, sq, dtype=dtype)
        heads = qkv.view(T, Hq + 2 * Hk, D)
        qk, v = heads[:, :Hq + Hk], heads[:, Hq + Hk:]
        want, mag = ref.rope(qk, pos, turns, 0, ms)
        bq.rope(qk, pos, turns, mscale=ms, out=qk)
        assert ((qk.double() - want).abs() <= want.abs() * ref.UBF16 + mag * 2.0 ** -20).all()
        k = qk[:, Hq:]
        want = [ref.append(a, b, t, off, ln, table, dtype)
                for a, b, t in ((cache.k, cache.ks, k), (cache.v, cache.vs, v))]
        bq.kv_append(cache, k, v, off, ln, table)
        assert torch.equal(cache.k, want[0][0]) and torch.equal(cache.v, want[1][0])
        assert torch.equal(cache.ks, want[0][1]) and torch.equal(cache.vs, want[1][1])
        o = bq.kv_attention(qk[:, :Hq], cache, off, ln, table, max(new), page * 4)
        want, _, tol, _ = ref.attention(qk[:, :Hq], cache.k, cache.v, cache.ks, cache.vs, off, ln,
                                     table, dtype)
        assert ((o.double() - want).abs() <= tol).all()
        out = bq.linear(o.view(T, Hq * D), wo, so, dtype=dtype)
        assert torch.isfinite(out).all()
        old = lens
    bq.check_device_status()
