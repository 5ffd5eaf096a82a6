"""GPU tests of the serving operators against plain implementations in 64 bits.

Tolerances are derived from the roundings that the definitions leave: a floating
output is off by half a step of its type (``eps / 2`` of its value) beside the
fp32 steps counted where they are used.  Levels, scales and int8 rows are equal."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import bit_integer_gemm_amd as lb  # noqa: E402

pytestmark = pytest.mark.gpu

BF, HF, FL = torch.bfloat16, torch.float16, torch.float32
STEP = 2.0 ** -24  # half a step of fp32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


# ---------------------------------------------------------------------------
# row quantisation and the linear layer
# ---------------------------------------------------------------------------

def quant_ref(x):
    """(q, sx): the exact quotient rounded, in float64 (127 x has at most 31 bits, so ties are seen).  A row that
    is not finite (a huge row may be, in fp16) has q = 0 and that as its scale."""
    x = x.double().numpy()
    amax = np.abs(x).max(1, keepdims=True)
    q = np.rint(np.divide(127.0 * x, amax, out=np.zeros_like(x), where=(amax > 0) & np.isfinite(amax)))
    return q.astype(np.int64), amax[:, 0].astype(np.float32) / np.float32(127)


def rows_with_ties(M, K, dtype, seed):
    """Normal rows with outliers; row 1 is all ties (amax 254 makes odd numbers half-integers), row 2 zero, row 3
    tiny, row 4 huge."""
    g = gen(seed)
    x = torch.randn(M, K, generator=g) * (1 + 30 * (torch.rand(K, generator=g) < 0.02))
    if M > 1:
        x[1] = torch.randint(-127, 128, (K,), generator=g).float()
        x[1, 0] = 254.0
    if M > 4:
        x[2] = 0
        x[3] *= 1e-7 if dtype == HF else 1e-37
        x[4] *= 600 if dtype == HF else 1e35
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF, HF, FL])
@pytest.mark.parametrize("M,K", [(1, 16), (5, 48), (7, 4096), (9, 11008), (3, 40000), (6, 131056)])
def test_quant_rows(dtype, M, K):
    x = rows_with_ties(M, K, dtype, 10 + M)
    wide = torch.full((M, K + 24), float("nan"), dtype=dtype, device="cuda")  # strided rows
    wide[:, :K] = x.cuda()
    q = torch.full((M, K), 77, dtype=torch.int8, device="cuda")
    sx = torch.empty(M, device="cuda")
    lb.lb_quant_rows_s8(wide[:, :K], q, sx)
    want, scale = quant_ref(x)
    assert np.array_equal(q.cpu().numpy(), want)
    assert np.array_equal(sx.cpu().numpy(), scale)


def test_quant_rows_not_finite():
    x = torch.randn(4, 64).to(BF)
    x[1, 3], x[2, 5] = float("inf"), float("nan")
    q, sx = torch.empty(4, 64, dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")
    lb.lb_quant_rows_s8(x.cuda(), q, sx)
    assert (q[1:3] == 0).all() and torch.isinf(sx[1]) and torch.isnan(sx[2])
    want, scale = quant_ref(x[[0, 3]])
    assert np.array_equal(q[[0, 3]].cpu().numpy(), want) and np.array_equal(sx[[0, 3]].cpu().numpy(), scale)


def linear_want(q, w, sx, sw, bias):
    """(product, result) in float64."""
    acc = q.astype(np.float64) @ w.double().numpy().T
    prod = acc * sx.astype(np.float64)[:, None] * sw.double().numpy()[None]
    return prod, prod if bias is None else prod + bias.double().numpy()[None]


def check_linear(out, prod, want, dtype):
    # float(acc), its two products and sx's own rounding: four fp32 half steps of the product; the sum: one of the result
    tol = half_step(dtype) * np.abs(want) + 5 * STEP * np.abs(prod) + 2 * STEP * np.abs(want)
    tol = tol * 1.001 + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    off = np.abs(out.cpu().double().numpy() - want)
    assert (off <= tol).all(), (off / tol).max()


SHAPES = [(1, 16, 16), (1, 4097, 4096), (2, 33, 144), (3, 1000, 1040), (5, 16, 2064), (15, 100, 272), (16, 640, 4096),
          (17, 31, 5504), (32, 129, 1024), (33, 65, 96), (48, 257, 160), (64, 1376, 4096), (65, 70, 112),
          (130, 515, 1008), (331, 200, 2048), (700, 1025, 528)]


@pytest.mark.parametrize("dtype", [BF, HF, FL])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(dtype, M, N, K):
    g = gen(M * 7 + N)
    x = (torch.randn(M, K, generator=g) * (1 + 20 * (torch.rand(K, generator=g) < 0.02))).to(dtype)
    w = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8)
    sw = torch.rand(N, generator=g) * 1e-3 + 1e-4
    bias = torch.randn(N, generator=g).to(dtype) if (M + N) % 2 else None
    wide = torch.full((M, K + 8), float("inf"), dtype=dtype, device="cuda")
    wide[:, :K] = x.cuda()
    flat = torch.full((M * N + 64,), 7.0, dtype=dtype, device="cuda")
    out = flat[:M * N].view(M, N)
    lb.lb_linear_w8a8(wide[:, :K], w.cuda(), sw.cuda(), out, bias=None if bias is None else bias.cuda())
    q, sx = quant_ref(x)
    prod, want = linear_want(q, w, sx, sw, bias)
    check_linear(out, prod, want, dtype)
    assert (flat[M * N:] == 7).all(), "write past out"


# one for each tile of the few-row kernel (rows x columns on 256 compute units), quantising for itself or not
TILES = [(4, 5000, 48), (2, 9001, 112), (4, 12288, 16400), (5, 5001, 48), (16, 9000, 240), (20, 5000, 80), (17, 3001, 2032),
         (30, 9001, 64), (33, 4000, 1040), (64, 5000, 80), (50, 9001, 48), (130, 6000, 80), (200, 4001, 144), (256, 4096, 272)]


@pytest.mark.parametrize("M,N,K", TILES)
def test_linear_tiles(M, N, K):
    test_linear(BF if N % 2 else HF, M, N, K)


# tiles with deep rings: 128 x 64, 64 x 128, 128 x 128; K of one stage and less, of
# fewer stages than the ring has, of more; rows and columns that fill no tile
@pytest.mark.parametrize("dtype", [BF, HF, FL])
@pytest.mark.parametrize("M,N", [(331, 4097), (300, 6144), (1030, 2070)])
@pytest.mark.parametrize("K", [16, 272, 784])
def test_linear_deep_tiles(M, N, K, dtype):
    test_linear(dtype, M, N, K)


@pytest.mark.parametrize("dtype", [BF, HF, FL])
@pytest.mark.parametrize("M,N,K", [(4, 50, 256), (40, 96, 512), (300, 777, 1024), (2048, 1376, 512)])
def test_scaled_product(dtype, M, N, K):
    g = gen(M + N)
    x = torch.randint(-128, 128, (M, K), generator=g, dtype=torch.int8)
    w = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8)
    sx, sw = torch.rand(M, generator=g) * 1e-2, torch.rand(N, generator=g) * 1e-3
    bias = torch.randn(N, generator=g).to(dtype)
    for b in (None, bias):
        out = torch.empty(M, N, dtype=dtype, device="cuda")
        lb.lb_gemm_s8_scaled(x.cuda(), w.cuda(), sx.cuda(), sw.cuda(), out, bias=None if b is None else b.cuda())
        prod, want = linear_want(x.numpy(), w, sx.numpy(), sw, b)
        check_linear(out, prod, want, dtype)


def test_scaled_product_every_tile():
    """Each tile of the scaled product, by the variant override, gives the same bits."""
    import os
    M, N, K = 300, 520, 784
    g = gen(5)
    x = torch.randint(-128, 128, (M, K), generator=g, dtype=torch.int8).cuda()
    w = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8).cuda()
    sx, sw = (torch.rand(M, generator=g) * 1e-2).cuda(), (torch.rand(N, generator=g) * 1e-3).cuda()
    bias = torch.randn(N, generator=g).to(HF).cuda()
    prod, want = linear_want(x.cpu().numpy(), w.cpu(), sx.cpu().numpy(), sw.cpu(), bias.cpu())
    first, old = None, os.environ.get("LB_AUTO_VARIANT")
    try:
        for v in range(9):
            os.environ["LB_AUTO_VARIANT"] = str(v)
            out = torch.empty(M, N, dtype=HF, device="cuda")
            lb.lb_gemm_s8_scaled(x, w, sx, sw, out, bias=bias)
            check_linear(out, prod, want, HF)
            first = out if first is None else first
            assert torch.equal(out, first), v
    finally:
        os.environ.pop("LB_AUTO_VARIANT", None)
        if old is not None:
            os.environ["LB_AUTO_VARIANT"] = old


def test_linear_rows_not_finite_or_zero():
    for M in (4, 70):
        x = torch.randn(M, 128).to(BF)
        x[0], x[1, 7], x[2, 9] = 0, float("nan"), float("-inf")
        w, sw = torch.randint(-128, 128, (40, 128), dtype=torch.int8), torch.rand(40)
        bias = torch.randn(40).to(BF)
        out = torch.empty(M, 40, dtype=BF, device="cuda")
        lb.lb_linear_w8a8(x.cuda(), w.cuda(), sw.cuda(), out, bias=bias.cuda())
        assert torch.equal(out[0].cpu(), bias) and torch.isnan(out[1:3]).all() and torch.isfinite(out[3:]).all()


# ---------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------

def empty_cache(pages, H, page, D, dtype, device="cuda"):
    """Four tensors that hold garbage: every level 15 with NaN scales."""
    c = [torch.full((pages, H, page, D // 2), 255, dtype=torch.uint8, device=device) for _ in range(2)]
    p = [torch.full((pages, H, page, 2), float("nan"), dtype=dtype, device=device) for _ in range(2)]
    return c[0], c[1], p[0], p[1]


def quantise_ref(x):
    """(levels, scale, low) in the definition's own fp32 steps (numpy's division is correctly rounded)."""
    dtype = x.dtype
    f = x.float().numpy()
    low, high = f.min(-1, keepdims=True), f.max(-1, keepdims=True)
    with np.errstate(over="ignore"):
        scale = torch.from_numpy((high - low) / np.float32(15)).to(dtype)
    s = scale.float().numpy()
    ok = (s > 0) & np.isfinite(s)
    u = np.rint(np.divide(f - low, s, out=np.zeros_like(f), where=ok))
    return np.clip(u, 0, 15), scale, torch.from_numpy(low).to(dtype)


def vectors(T, H, D, dtype, seed):
    g = gen(seed)
    x = torch.randn(T, H, D, generator=g) * torch.exp(torch.randn(T, H, 1, generator=g)) + torch.randn(T, H, 1, generator=g)
    if T > 6:
        x[1] = 0.75                                                    # constant: scale 0
        x[2] = torch.randint(0, 31, (H, D), generator=g).float()      # range 30: every odd number a tie
        x[2, :, 0], x[2, :, 1] = 0, 30
        x[3] *= 3e-6 if dtype == HF else 1e-38                         # scales among the subnormals
        x[4] *= 1000 if dtype == HF else 1e36
        x[5] = 0
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,H,page", [(1, 1, 16), (7, 3, 16), (33, 8, 48), (100, 5, 64)])
def test_cache_write_and_read(dtype, D, T, H, page):
    pages = -(-T // page) + 2
    k, v = vectors(T, H, D, dtype, 1), vectors(T, H, D, dtype, 2)
    slots = torch.randperm(pages * page, generator=gen(3))[:T]
    if T > 6:
        slots[6] = -1
    Kc, Vc, Kp, Vp = empty_cache(pages, H, page, D, dtype)
    before = [t.clone() for t in (Kc, Vc, Kp, Vp)]
    qkv = torch.full((T, 3, H, D), float("nan"), dtype=dtype, device="cuda")
    qkv[:, 1], qkv[:, 2] = k.cuda(), v.cuda()
    lb.lb_kv4_write(qkv[:, 1], qkv[:, 2], slots.cuda(), Kc, Vc, Kp, Vp)
    ask = torch.cat([slots, torch.tensor([-1, pages * page, -2 ** 40, 2 ** 40])]).cuda()
    ko = torch.full((T + 4, H, D), 3.0, dtype=dtype, device="cuda")
    vo = ko.clone()
    lb.lb_kv4_read(Kc, Vc, Kp, Vp, ask, ko, vo)
    keep = (slots >= 0).numpy()
    for x, c, p, out in ((k, Kc, Kp, ko), (v, Vc, Vp, vo)):
        u, s, low = quantise_ref(x)
        c2 = c.cpu().permute(0, 2, 1, 3).reshape(pages * page, H, D // 2)[slots[keep]].numpy()
        p2 = p.cpu().permute(0, 2, 1, 3).reshape(pages * page, H, 2)[slots[keep]]
        assert np.array_equal(c2, (u[..., 0::2] + 16 * u[..., 1::2]).astype(np.uint8)[keep])
        assert torch.equal(p2, torch.cat([s, low], -1)[keep])
        val = torch.from_numpy(u.astype(np.float32)) * s.float() + low.float()  # u s is exact in fp32
        assert torch.equal(out[:T].cpu()[keep], val.to(dtype)[keep])
        assert (out[T:] == 0).all() and (T <= 6 or (out[6] == 0).all())
        # off by at most half a level (one and a half where s rounds down), and half a step of the value read
        err = (out[:T].cpu()[keep].double() - x[keep].double()).abs()
        tiny = torch.finfo(dtype).smallest_normal
        room = 0.5 + 15 * half_step(dtype)
        sd = s[keep].double()
        assert (err <= room * sd + half_step(dtype) * (x[keep].double().abs() + sd) + 16 * tiny * torch.finfo(dtype).eps).all()
    # nothing else was touched
    rest = torch.ones(pages * page, dtype=torch.bool)
    rest[slots[keep]] = False
    for now, old in zip((Kc, Vc, Kp, Vp), before):
        a, b = (t.cpu().view(torch.uint8).permute(0, 2, 1, 3).reshape(pages * page, -1)[rest] for t in (now, old))
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_cache_not_finite(dtype):
    T, H, D, page = 5, 2, 128, 16
    k = torch.randn(T, H, D).to(dtype)
    k[1, 0, 5], k[2, 1, 127], k[3, 0, 0] = float("nan"), float("inf"), float("-inf")
    if dtype == BF:
        k[4, 1, 0], k[4, 1, 1] = 3e38, -3e38  # a range beyond fp32
    cache = empty_cache(1, H, page, D, dtype)
    slots = torch.arange(T).cuda()
    lb.lb_kv4_write(k.cuda(), k.cuda(), slots, *cache)
    out = torch.empty(T, H, D, dtype=dtype, device="cuda")
    lb.lb_kv4_read(*cache, slots, out, torch.empty_like(out))
    bad = torch.zeros(T, H, dtype=torch.bool)
    bad[1, 0] = bad[2, 1] = bad[3, 0] = True
    bad[4, 1] = dtype == BF
    assert torch.equal(torch.isnan(out.cpu()).all(-1), bad) and torch.equal(torch.isnan(out.cpu()).any(-1), bad)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

class Batch:
    """Sequences in a paged cache whose unused places hold NaN, and their 64-bit attention."""

    def __init__(self, lens, nqs, Hq, Hkv, D, page, dtype, seed=0, extra_pages=2, spread=1.0, first_page=0, pages=None):
        g = gen(seed)
        self.lens, self.nqs, self.Hq, self.Hkv, self.D, self.page, self.dtype = lens, nqs, Hq, Hkv, D, page, dtype
        used = [-(-n // page) for n in lens]
        self.pages = pages or sum(used) + extra_pages + first_page
        self.cache = empty_cache(self.pages, Hkv, page, D, dtype)
        ids = (first_page + torch.randperm(sum(used) + extra_pages, generator=g)).to(torch.int32)
        width = max(max(used), 1) + 1
        self.table = torch.full((len(lens), width + 3), 2 ** 31 - 1, dtype=torch.int32)  # rows ldt apart
        self.kv, slots, ks, vs, at = [], [], [], [], 0
        for b, n in enumerate(lens):
            self.table[b, :used[b]] = ids[at:at + used[b]]
            at += used[b]
            k = torch.randn(n, Hkv, D, generator=g).to(dtype)
            v = (torch.randn(n, Hkv, D, generator=g) * spread + 0.3).to(dtype)
            t = torch.arange(n)
            slots.append(self.table[b].long()[t // page] * page + t % page)
            ks.append(k)
            vs.append(v)
        self.slots = torch.cat(slots).cuda()
        if len(self.slots):
            lb.lb_kv4_write(torch.cat(ks).cuda(), torch.cat(vs).cuda(), self.slots, *self.cache)
        for k, v in zip(ks, vs):
            self.kv.append(tuple(torch.from_numpy(u) * s.double() + low.double() for u, s, low in map(quantise_ref, (k, v))))
        self.smax = max([float(quantise_ref(k)[1].float().max()) for k in ks if len(k)] + [0.0])
        self.table = self.table.cuda()[:, :width]
        self.q_off = torch.tensor(np.concatenate([[0], np.cumsum(nqs)]), dtype=torch.int32).cuda()
        self.total = sum(nqs)
        self.q = torch.randn(self.total, Hq, D, generator=g).to(dtype)

    def run(self, window=0, causal=True, scale=None, **kw):
        wide = torch.full((self.total, self.Hq * self.D + 16), float("nan"), dtype=self.dtype, device="cuda")
        q = wide[:, :self.Hq * self.D].unflatten(1, (self.Hq, self.D))
        q.copy_(self.q)
        base = torch.full((self.total, self.Hq * self.D + 8), 5.0, dtype=self.dtype, device="cuda")
        out = base[:, :self.Hq * self.D].unflatten(1, (self.Hq, self.D))
        lse = torch.full((self.total, self.Hq), 9.0, device="cuda")
        lb.lb_attn_kv4(q, *self.cache, self.table, self.q_off, torch.tensor(self.lens, dtype=torch.int32).cuda(), out,
                       lse=lse, window=window, causal=causal, scale=scale, **kw)
        assert (base[:, self.Hq * self.D:] == 5).all(), "write between rows"
        return out, lse

    def want(self, window=0, causal=True, scale=None, kv=None):
        """(out, lse, error bound of a score) in float64, sequence by sequence."""
        scale = self.D ** -0.5 if scale is None else scale
        out = torch.zeros(self.total, self.Hq, self.D, dtype=torch.float64)
        lse = torch.full((self.total, self.Hq), -math.inf, dtype=torch.float64)
        top = torch.zeros(self.total, self.Hq, dtype=torch.float64)
        G, at = self.Hq // self.Hkv, 0
        for b, (n, nq) in enumerate(zip(self.lens, self.nqs)):
            if n == 0:
                at += nq
                continue
            k, v = (kv or self.kv)[b]
            pos = torch.arange(nq) + n - nq
            t = torch.arange(n)
            see = torch.ones(nq, n, dtype=torch.bool)
            if causal:
                see &= t <= pos[:, None]
            if window:
                see &= t > pos[:, None] - window
            q = self.q[at:at + nq].double()
            for h in range(self.Hq):
                z = (q[:, h] @ k[:, h // G].T) * scale
                z = z.masked_fill(~see, -math.inf)
                m = z.max(1).values
                some = m > -math.inf
                e = torch.exp(z[some] - m[some, None])
                rows = at + torch.arange(nq)[some]
                out[rows, h] = (e @ v[:, h // G]) / e.sum(1, keepdim=True)
                lse[rows, h] = m[some] + torch.log(e.sum(1))
                top[rows, h] = z[some].masked_fill(~see[some], 0).abs().max(1).values
            at += nq
        # A score: D/32 products of 32 terms in sequence, each adding about 8 rounded steps, of partial sums no larger
        # than (base + 15) sum |q| with base 128 (bf16) or 64 (fp16); then s, m, the softmax scale: six half steps.
        mag = (143 if self.dtype == BF else 79) * self.q.double().abs().sum(-1)
        score = (self.D / 32 + 8) * 2 * STEP * mag * self.smax * scale + 6 * STEP * (top + 1)
        return out, lse, score

    def check(self, got, want, vmax=None):
        (out, lse), (wout, wlse, score) = got, want
        out, lse = out.cpu().double(), lse.cpu().double()
        if vmax is None:
            vmax = max([float(v.abs().max()) for _, v in self.kv if len(v)] + [0.0])
        # weights off by e^score (both above and below the fraction) and, in two bf16 parts, by 2^-16; the fp32 sums of
        # weights and outputs by less than 2^-16; the division and one rounding to the type
        tol = half_step(self.dtype) * wout.abs() + (2 * score[..., None] + 2.0 ** -15) * 2 * vmax
        tol = tol + torch.finfo(self.dtype).smallest_normal * torch.finfo(self.dtype).eps
        off = (out - wout).abs()
        assert (off <= tol).all(), (float((off / tol).max()), float(off.max()))
        none = wlse == -math.inf
        assert torch.equal(lse == -math.inf, none) and (out[none] == 0).all()
        ltol = score + 2.0 ** -20 * (1 + wlse.abs())
        assert ((lse - wlse).abs()[~none] <= ltol[~none]).all()


GROUPS = [(1, 1), (3, 3), (8, 2), (6, 2), (16, 1), (40, 2), (71, 1)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", GROUPS)
def test_attention_single_tokens(dtype, D, Hq, Hkv):
    """One query each, lengths around the blocks' and pages' edges, an empty sequence among them."""
    b = Batch([1, 0, 15, 16, 17, 31, 32, 33, 100, 300], [1] * 10, Hq, Hkv, D, 16, dtype, seed=D + Hq)
    b.check(b.run(max_q=1), b.want())


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D,page", [(64, 48), (128, 64), (256, 32)])
@pytest.mark.parametrize("window", [0, 1, 20, 200])
def test_attention_ragged_queries(dtype, D, page, window):
    """Sequences with no, one, some and many queries; with more queries than keys, so that the first see nothing."""
    b = Batch([130, 5, 64, 0, 257, 40, 333], [3, 9, 1, 2, 70, 0, 33], 8, 2, D, page, dtype, seed=window)
    b.check(b.run(window=window, max_q=70), b.want(window=window))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("Hq", [12, 24])
def test_attention_not_causal(dtype, window, Hq):
    b = Batch([130, 5, 600], [3, 9, 40], Hq, 3, 128, 16, dtype, seed=4)
    b.check(b.run(causal=False, window=window, scale=0.2), b.want(causal=False, window=window, scale=0.2))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("Hq,Hkv,D,nq", [(8, 1, 128, 1), (4, 4, 64, 1), (16, 2, 256, 3), (16, 2, 128, 40)])
def test_attention_split_keys(dtype, Hq, Hkv, D, nq):
    """Long contexts, whose keys are split among workgroups, with as much workspace as asked for, some and none."""
    b = Batch([6000, 1, 3000], [nq, 1, nq], Hq, Hkv, D, 64, dtype, seed=nq)
    want = b.want()
    need = lb.lb_attn_kv4_workspace(3, b.total, nq, Hq, Hkv, D, 6000)
    assert need > 0
    for size in (need, need // 3, 0):
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        got = b.run(max_q=nq, max_len=6000, workspace=ws)
        b.check(got, want)
        again = b.run(max_q=nq, max_len=6000, workspace=ws)
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1]), "not the same bits twice"


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lens,nq,Hq,Hkv,D", [
    ([1, 4000, 0, 700, 31, 3333, 32, 2000, 3999, 5] * 4, 1, 8, 8, 64),     # shares that cut and that hold many
    ([3100] * 33, 1, 8, 8, 128),                                           # equal tiles, which stay whole
    ([3500, 100, 40, 0, 2500, 3600, 3072, 1, 900, 77, 64, 3000], 5, 64, 8, 64),   # three tiles of rows to a head
    ([6000, 50, 3000] * 11, 1, 16, 8, 256)])
def test_attention_shares(dtype, lens, nq, Hq, Hkv, D):
    """More tiles than compute units and lengths that differ: the work in equal shares, and with no workspace a
    tile to a workgroup."""
    b = Batch(lens, [nq] * len(lens), Hq, Hkv, D, 32, dtype, seed=len(lens))
    want = b.want()
    need = lb.lb_attn_kv4_workspace(len(lens), b.total, nq, Hq, Hkv, D, max(lens))
    assert need > 0
    for size in (need, 0):
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        got = b.run(max_q=nq, max_len=max(lens), workspace=ws)
        b.check(got, want)
        again = b.run(max_q=nq, max_len=max(lens), workspace=ws)
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1]), "not the same bits twice"


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_chunks_of_several_sequences(dtype, D):
    """Many rows of a key head, tiles in the order of their keys; one sequence's keys in ranges."""
    b = Batch([300, 700, 90, 1100], [200, 60, 90, 1], 8, 2, D, 48, dtype, seed=D)
    b.check(b.run(max_q=200), b.want())
    b = Batch([2600], [100], 6, 2, D, 64, dtype, seed=D)
    want = b.want()
    need = lb.lb_attn_kv4_workspace(1, 100, 100, 6, 2, D, 2600)
    assert need > 0
    for size in (need, need // 2, 0):
        b.check(b.run(max_q=100, max_len=2600, workspace=torch.empty(size, dtype=torch.uint8, device="cuda")), want)


def test_attention_hints_are_only_hints():
    """max_len far below and above the lengths, and a table wider than they need."""
    b = Batch([900, 37, 2000], [1, 1, 1], 8, 2, 64, 16, HF, seed=12)
    want = b.want()
    for max_len in (0, 1, 100, 10 ** 6):
        b.check(b.run(max_q=1, max_len=max_len), want)
    b = Batch([900, 37, 500], [90, 30, 5], 8, 2, 64, 16, BF, seed=13)
    want = b.want()
    for max_len in (0, 64, 10 ** 6):
        b.check(b.run(max_len=max_len), want)


@pytest.mark.parametrize("nq", [1, 60])
def test_attention_value_that_is_not_finite(nq):
    """A value vector that is NaN makes NaN of the rows that see it and leaves the others, and every lse."""
    b = Batch([100, 50], [nq, nq] if nq == 1 else [nq, 40], 8, 2, 128, 16, BF, seed=14)
    want = b.want()
    slot = int(b.slots[80])
    b.cache[3][slot // 16, 1, slot % 16] = float("nan")   # sequence 0, key 80, key head 1
    out, lse = b.run()
    bad = torch.zeros(b.total, 8, dtype=torch.bool)
    for i in range(b.nqs[0]):
        bad[i, 4:] = 100 - b.nqs[0] + i >= 80
    assert torch.equal(torch.isnan(out.cpu()).all(-1), bad) and torch.equal(torch.isnan(out.cpu()).any(-1), bad)
    keep = ~bad
    fixed = torch.where(bad[..., None], want[0].float(), out.cpu().float()).to(BF)
    b.check((fixed, lse), want, vmax=10.0)
    assert keep.any()


@pytest.mark.parametrize("spread", [1e-3, 100.0])
def test_attention_small_and_large_values(spread):
    """The values' scales reach far below and above one in fp16."""
    b = Batch([200, 900], [1, 5], 8, 2, 128, 16, HF, seed=1, spread=spread)
    b.check(b.run(), b.want())


@pytest.mark.parametrize("nq", [1, 30])
def test_attention_constant_and_far_keys(nq):
    """Vectors of scale zero, and scores so far apart that one key takes all the weight."""
    b = Batch([150], [nq], 4, 2, 64, 16, BF, seed=2)
    k, v = torch.randn(150, 2, 64).to(BF), torch.randn(150, 2, 64).to(BF)
    k[10], v[20], k[30], v[30] = 0.5, -2.0, 0, 0
    k[77] = (k[77].float() * 30).to(BF)
    lb.lb_kv4_write(k.cuda(), v.cuda(), b.slots, *b.cache)
    b.kv = [tuple(torch.from_numpy(u) * s.double() + low.double() for u, s, low in map(quantise_ref, (k, v)))]
    b.smax = float(quantise_ref(k)[1].float().max())
    b.check(b.run(), b.want())


@pytest.mark.parametrize("nq,Hq", [(1, 4), (24, 4), (49, 16)])
def test_attention_nan_stays_in_its_row(nq, Hq):
    """A key that is NaN makes NaN of the queries that see it, of its key head, and of no others; so does a query."""
    b = Batch([100, 50], [nq, nq], Hq, 2, 128, 16, HF, seed=3)
    kp = b.cache[2].permute(0, 2, 1, 3).reshape(-1, 2, 2)
    slot = int(b.slots[90])
    b.cache[2][slot // 16, 1, slot % 16] = float("nan")   # sequence 0, key 90, head 1
    b.q[b.total - 1, 0, 5] = float("nan")
    out, lse = b.run()
    bad = torch.zeros(b.total, Hq, dtype=torch.bool)
    for i in range(nq):
        bad[i, Hq // 2:] = 100 - nq + i >= 90
    bad[b.total - 1, 0] = True
    assert kp is not None
    assert torch.equal(torch.isnan(out.cpu()).any(-1), bad) and torch.equal(torch.isnan(lse.cpu()), bad)


@pytest.mark.parametrize("nq,Hq", [(1, 4), (24, 4), (30, 16)])
def test_attention_pages_outside_the_cache(nq, Hq):
    """Keys of a page number outside the cache are not seen; lens beyond the table's width counts as its width."""
    b = Batch([64, 80], [nq, nq], Hq, 2, 64, 16, BF, seed=6)
    b.table[0, 1], b.table[1, 2] = -7, b.pages
    got = b.run()
    kv = []
    for (k, v), hole in zip(b.kv, (range(16, 32), range(32, 48))):
        keep = [t for t in range(len(k)) if t not in hole]
        kv.append((k, v, keep))
    # the same softmax with the holes' scores at minus infinity: keys so that only their absence matters
    out = torch.zeros(b.total, Hq, 64, dtype=torch.float64)
    lse = torch.zeros(b.total, Hq, dtype=torch.float64)
    for s, (k, v, keep) in enumerate(kv):
        for i in range(nq):
            pos = len(k) - nq + i
            t = [j for j in keep if j <= pos]
            for h in range(Hq):
                z = (k[t, h // (Hq // 2)] @ b.q[s * nq + i, h].double()) / 8
                out[s * nq + i, h] = torch.softmax(z, 0) @ v[t, h // (Hq // 2)]
                lse[s * nq + i, h] = torch.logsumexp(z, 0)
    b.check(got, (out, lse, b.want()[2]))
    full = Batch([48, 48], [nq, nq], Hq, 2, 64, 16, BF, seed=7)
    full.table = full.table[:, :3]
    want = full.want()
    full.lens = [100000, 2 ** 31 - 1]
    full.check(full.run(max_len=48), want)


def test_attention_rows_outside_every_sequence():
    b = Batch([20, 30], [2, 3], 4, 2, 64, 16, HF, seed=8)
    want = b.want()
    q_off = b.q_off.clone()
    b.q = torch.cat([b.q, torch.randn(2, 4, 64).to(HF)])
    b.total += 2
    for kw in (dict(), dict(workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))):
        out, lse = b.run(max_q=3, **kw)
        b.total -= 2
        b.check((out[:5], lse[:5]), want)
        b.total += 2
        assert (out[5:] == 5).all() and (lse[5:] == 9).all()
    assert torch.equal(q_off, b.q_off)


def test_attention_and_cache_beyond_four_gib():
    """Slots whose byte offsets pass 2^32 in the levels, written, read back and attended over."""
    D, H, page = 256, 8, 128
    pages = (5 * 2 ** 30) // (H * page * D // 2)
    g = gen(9)
    cache = tuple(torch.empty(pages, H, page, D // 2, dtype=torch.uint8, device="cuda") for _ in range(2)) + \
        tuple(torch.empty(pages, H, page, 2, dtype=HF, device="cuda") for _ in range(2))
    n = 300
    table = torch.tensor([[pages - 1, pages // 2, pages - 7]], dtype=torch.int32)
    t = torch.arange(n)
    slots = (table[0].long()[t // page] * page + t % page).cuda()
    k, v = torch.randn(n, H, D, generator=g).to(HF), torch.randn(n, H, D, generator=g).to(HF)
    lb.lb_kv4_write(k.cuda(), v.cuda(), slots, *cache)
    ko, vo = torch.empty_like(k.cuda()), torch.empty_like(v.cuda())
    lb.lb_kv4_read(*cache, slots, ko, vo)
    b = Batch([n], [2], 16, H, D, page, HF, seed=9)
    for x, o in ((k, ko), (v, vo)):
        u, s, low = quantise_ref(x)
        assert torch.equal(o.cpu(), (torch.from_numpy(u.astype(np.float32)) * s.float() + low.float()).to(HF))
    b.kv = [tuple(torch.from_numpy(u) * s.double() + low.double() for u, s, low in map(quantise_ref, (k, v)))]
    b.cache, b.table = cache, table.cuda()
    b.check(b.run(), b.want())


# ---------------------------------------------------------------------------
# together, on other streams and in graphs
# ---------------------------------------------------------------------------

def layer_step(x, w, sw, out, slots, cache, table, q_off, lens, attn, ws1, ws2, stream=None):
    """A projection, the cache's append and attention over it, as a decoder layer strings them together."""
    lb.lb_linear_w8a8(x, w, sw, out, workspace=ws1, stream=stream)
    B = x.shape[0]
    q = out[:, :1024].unflatten(1, (8, 128))
    k = out[:, 1024:1280].unflatten(1, (2, 128))
    v = out[:, 1280:].unflatten(1, (2, 128))
    lb.lb_kv4_write(k, v, slots, *cache, stream=stream)
    lb.lb_attn_kv4(q, *cache, table, q_off, lens, attn, max_q=1, max_len=2000, workspace=ws2, stream=stream)
    return B


def layer_state(B=3, seed=0):
    g = gen(seed)
    d = dict(x=torch.randn(B, 512, generator=g).to(BF).cuda(), w=torch.randint(-127, 128, (1536, 512), generator=g, dtype=torch.int8).cuda(),
             sw=(torch.rand(1536, generator=g) * 1e-3).cuda(), out=torch.empty(B, 1536, dtype=BF, device="cuda"))
    pages, page = 64 * B, 32
    cache = empty_cache(pages, 2, page, 128, BF)
    slots = torch.arange(pages * page).cuda()
    lb.lb_kv4_write(*(torch.randn(pages * page, 2, 128, generator=g).to(BF).cuda() for _ in range(2)), slots, *cache)
    lens = torch.tensor([2000, 700, 33][:B], dtype=torch.int32).cuda()
    table = torch.arange(pages, dtype=torch.int32).view(B, 64).cuda()
    d |= dict(cache=cache, table=table, lens=lens, q_off=torch.arange(B + 1, dtype=torch.int32).cuda(),
              slots=(torch.arange(B).cuda() * 64 * page + lens.long() - 1), attn=torch.empty(B, 8, 128, dtype=BF, device="cuda"),
              ws1=torch.empty(lb.lb_linear_w8a8_workspace(B, 512, 1536), dtype=torch.uint8, device="cuda"),
              ws2=torch.empty(lb.lb_attn_kv4_workspace(B, B, 1, 8, 2, 128, 2000), dtype=torch.uint8, device="cuda"))
    return d


def test_layer_on_a_side_stream():
    d = layer_state()
    layer_step(**d)
    torch.cuda.synchronize()
    want = d["attn"].clone()
    d["attn"].zero_()
    d["out"].zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    layer_step(**d, stream=s)                     # the stream as an argument
    s.synchronize()
    assert torch.equal(d["attn"], want)
    d["attn"].zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):                    # and as torch's current one
        layer_step(**d)
    s.synchronize()
    assert torch.equal(d["attn"], want)
    with pytest.raises(ValueError, match="workspace"):
        lb.lb_linear_w8a8(d["x"], d["w"], d["sw"], d["out"], stream=s)


def test_layer_in_a_graph():
    """Captured once, replayed on changing inputs with eager work between the replays."""
    d = layer_state()
    layer_step(**d)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer_step(**d)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer_step(**d)
    for i in range(4):
        d["x"].copy_(torch.randn(3, 512, generator=gen(50 + i)).to(BF))
        d["lens"].copy_(torch.tensor([2000 - 300 * i, 700 + i, 33], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = d["attn"].clone()
        d["attn"].zero_()
        layer_step(**d)
        torch.cuda.synchronize()
        assert torch.equal(got, d["attn"]) and torch.isfinite(got).all(), i


# ---------------------------------------------------------------------------
# prompts: values and weights of any size
# ---------------------------------------------------------------------------

def refill(b, k, v, seq=0):
    """Other keys and values (n, Hkv, D) for a sequence of a batch."""
    at = sum(b.lens[:seq])
    lb.lb_kv4_write(k.cuda(), v.cuda(), b.slots[at:at + len(k)].contiguous(), *b.cache)
    held = [quantise_ref(x) for x in (k, v)]
    b.kv[seq] = tuple(torch.from_numpy(u) * s.double() + low.double() for u, s, low in held)
    b.smax = max(b.smax, float(held[0][1].float().max()))


def largest_seen(b, window=0):
    """The largest value that each row sees (total, 1, 1), of any head; rows that see nothing: 0."""
    rows = []
    for n, nq, (_, v) in zip(b.lens, b.nqs, b.kv):
        for pos in range(n - nq, n):
            seen = v[max(0, pos + 1 - window) if window else 0:max(0, pos + 1)]
            rows.append(float(seen.abs().max()) if len(seen) else 0.0)
    return torch.tensor(rows, dtype=torch.float64)[:, None, None]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype,times", [(HF, 2.0 ** 10), (BF, 2.0 ** 10), (BF, 2.0 ** 20), (BF, 2.0 ** 23), (BF, 2.0 ** 36),
                                         (BF, 1e30)])
def test_attention_prompt_large_value_that_only_some_rows_see(dtype, D, times):
    """A vector of values far above the others: the rows before it come out as if it were not there."""
    b = Batch([700, 260], [200, 100], 8, 2, D, 48, dtype, seed=D)
    k, v = torch.randn(700, 2, D, generator=gen(1)).to(dtype), torch.randn(700, 2, D, generator=gen(2)).to(dtype)
    v[650] = (v[650].float() * times).to(dtype)
    refill(b, k, v)
    b.check(b.run(max_q=200), b.want(), vmax=largest_seen(b))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("times", [2.0 ** 23, 1e12, 1e30])
def test_attention_prompt_large_values_before_the_window(D, times):
    """Values that no row sees, in the first tile of keys: a page that a server has given to another sequence."""
    b = Batch([700], [200], 8, 2, D, 16, BF, seed=D)
    k, v = torch.randn(700, 2, D, generator=gen(1)).to(BF), torch.randn(700, 2, D, generator=gen(2)).to(BF)
    v[384:401] = (v[384:401].float() * times).to(BF)   # the first query stands at 500 and sees 401 .. 500
    refill(b, k, v)
    b.check(b.run(window=100, max_q=200), b.want(window=100), vmax=largest_seen(b, 100))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_prompt_small_values_beside_zeros(D):
    """Values of all sizes in one prompt, some exactly zero, and a sequence whose values are all tiny."""
    b = Batch([600, 300], [150, 150], 8, 2, D, 16, BF, seed=D)
    for seq, n in ((0, 600), (1, 300)):
        k, v = torch.randn(n, 2, D, generator=gen(3)), torch.randn(n, 2, D, generator=gen(4))
        size = 2.0 ** torch.randint(-9, 9, (n, 1, 1), generator=gen(5)).float() if seq == 0 else torch.tensor(2.0 ** -100)
        v = v * size
        v[5::7] = 0
        refill(b, k.to(BF), v.to(BF), seq)
    b.check(b.run(max_q=150), b.want(), vmax=largest_seen(b))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n,nq,octaves", [(131072, 1, 24.4), (131072, 1, 3), (100000, 3, 24.4), (20000, 64, 24.4), (20000, 64, 5),
                                          (60000, 64, 0)])
def test_attention_sum_of_many_equal_weights(dtype, n, nq, octaves):
    """The log of a long sum: one key of weight 1 and many of 2^-octaves, which fp32 sums lose one by one.

    A weight is off by a step of exp2 and its score's error; the sixteen of a lane are added in turn, the lane's sums of
    all blocks without loss, then 4 lanes, 16 waves and 64 ranges at most: 15 + 2 + 2 + 16 + 64 half steps, and 4 of
    the exponential and the logarithm, below 2^-17."""
    b = Batch([n], [nq], 4, 1, 64, 16, dtype, seed=1)
    k, v = torch.full((n, 1, 64), -octaves * math.log(2) / 8), torch.randn(n, 1, 64, generator=gen(7))
    k[3] = 0
    b.smax = 0.0   # constant keys: no scale
    refill(b, k.to(dtype), v.to(dtype))
    b.q = torch.ones_like(b.q)
    _, wlse, score = b.want()
    for size in (0, lb.lb_attn_kv4_workspace(1, nq, nq, 4, 1, 64, n)):
        lse = b.run(max_q=nq, max_len=n, workspace=torch.empty(size, dtype=torch.uint8, device="cuda"))[1].cpu().double()
        assert ((lse - wlse).abs() <= score + 2.0 ** -17 + 2.0 ** -22 * wlse.abs()).all(), float((lse - wlse).abs().max())


def check_weighted(b, got, want, scale=None):
    """Rows against what they see: off by half a step of the output, by the scores' errors, and by 2^-10 of the
    weighted mean of the values' magnitudes (weights and values are held to 2^-12 at least, values in two roundings),
    however small that is beside the largest value."""
    mean = b.want(kv=[(k, v.abs().amax(-1, keepdim=True).expand_as(v)) for k, v in b.kv], scale=scale)[0]
    out, (wout, wlse, score) = got[0].cpu().double(), want
    tol = half_step(b.dtype) * wout.abs() + (2 * score[..., None] + 2.0 ** -10) * mean
    off = (out - wout).abs()
    assert (off <= tol + torch.finfo(b.dtype).smallest_normal).all(), float((off / tol).max())
    assert ((got[1].cpu().double() - wlse).abs() <= score + 2.0 ** -20 * (1 + wlse.abs())).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype,octaves", [(HF, 5), (HF, 24.4)] + [(BF, o) for o in (5, 24.4, 25.2, 27.5, 31, 36)])
def test_attention_prompt_light_keys_beside_a_heavy_one(dtype, D, octaves):
    """One key takes nearly all the weight and has no value: the output is what the many others add (in fp16 as long
    as that is a normal number)."""
    n, nq = 20000, 64
    b = Batch([n], [nq], 4, 1, D, 16, dtype, seed=D)
    k = torch.full((n, 1, D), -octaves * math.log(2) / math.sqrt(D))
    v = 1 + 0.3 * torch.randn(n, 1, D, generator=gen(7))
    k[3], v[3] = 0, 0
    b.smax = 0.0   # constant keys: no scale
    refill(b, k.to(dtype), v.to(dtype))
    b.q = torch.ones_like(b.q)
    for size in (0, lb.lb_attn_kv4_workspace(1, nq, nq, 4, 1, D, n)):
        check_weighted(b, b.run(max_q=nq, max_len=n, workspace=torch.empty(size, dtype=torch.uint8, device="cuda")), b.want())


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("scale", [0.05, 0.5, 2.0])
def test_attention_prompt_scores_far_apart(dtype, D, scale):
    """Scores that differ by a few to hundreds of octaves, the maximum rising and lying far back."""
    b = Batch([900, 300], [120, 90], 6, 2, D, 16, dtype, seed=D)
    check_weighted(b, b.run(max_q=120, scale=scale), b.want(scale=scale), scale=scale)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 3, 2 ** 31 - 400, 2 ** 30])
@pytest.mark.parametrize("lens,nqs,Hq", [([5, 40, 3], [9, 1, 1], 8), ([5, 130, 70], [260, 3, 200], 4)])
def test_attention_largest_windows(lens, nqs, Hq, window, causal, dtype):
    """Windows up to the type's end, which hide nothing, with more queries than keys: a few and many."""
    b = Batch(lens, nqs, Hq, 2, 64, 16, dtype, seed=5)
    got, none = b.run(window=window, causal=causal, max_q=max(nqs)), b.run(causal=causal, max_q=max(nqs))
    b.check(got, b.want(causal=causal))
    assert torch.equal(got[0], none[0]) and torch.equal(got[1], none[1])


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("nq,Hq", [(1, 2), (5, 2), (60, 8)])
def test_attention_keys_next_to_two_to_the_31(nq, Hq, dtype):
    """The last key numbers that 32 bits hold, seen through a window: single tokens, some, a prompt's chunk."""
    page, D, window = 16, 64, 3000
    width = (2 ** 31 - 1040) // page                         # the widest table that is taken
    b = Batch([4096], [nq], Hq, 1, D, page, dtype, seed=3)    # its keys stand at the end of a sequence of n
    n, used = width * page, 4096 // page
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    table[:, width - used:] = b.table[:, :used]
    want, b.table, b.lens = b.want(window=window), table, [n]
    for max_len in (n, 4096):
        got = b.run(window=window, max_q=nq, max_len=max_len)
        b.lens = [4096]
        b.check(got, want)
        b.lens = [n]
    with pytest.raises(lb.LbError):
        b.table = torch.zeros(1, width + 1, dtype=torch.int32, device="cuda")
        b.run(window=window, max_q=nq)


# ---------------------------------------------------------------------------
# more rows, tokens and sequences than one launch holds (2^32 threads)
# ---------------------------------------------------------------------------

def test_linear_more_rows_than_a_launch_holds():
    M, N, K = 2 ** 28 + 100, 5, 16
    x = torch.randn(M, K, dtype=BF, device="cuda")
    g = gen(1)
    w, sw = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8), torch.rand(N, generator=g) + 0.1
    bias = torch.randn(N, generator=g).to(BF)
    out = torch.full((M, N), 7.0, dtype=BF, device="cuda")
    lb.lb_linear_w8a8(x, w.cuda(), sw.cuda(), out, bias=bias.cuda())
    rows = torch.cat([torch.arange(300), torch.tensor([2 ** 23 - 1, 2 ** 23, 2 ** 24, 2 ** 24 + 1, 2 ** 28 - 1, 2 ** 28]),
                      torch.randint(0, M, (3000,), generator=g), torch.arange(M - 300, M)]).cuda()
    q, sx = quant_ref(x[rows].cpu())
    check_linear(out[rows], *linear_want(q, w, sx, sw, bias), BF)


def test_cache_more_tokens_than_a_launch_holds():
    T, H, D, page = 16500, 32767, 64, 16
    if torch.cuda.mem_get_info()[0] < 170 * 2 ** 30:
        pytest.skip("needs 170 GiB")
    x = torch.empty(T, H, D, dtype=HF, device="cuda")
    ends = torch.tensor([0, 1, 8191, 8192, 8193, T - 2, T - 1]).cuda()
    x[ends] = torch.randn(len(ends), H, D, dtype=HF, device="cuda")
    slots = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    slots[ends] = torch.arange(len(ends)).cuda() * 2
    cache = empty_cache(1, H, page, D, HF)
    lb.lb_kv4_write(x, x, slots, *cache)
    small = empty_cache(1, H, page, D, HF)
    lb.lb_kv4_write(x[ends], x[ends], slots[ends], *small)
    for a, b in zip(cache, small):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    want = torch.empty(len(ends), H, D, dtype=HF, device="cuda")
    lb.lb_kv4_read(*small, slots[ends], want, torch.empty_like(want))
    back = torch.empty_like(x)
    lb.lb_kv4_read(*cache, slots, x, back)
    for got in (x, back):
        assert torch.equal(got[ends], want)
        assert not got[2:8191].any() and not got[8194:T - 2].any()


@pytest.mark.parametrize("max_q", [1, 256])
def test_attention_more_sequences_than_a_launch_holds(max_q):
    """2^24 tiles of rows and more; 61 different sequences over and over."""
    P, H, D = 61, 16, 64
    B = (2 ** 20 if max_q == 1 else 2 ** 19) + 77
    b = Batch([1 + i % 16 for i in range(P)], [1] * P, H, H, D, 16, BF, seed=2)
    want = b.want()
    of = torch.arange(B, device="cuda") % P
    q = b.q.cuda()[of].contiguous()
    out, lse = torch.full_like(q, 5.0), torch.full((B, H), 9.0, device="cuda")
    lens = torch.tensor(b.lens, dtype=torch.int32).cuda()[of].contiguous()
    lb.lb_attn_kv4(q, *b.cache, b.table[of].contiguous(), torch.arange(B + 1, dtype=torch.int32, device="cuda"), lens, out,
                   lse=lse, max_q=max_q, max_len=16)
    b.check((out[:P], lse[:P]), want)
    assert torch.equal(out, out[:P][of]) and torch.equal(lse, lse[:P][of])


# ---------------------------------------------------------------------------
# the cache at the end of its type
# ---------------------------------------------------------------------------

def quantise_at_the_end(x):
    """quantise_ref, with the scale that the cache takes where 15 scales above the minimum would be infinite."""
    u, scale, low = quantise_ref(x)
    top = (15 * scale.float() + low.float()).to(x.dtype)
    down = (scale.view(torch.int16) - 1).view(x.dtype)
    scale = torch.where(torch.isinf(top) & torch.isfinite(scale), down, scale)
    s, f = scale.float().numpy(), x.float().numpy()
    ok = (s > 0) & np.isfinite(s)
    return np.clip(np.rint(np.divide(f - low.float().numpy(), s, out=np.zeros_like(f), where=ok)), 0, 15), scale, low


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_cache_finite_numbers_stay_finite(dtype, D):
    """Vectors that reach the type's largest number, whose scale rounded up would stand for infinity."""
    T, H, page, most = 500, 2, 16, torch.finfo(dtype).max
    g = gen(D)
    # (a bf16 range beyond fp32 stands for NaN, as the header says)
    lo = (torch.rand(T, H, 1, generator=g, dtype=torch.float64) * (0.8 if dtype == BF else 1.6) - (0 if dtype == BF else 0.8)) * most
    lo[0] = 0
    x = lo + (most - lo) * torch.rand(T, H, D, generator=g, dtype=torch.float64)
    x[..., 3:4], x[..., 5] = lo, most
    x = x.to(dtype)
    assert torch.isfinite(x).all()
    cache, slots = empty_cache(T // page + 1, H, page, D, dtype), torch.arange(T).cuda()
    lb.lb_kv4_write(x.cuda(), x.flip(0).cuda(), slots, *cache)
    k, v = torch.empty(T, H, D, dtype=dtype, device="cuda"), torch.empty(T, H, D, dtype=dtype, device="cuda")
    lb.lb_kv4_read(*cache, slots, k, v)
    u, s, low = quantise_at_the_end(x)
    down = s != quantise_ref(x)[1]
    assert down.any() and not down.all()
    want = (torch.from_numpy(u) * s.float() + low.float()).to(dtype)
    assert torch.isfinite(want).all()
    assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), want.flip(0))
    # half a level, and a scale off by a step over 15 levels
    step = s.double() * torch.finfo(dtype).eps * 15
    off = (k.cpu().double() - x.double()).abs()
    assert (off <= s.double() / 2 + step + half_step(dtype) * x.double().abs()).all()


# ---------------------------------------------------------------------------
# the scaled product's large tiles
# ---------------------------------------------------------------------------

LARGE = [(4090, 4095, 528, 1, (256, 256)), (4096, 4096, 528, 1, (256, 256)),     # one round of them
         (4692, 8190, 1040, 2, (256, 256)), (4692, 8192, 1040, 2, (256, 256)),   # whole rounds, then the last rows
         (8190, 5038, 1040, 2, (256, 256)), (8190, 5036, 1040, 2, (256, 256)),   # whole rounds, then the last columns
         (2850, 4349, 48, 1, (192, 256)), (2850, 4348, 48, 1, (192, 256)),
         (4349, 2850, 48, 1, (256, 192)), (4349, 2852, 48, 1, (256, 192)),
         (4100, 4101, 48, 1, (64, 64)), (8192, 11005, 48, 1, (128, 128))]


@pytest.mark.parametrize("dtype", [BF, HF, FL])
@pytest.mark.parametrize("M,N,K,launches,tile", LARGE)
def test_scaled_product_large_tiles(M, N, K, launches, tile, dtype):
    """Every launch that the linear layer's rules give the scaled product, unforced, with bias and edges."""
    plan = lb.lb_auto_plan(lb.LB_PLAN_SCALED, M, N, K, 256)
    assert (plan["launches"], plan["tile_m"], plan["tile_n"]) == (launches, *tile)
    if torch.cuda.get_device_properties(0).multi_processor_count != 256:
        pytest.skip("planned for 256 compute units")
    g = gen(M + N)
    x = torch.randint(-128, 128, (M, K), generator=g, dtype=torch.int8).cuda()
    w = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8).cuda()
    sx, sw = (torch.rand(M, generator=g) * 1e-2).cuda(), (torch.rand(N, generator=g) * 1e-3).cuda()
    prod = torch.mm(x.double(), w.double().t().contiguous()) * sx.double()[:, None] * sw.double()
    for bias in (None, torch.randn(N, generator=g).to(dtype).cuda()):
        flat = torch.full((M * N + 64,), 7.0, dtype=dtype, device="cuda")
        lb.lb_gemm_s8_scaled(x, w, sx, sw, flat[:M * N].view(M, N), bias=bias)
        want = prod if bias is None else prod + bias.double()
        # as check_linear
        tol = (half_step(dtype) + 2 * STEP) * want.abs() + 5 * STEP * prod.abs()
        tol = tol * 1.001 + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
        assert ((flat[:M * N].view(M, N).double() - want).abs() <= tol).all()
        assert (flat[M * N:] == 7).all(), "write past out"


@pytest.mark.parametrize("dtype", [BF, HF, FL])
def test_linear_layer_in_two_launches(dtype):
    """The whole layer, rows quantised, by columns in two launches."""
    M, N, K = 8190, 5038, 1040
    assert lb.lb_auto_plan(lb.LB_PLAN_SCALED, M, N, K, 256)["launches"] == 2
    test_linear(dtype, M, N, K)


# ---------------------------------------------------------------------------
# scales, slots, lengths and offsets that start anywhere
# ---------------------------------------------------------------------------

def shifted(t, by=1):
    """The same values, `by` elements into an allocation, with NaN or the type's largest before and after."""
    far = float("nan") if t.is_floating_point() else torch.iinfo(t.dtype).max
    wide = torch.full((t.numel() + 16,), far, dtype=t.dtype, device="cuda")
    wide[by:by + t.numel()] = t.reshape(-1).cuda()
    return wide[by:by + t.numel()].view(t.shape)


@pytest.mark.parametrize("by", [1, 2, 3])
@pytest.mark.parametrize("M,N,K", [(5, 48, 64), (331, 4097, 272), (2850, 4349, 48), (4090, 4095, 528), (4692, 8190, 1040)])
def test_row_scales_start_anywhere(M, N, K, by):
    g = gen(M)
    x = torch.randint(-128, 128, (M, K), generator=g, dtype=torch.int8).cuda()
    w = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8).cuda()
    sx, sw = torch.rand(M, generator=g).cuda(), torch.rand(N, generator=g).cuda()
    want, got = (torch.empty(M, N, dtype=BF, device="cuda") for _ in range(2))
    lb.lb_gemm_s8_scaled(x, w, sx, sw, want)
    lb.lb_gemm_s8_scaled(x, w, shifted(sx, by), sw, got)
    assert torch.equal(got, want)
    f, q = torch.randn(M, K, generator=g).to(BF).cuda(), torch.empty_like(x)
    lb.lb_quant_rows_s8(f, q, sx)
    moved, again = shifted(sx, by), torch.empty_like(q)
    moved.zero_()
    lb.lb_quant_rows_s8(f, again, moved)
    assert torch.equal(q, again) and torch.equal(moved, sx)


@pytest.mark.parametrize("nq,n", [(1, 90), (1, 4000), (70, 300)])
def test_numbers_of_the_cache_start_anywhere(nq, n):
    b = Batch([n, 5], [nq, 3], 8, 2, 64, 16, BF, seed=nq)
    want = b.run(max_q=max(nq, 3))
    b.q_off, b.table = shifted(b.q_off), shifted(b.table.contiguous(), 3)
    lens = shifted(torch.tensor(b.lens, dtype=torch.int32), 1)
    q = b.q.cuda()
    out, lse = torch.empty_like(q), shifted(torch.empty(b.total, 8))
    lb.lb_attn_kv4(q, *b.cache, b.table, b.q_off, lens, out, lse=lse, max_q=max(nq, 3))
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    k, v = torch.empty(len(b.slots), 2, 64, dtype=BF, device="cuda"), torch.empty(len(b.slots), 2, 64, dtype=BF, device="cuda")
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    lb.lb_kv4_read(*b.cache, b.slots, k, v)
    lb.lb_kv4_read(*b.cache, shifted(b.slots), k2, v2)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    old = [t.clone() for t in b.cache]
    lb.lb_kv4_write(k, v, b.slots, *b.cache)
    mid = [t.clone() for t in b.cache]
    for t, o in zip(b.cache, old):
        t.copy_(o)
    lb.lb_kv4_write(k, v, shifted(b.slots), *b.cache)
    for t, o in zip(b.cache, mid):
        assert torch.equal(t.view(torch.uint8), o.view(torch.uint8))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("power", [-90, 90])
@pytest.mark.parametrize("nqs", [[1, 1], [5, 3], [120, 90]])
def test_attention_values_at_the_ends_of_their_range(D, power, nqs):
    b = Batch([900, 300], nqs, 6, 2, D, 16, BF, seed=D)
    for seq, n in enumerate(b.lens):
        refill(b, torch.randn(n, 2, D, generator=gen(seq)).to(BF), (torch.randn(n, 2, D, generator=gen(9)) * 2.0 ** power).to(BF), seq)
    check_weighted(b, b.run(max_q=max(nqs)), b.want())
