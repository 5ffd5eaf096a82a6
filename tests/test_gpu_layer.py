"""GPU tests of the decoder layer's other operators against plain implementations in 64 bits: norms with gate and
residual, rotary positions, the 4-bit linear layer, the mixture of experts.

Tolerances are derived: a 16-bit output is off by half a step of its type beside the fp32 steps counted where they
are used.  Where a worst-case count is far above what random roundings give, the 2-norm of the error is held as well:
half steps of the output bound it, and what fp32 adds is at most a sixteenth of that."""
import math

import pytest

torch = pytest.importorskip("torch")
import bit_integer_gemm_amd as lb  # noqa: E402

pytestmark = pytest.mark.gpu

BF, HF, FL = torch.bfloat16, torch.float16, torch.float32
STEP = 2.0 ** -24  # half a step of fp32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def floor_of(dtype):
    """Below the smallest normal number a rounding is off by half the smallest subnormal one."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def strided(x, pad, fill=float("nan")):
    """x on the GPU as the leading columns of wider rows."""
    flat = x.reshape(x.shape[0], -1)
    wide = torch.full((x.shape[0], flat.shape[1] + pad), fill, dtype=x.dtype, device="cuda")
    wide[:, :flat.shape[1]] = flat.cuda()
    return wide[:, :flat.shape[1]].unflatten(1, x.shape[1:]) if x.dim() > 2 else wide[:, :flat.shape[1]]


def guarded(shape, dtype, fill=7.0):
    """(tensor, check): a dense tensor with a margin behind it that has to stay as it is."""
    n = math.prod(shape)
    flat = torch.full((n + 256,), fill, dtype=dtype, device="cuda")
    return flat[:n].view(shape), lambda: (flat[n:] == fill).all().item()


# ---------------------------------------------------------------------------
# norms, gate and residual
# ---------------------------------------------------------------------------

EPS = 1e-5


def norm_ref(y, r, post_w, gate, w, alpha):
    """(r', x, what alpha gate z is) in float64."""
    z = torch.zeros(1, dtype=torch.float64)
    if y is not None:
        z = y.double()
        if post_w is not None:
            z = z / (z.square().mean(1, keepdim=True) + EPS).sqrt() * post_w.double()
        if gate is not None:
            z = z * gate.double()
        z = alpha * z
    out = z + (0 if r is None else r.double())
    return out, out / (out.square().mean(1, keepdim=True) + EPS).sqrt() * (1 if w is None else w.double()), z


def check_norm(got_r, got_x, ref, dtype, rtype, w):
    want_r, want_x, z = ref
    # a row's sum of squares: at most 32 products and additions of a thread, 6 between lanes, 16 between waves, and
    # the mean's, eps's, root's and quotient's roundings: 60 half steps at most, half of that in the root; four products
    dz = (30 + 8) * STEP * z.abs()
    dr = dz + STEP * want_r.abs()
    if got_r is not None:
        tol = dr + half_step(rtype) * (want_r.abs() + dr) + floor_of(rtype)
        assert ((got_r.cpu().double() - want_r).abs() <= tol).all()
    if got_x is not None:
        n = want_r.shape[1]
        inv = 1 / (want_r.square().mean(1, keepdim=True) + EPS).sqrt()
        # r' off by dr moves the root mean square by at most dr's own, and x with it
        dx = dr * inv * w.double().abs() + want_x.abs() * (38 * STEP + (dr.square().sum(1, keepdim=True) / n).sqrt() * inv)
        tol = dx + half_step(dtype) * (want_x.abs() + dx) + floor_of(dtype)
        assert ((got_x.cpu().double() - want_x).abs() <= tol).all()


@pytest.mark.parametrize("dtype,rtype", [(BF, BF), (BF, FL), (HF, HF), (HF, FL), (FL, FL)])
@pytest.mark.parametrize("M,H", [(1, 8), (3, 520), (2, 4096), (5, 8200), (3, 16392), (2, 32768), (700, 136)])
def test_residual_norm(dtype, rtype, M, H):
    g = gen(M + H)
    y = (torch.randn(M, H, generator=g) * (1 + 20 * (torch.rand(H, generator=g) < 0.02))).to(dtype)
    r = (3 * torch.randn(M, H, generator=g)).to(rtype)
    w, wp = ((1 + 0.2 * torch.randn(H, generator=g)).to(dtype) for _ in "ab")
    row, token = torch.randn(H, generator=g).to(dtype), torch.randn(M, H, generator=g).to(dtype)
    if M > 2:
        y[1] = 0
        r[1] = 0   # a row of nothing
    for post, gate, alpha in ((None, None, 1.0), (wp, row, 0.5), (wp, token, 1.0), (None, token, -2.0), (wp, None, 1.0)):
        ro, r_kept = guarded((M, H), rtype)
        xo, x_kept = guarded((M, H), dtype)
        lb.lb_residual_norm(strided(y, 16), strided(r, 8), ro, xo, w=w.cuda(), post_w=None if post is None else post.cuda(),
                            gate=None if gate is None else row.cuda() if gate is row else strided(token, 24), alpha=alpha,
                            eps=EPS)
        check_norm(ro, xo, norm_ref(y, r, post, gate, w, alpha), dtype, rtype, w)
        assert r_kept() and x_kept(), "write past the rows"


@pytest.mark.parametrize("dtype", [BF, FL])
def test_residual_norm_parts_left_out(dtype):
    """Only the norm, only the residual, no residual before; in place."""
    g = gen(5)
    M, H = 6, 1032
    y, r = torch.randn(M, H, generator=g).to(dtype), torch.randn(M, H, generator=g)
    w, wp = ((1 + 0.2 * torch.randn(H, generator=g)).to(dtype) for _ in "ab")
    x = torch.empty(M, H, dtype=dtype, device="cuda")
    lb.lb_residual_norm(None, r.cuda(), None, x, w=w.cuda(), eps=EPS)
    check_norm(None, x, norm_ref(None, r, None, None, w, 1.0), dtype, FL, w)
    ro = torch.empty(M, H, device="cuda")
    lb.lb_residual_norm(y.cuda(), r.cuda(), ro, None, post_w=wp.cuda(), alpha=0.25, eps=EPS)
    check_norm(ro, None, norm_ref(y, r, wp, None, None, 0.25), dtype, FL, None)
    lb.lb_residual_norm(y.cuda(), None, ro, x, w=w.cuda(), post_w=wp.cuda(), eps=EPS)
    check_norm(ro, x, norm_ref(y, None, wp, None, w, 1.0), dtype, FL, w)
    yy, rr = strided(y, 8), strided(r, 8)
    lb.lb_residual_norm(yy, rr, rr, yy, w=w.cuda(), post_w=wp.cuda(), eps=EPS)
    check_norm(rr, yy, norm_ref(y, r, wp, None, w, 1.0), dtype, FL, w)


def test_residual_norm_not_finite():
    """A row that holds an infinity or a NaN spoils itself and no other."""
    y = torch.randn(4, 64).to(BF)
    y[1, 3], y[2, 5] = float("inf"), float("nan")
    r, w = torch.randn(4, 64), torch.ones(64, dtype=BF)
    ro, x = torch.empty(4, 64, device="cuda"), torch.empty(4, 64, dtype=BF, device="cuda")
    lb.lb_residual_norm(y.cuda(), r.cuda(), ro, x, w=w.cuda(), eps=EPS)
    assert x[1].isnan().any() and x[2].isnan().all()
    keep = [0, 3]
    check_norm(ro[keep], x[keep], norm_ref(y[keep], r[keep], None, None, w, 1.0), BF, FL, w)


def test_residual_norm_refuses():
    y, r = torch.zeros(2, 64, dtype=BF, device="cuda"), torch.zeros(2, 64, device="cuda")
    w = torch.zeros(64, dtype=BF, device="cuda")
    with pytest.raises(TypeError):
        lb.lb_residual_norm(y, r.half(), r.half(), y, w=w)
    with pytest.raises(TypeError):
        lb.lb_residual_norm(y, r, r, y, w=w.float())
    with pytest.raises(ValueError):
        lb.lb_residual_norm(y, r[:1], r, y, w=w)
    with pytest.raises(ValueError):
        lb.lb_residual_norm(y, r, r, y, w=w, gate=w[:32])
    with pytest.raises(lb.LbError, match="null"):
        lb.lb_residual_norm(y, r, r, y)


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------

def rope_ref(x, pos, freqs, layout, mult):
    """(turned, |a| + |b| of each number's pair) in float64."""
    R = 2 * freqs.numel()
    angle = (pos.double()[:, None] * freqs)[:, None]
    c, s = angle.cos() * mult, angle.sin() * mult
    y = x.double().clone()
    size = torch.zeros_like(y)
    i = torch.arange(R // 2)
    a, b = (i, i + R // 2) if layout == "half" else (2 * i, 2 * i + 1)
    y[..., a], y[..., b] = x.double()[..., a] * c - x.double()[..., b] * s, x.double()[..., b] * c + x.double()[..., a] * s
    size[..., a] = size[..., b] = x.double()[..., a].abs() + x.double()[..., b].abs()
    return y, size


def check_rope(got, x, pos, freqs, layout, mult):
    want, size = rope_ref(x, pos, freqs, layout, mult)
    # the angle in turns: three fp64 half steps of it, and fp32's of a fraction below a half (2^-26 turns); sine and
    # cosine within 2 units (2^-23 each), mult's product, the pair's products and their sum
    angle = 3 * 2.0 ** -53 * float(pos.double().abs().max()) * float(freqs.max()) + 2 * math.pi * 2.0 ** -26
    tol = (angle + 2 * 2.0 ** -23 + 4 * STEP) * mult * size
    tol = tol + half_step(x.dtype) * (want.abs() + tol) * (size > 0) + floor_of(x.dtype)
    assert ((got.cpu().double() - want).abs() <= tol).all()


ROPE_SIZES = [(1, 1, 1, 16, 16), (1, 32, 8, 128, 128), (5, 32, 8, 128, 32), (3, 5, 1, 256, 256), (70, 4, 2, 64, 32),
              (1100, 3, 1, 64, 64), (1025, 2, 2, 80, 16), (2, 1, 0, 512, 256)]


@pytest.mark.parametrize("dtype", [BF, HF, FL])
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("T,Hq,Hk,D,R", ROPE_SIZES)
def test_rope(dtype, layout, T, Hq, Hk, D, R):
    g = gen(T + D)
    x = torch.randn(T, Hq + 2 * Hk, D, generator=g).to(dtype)
    pos = torch.randint(0, 3000, (T,), generator=g)
    pos[0], pos[T // 2] = 200003, -17
    freqs, mult = lb.lb_rope_freqs(R, scaling="parts", factor=8.0, before=4096.0)
    dev = x.cuda()
    q, k = dev[:, :Hq], dev[:, Hq:Hq + Hk] if Hk else None
    qo, q_kept = guarded((T, Hq, D), dtype)
    ko, k_kept = guarded((T, Hk, D), dtype)
    lb.lb_rope(q, k, pos.cuda(), freqs, qo, ko if Hk else None, layout=layout, mult=mult)
    check_rope(qo, x[:, :Hq], pos, freqs.cpu(), layout, mult)
    if Hk:
        check_rope(ko, x[:, Hq:Hq + Hk], pos, freqs.cpu(), layout, mult)
    assert q_kept() and k_kept(), "write past the heads"
    # in place, in the rows where queries, keys and values lie: the same numbers, and the values left alone
    lb.lb_rope(q, k, pos.cuda(), freqs, q, k, layout=layout, mult=mult)
    assert torch.equal(q, qo) and (not Hk or (torch.equal(k, ko) and torch.equal(dev[:, Hq + Hk:].cpu(), x[:, Hq + Hk:])))


def test_rope_far_positions():
    """Angles of far positions: 2^40 is off by 2^-13 of a turn in fp64 products, and not at all here for powers of two."""
    x = torch.randn(3, 2, 32, generator=gen(1))
    pos = torch.tensor([2 ** 31, 2 ** 31 - 1, 10 ** 7])
    freqs = torch.tensor([1.0, 0.5, 0.1, 1e-3] * 4, dtype=torch.float64)
    out = torch.empty(3, 2, 32, device="cuda")
    lb.lb_rope(x.cuda(), None, pos.cuda(), freqs.cuda(), out, None)
    check_rope(out, x, pos, freqs, "half", 1.0)


def test_rope_refuses():
    q = torch.zeros(2, 4, 64, dtype=BF, device="cuda")
    pos, f = torch.zeros(2, dtype=torch.int64, device="cuda"), torch.zeros(32, dtype=torch.float64, device="cuda")
    with pytest.raises(TypeError):
        lb.lb_rope(q, q, pos.int(), f, q, q)
    with pytest.raises(TypeError):
        lb.lb_rope(q, q, pos, f.float(), q, q)
    with pytest.raises(ValueError):
        lb.lb_rope(q, q, pos[:1], f, q, q)
    with pytest.raises(lb.LbError):
        lb.lb_rope(q, q, pos, torch.zeros(40, dtype=torch.float64, device="cuda"), q, q)
    with pytest.raises(lb.LbError):
        lb.lb_rope(q, q, pos, f[:12], q, q)


# ---------------------------------------------------------------------------
# linear layer with 4-bit weights
# ---------------------------------------------------------------------------

def weights(lead, N, K, group, dtype, g):
    """(packed, numbers of the groups, weights in float64)"""
    u = torch.randint(0, 16, (*lead, N, K), generator=g, dtype=torch.uint8)
    s = torch.randn(*lead, N, K // group, generator=g).mul(0.2).exp() / (4.6 * math.sqrt(K))
    p = torch.stack([s, s * (torch.randn(s.shape, generator=g) * 0.4 - 7.5)], -1).to(dtype)
    d = p.double()
    w = (u.unflatten(-1, (K // group, group)).double() * d[..., :1] + d[..., 1:]).flatten(-2)
    return u[..., 0::2] | (u[..., 1::2] << 4), p, w


def sizes_of(p, K):
    """The largest magnitude of a group's terms: s (16 + 15) beside |b - 16 s|, for each weight."""
    d = p.double()
    return (31 * d[..., 0].abs() + (d[..., 1] - 16 * d[..., 0]).abs()).repeat_interleave(K // p.shape[-2], -1)


def product_bound(x, p, K):
    """Off by at most, before the output's rounding: a group's sums come from at most 4 matrix instructions of 8
    rounded steps (whole steps, should they cut); two FMAs a group, the waves' join and the bias, half a step each."""
    return (2 * 32 + 2 * p.shape[-2] + 20) * STEP * (x.double().abs() @ sizes_of(p, K).T)


def check_output(got, want, before, dtype):
    tol = before + half_step(dtype) * (want.abs() + before) + floor_of(dtype)
    off = (got.cpu().double() - want).abs()
    assert (off <= tol).all(), (off / tol).max()
    if want.norm() > 0:
        rel = float(off.norm() / want.norm())
        assert rel <= half_step(dtype) * (1 + 2 ** -4) + float(floor_of(dtype) * math.sqrt(want.numel()) / want.norm()), rel


LINEAR = [(1, 1, 32, 32), (1, 16, 128, 128), (1, 4096, 512, 64), (1, 333, 4096, 128), (2, 33, 288, 32), (3, 100, 5504, 32),
          (4, 47, 2048, 128), (8, 640, 1088, 64), (9, 31, 11008, 128), (15, 65, 960, 64), (16, 257, 4096, 128), (17, 96, 512, 128),
          (31, 1000, 256, 32), (33, 65, 1152, 128), (61, 129, 5504, 32), (64, 200, 384, 64), (65, 70, 640, 128),
          (130, 515, 1024, 64), (331, 200, 2048, 128), (700, 1025, 544, 32), (513, 260, 4096, 128)]


# tiles of each size with whole and odd ends, whole rounds beside a rest of columns, rows in parts of a long K
LINEAR_WIDE = [(600, 9000, 256, 128), (601, 8999, 160, 32), (1030, 8193, 128, 64), (1030, 8200, 320, 64), (1000, 4001, 2048, 128),
               (1000, 4000, 1952, 32), (3000, 2816, 256, 32), (40, 300, 8192, 128), (1, 40, 65536, 128), (2, 5, 131072, 32),
               (16, 130, 11008, 64), (14, 20000, 96, 32), (1, 70000, 64, 64),
               (1, 20480, 1024, 128), (9, 20480, 1024, 32), (2, 32768, 640, 128)]   # (weights that fill an allocation of whole pages to its end)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("M,N,K,group", LINEAR + LINEAR_WIDE)
def test_linear_w4(dtype, M, N, K, group):
    g = gen(M * 3 + N)
    x = (torch.randn(M, K, generator=g) * (1 + 20 * (torch.rand(K, generator=g) < 0.02))).to(dtype)
    w, p, wd = weights((), N, K, group, dtype, g)
    bias = torch.randn(N, generator=g).to(dtype) if (M + N) % 2 else None
    out, kept = guarded((M, N), dtype)
    lb.lb_linear_w4(strided(x, 8, float("inf")), w.cuda(), p.cuda(), out, bias=None if bias is None else bias.cuda())
    want = x.double() @ wd.T
    if bias is not None:
        want = want + bias.double()
    check_output(out, want, product_bound(x, p, K), dtype)
    assert kept(), "write past out"


@pytest.mark.parametrize("M", [1, 5, 40, 300])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_linear_w4_places(M, dtype):
    """One activation at a time: its weight comes back exactly, whatever its place in the line."""
    K, N, group = 544, 50, 32
    g = gen(M)
    w, p, _ = weights((), N, K, group, dtype, g)
    p = torch.stack([torch.ones(N, K // group), torch.arange(N * (K // group)).view(N, -1) % 7 - 8.0], -1).to(dtype)
    lev = torch.stack([w & 15, w >> 4], -1).flatten(-2).double() + p[..., 1].double().repeat_interleave(group, 1)
    k = torch.randperm(K, generator=g)[:M]
    x = torch.zeros(M, K, dtype=dtype)
    x[torch.arange(M), k] = 2.0
    out = torch.empty(M, N, dtype=dtype, device="cuda")
    lb.lb_linear_w4(x.cuda(), w.cuda(), p.cuda(), out)
    assert torch.equal(out.cpu().double(), 2 * lev[:, k].T)


@pytest.mark.parametrize("M", [1, 20, 200])
def test_linear_w4_not_finite(M):
    """Rows of x that are not finite spoil themselves and no other; nothing finite comes out of them."""
    g = gen(3)
    K, N = 512, 40
    w, p, wd = weights((), N, K, 128, BF, g)
    x = torch.randn(M + 2, K, generator=g).to(BF)
    x[0, 100], x[M + 1, 511] = float("nan"), float("inf")
    out = torch.empty(M + 2, N, dtype=BF, device="cuda")
    lb.lb_linear_w4(x.cuda(), w.cuda(), p.cuda(), out)
    assert out[0].isnan().all() and not out[M + 1].isfinite().any()
    check_output(out[1:M + 1], x[1:M + 1].double() @ wd.T, product_bound(x[1:M + 1], p, K), BF)


def test_linear_w4_signed_levels():
    """A scale alone: levels -8..7 as u = level + 8 with the minimum -8 s, exact."""
    g = gen(4)
    lev = torch.randint(-8, 8, (48, 256), generator=g)
    s = torch.randn(48, 2, generator=g).abs().to(HF)
    w = lev.add(8).to(torch.uint8)
    x = torch.randint(-3, 4, (7, 256), generator=g).to(HF)
    out = torch.empty(7, 48, dtype=HF, device="cuda")
    p = torch.stack([s, -8 * s], -1)
    lb.lb_linear_w4(x.cuda(), (w[:, 0::2] | (w[:, 1::2] << 4)).cuda(), p.cuda(), out)
    want = x.double() @ (lev.double() * s.double().repeat_interleave(128, 1)).T
    check_output(out, want, product_bound(x, p, 256), HF)


def test_linear_w4_refuses():
    x, out = torch.zeros(2, 256, dtype=BF, device="cuda"), torch.zeros(2, 8, dtype=BF, device="cuda")
    w, p = torch.zeros(8, 128, dtype=torch.uint8, device="cuda"), torch.zeros(8, 2, 2, dtype=BF, device="cuda")
    with pytest.raises(TypeError):
        lb.lb_linear_w4(x, w, p.half(), out)
    with pytest.raises(ValueError):
        lb.lb_linear_w4(x, w[:, :64], p, out)
    with pytest.raises(lb.LbError):
        lb.lb_linear_w4(x, w, torch.zeros(8, 16, 2, dtype=BF, device="cuda"), out)
    with pytest.raises(ValueError):
        lb.lb_linear_w4(x, w, p, out.t().contiguous().t())


# ---------------------------------------------------------------------------
# mixture of experts
# ---------------------------------------------------------------------------

def experts(E, H, I, group, dtype, g):
    wr = torch.randn(E, H, generator=g).div(math.sqrt(H)).mul(2).to(dtype)
    return wr, weights((E,), 2 * I, H, group, dtype, g), weights((E,), H, I, group, dtype, g)


def moe_ref(x, wr, up, down, k, renorm, scale):
    """(out, ids, weights, sure, bound): in float64; sure: tokens whose choice fp32 logits cannot change; bound: how
    far out may be off before its rounding."""
    _, p1, w1 = up
    _, p2, w2 = down
    T, H = x.shape
    E, I = wr.shape[0], w1.shape[1] // 2
    xd = x.double()
    logits = xd @ wr.double().T
    # products of 32 terms in order, 8 rounded steps each, and the waves' join
    dl = (2 * 8 * 4 + 2 * H / 32 + 20) * STEP * (xd.abs() @ wr.double().abs().T)
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    ids = order.indices[:, :k]
    top = order.values[:, :min(k + 1, E)]
    sure = (top[:, :-1] - top[:, 1:] > 2 * dl.max()).all(1) if top.shape[1] > 1 else torch.ones(T, dtype=torch.bool)
    p = torch.softmax(logits, 1).gather(1, ids)
    if renorm:
        p = p / p.sum(1, keepdim=True)
    p = p * scale
    out, bound = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    # p's exponentials and sums: the logits' errors twice, and some twenty half steps
    dp = 2 * dl.max(1, keepdim=True).values + (E + 40) * STEP
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        du = product_bound(x[t], p1[e], H)
        u = xd[t] @ w1[e].T
        gate, lift = u[:, :I], u[:, I:]
        s = gate * torch.sigmoid(gate)
        h = s * lift
        # silu's slope is below 1.1; exponential, quotient and product: 2^-20; two bf16 parts: 2^-17
        dh = 1.1 * du[:, :I] * (lift.abs() + du[:, I:]) + s.abs() * du[:, I:] + h.abs() * (2 ** -17 + 2 ** -20)
        y = h @ w2[e].T
        dy = dh @ w2[e].abs().T + product_bound(h, p2[e], I)
        pj = p[t, j][:, None]
        out[t] += pj * y
        bound[t] += pj * (dy + y.abs() * (dp[t] + 4 * STEP + k * STEP))
    return out, ids, p, sure, dp, bound


MOE = [(1, 1, 1, 32, 32, 32), (1, 8, 2, 256, 320, 64), (1, 128, 8, 512, 128, 128), (2, 4, 4, 1024, 32, 32),
       (5, 64, 6, 288, 416, 32), (16, 8, 2, 512, 256, 128), (17, 16, 1, 640, 192, 64), (33, 60, 7, 256, 128, 128),
       (64, 8, 3, 384, 384, 128), (64, 200, 2, 128, 64, 64), (150, 16, 4, 256, 64, 32), (3, 1000, 64, 64, 32, 32)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,E,k,H,I,group", MOE)
def test_moe_w4(dtype, T, E, k, H, I, group):
    g = gen(T + E + H)
    x = torch.randn(T, H, generator=g).to(dtype)
    wr, up, down = experts(E, H, I, group, dtype, g)
    renorm, scale = bool((T + E) % 2), 1.0 if T % 3 else 2.5
    want, ids, p, sure, dp, bound = moe_ref(x, wr, up, down, k, renorm, scale)
    out, kept = guarded((T, H), dtype)
    got_ids, got_p = torch.full((T, k), -1, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    args = [a.cuda() for a in (wr, up[0], up[1], down[0], down[1])]
    lb.lb_moe_w4(strided(x, 8), *args, out, top_k=k, renorm=renorm, scale=scale, ids=got_ids, weights=got_p)
    assert sure.double().mean() > 0.5, "the inputs say nothing"
    assert torch.equal(got_ids.cpu().long()[sure], ids[sure])
    assert ((got_p.cpu().double() - p).abs()[sure] <= (dp * p)[sure] * 1.01).all()
    check_output(out[sure.cuda()], want[sure], bound[sure], dtype)
    assert kept(), "write past out"
    again = torch.empty_like(out)   # without ids and weights: the same bits
    lb.lb_moe_w4(x.cuda(), *args, again, top_k=k, renorm=renorm, scale=scale)
    assert torch.equal(out, again)


def test_moe_w4_ties():
    """Equal logits: the lowest expert first, whatever their number."""
    g = gen(9)
    wr, up, down = experts(12, 64, 32, 32, BF, g)
    wr[:] = wr[0]
    x = torch.randn(4, 64, generator=g).to(BF)
    ids = torch.empty(4, 5, dtype=torch.int32, device="cuda")
    out = torch.empty(4, 64, dtype=BF, device="cuda")
    lb.lb_moe_w4(x.cuda(), *(a.cuda() for a in (wr, up[0], up[1], down[0], down[1])), out, top_k=5, ids=ids)
    assert (ids.cpu() == torch.arange(5)).all()
    want, _, _, _, _, bound = moe_ref(x, wr, up, down, 5, False, 1.0)
    check_output(out, want, bound, BF)


@pytest.mark.parametrize("T,E", [(4, 64), (20, 8)])
def test_moe_w4_not_finite(T, E):
    """Tokens that are not finite spoil themselves and no other."""
    g = gen(T)
    wr, up, down = experts(E, 128, 64, 64, HF, g)
    x = torch.randn(T, 128, generator=g).to(HF)
    x[1, 5], x[T - 1, 7] = float("nan"), float("inf")
    out = torch.empty(T, 128, dtype=HF, device="cuda")
    ids = torch.empty(T, 3, dtype=torch.int32, device="cuda")
    lb.lb_moe_w4(x.cuda(), *(a.cuda() for a in (wr, up[0], up[1], down[0], down[1])), out, top_k=3, ids=ids)
    assert out[1].isnan().all() and not out[T - 1].isfinite().all()
    assert ((ids >= 0) & (ids < E)).all() and all(len(set(r)) == 3 for r in ids.tolist())
    keep = [t for t in range(T) if t not in (1, T - 1)]
    want, _, _, sure, _, bound = moe_ref(x[keep], wr, up, down, 3, False, 1.0)
    assert sure.all()
    check_output(out[keep], want, bound, HF)


def test_moe_w4_refuses():
    g = gen(1)
    wr, up, down = experts(4, 64, 32, 32, BF, g)
    args = [a.cuda() for a in (wr, up[0], up[1], down[0], down[1])]
    x, out = torch.zeros(2, 64, dtype=BF, device="cuda"), torch.empty(2, 64, dtype=BF, device="cuda")
    for k in (0, 5):
        with pytest.raises(lb.LbError):
            lb.lb_moe_w4(x, *args, out, top_k=k)
    with pytest.raises(lb.LbError, match="workspace"):
        lb.lb_moe_w4(x, *args, out, top_k=2, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        lb.lb_moe_w4(x, *args, out, top_k=2, ids=torch.empty(2, 3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="workspace"):
        lb.lb_moe_w4(x, *args, out, top_k=2, stream=torch.cuda.Stream())


# ---------------------------------------------------------------------------
# streams and graphs
# ---------------------------------------------------------------------------

def calls(seed):
    """(name, inputs that change, call, outputs) of each operator."""
    g = gen(seed)
    x = torch.randn(6, 256, generator=g).to(BF).cuda()
    big = torch.randn(300, 256, generator=g).to(BF).cuda()
    w, p, _ = weights((), 96, 256, 64, BF, g)
    w, p = w.cuda(), p.cuda()
    wr, up, down = experts(16, 256, 128, 64, BF, g)
    moe = [a.cuda() for a in (wr, up[0], up[1], down[0], down[1])]
    one, norm_w = torch.empty(6, 96, dtype=BF, device="cuda"), torch.ones(256, dtype=BF, device="cuda")
    many = torch.empty(300, 96, dtype=BF, device="cuda")
    ws = [torch.empty(max(n, 1), dtype=torch.uint8, device="cuda") for n in
          (lb.lb_linear_w4_workspace(6, 256, 96, 64), lb.lb_linear_w4_workspace(300, 256, 96, 64),
           lb.lb_moe_w4_workspace(6, 256, 128, 16, 4))]
    mixed, normed, res = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    freqs, _ = lb.lb_rope_freqs(64)
    pos = torch.arange(6, device="cuda")
    turned = torch.empty(6, 4, 64, dtype=BF, device="cuda")
    return [
        ("linear", x, lambda s: lb.lb_linear_w4(x, w, p, one, workspace=ws[0], stream=s), [one]),
        ("linear rows", big, lambda s: lb.lb_linear_w4(big, w, p, many, workspace=ws[1], stream=s), [many]),
        ("moe", x, lambda s: lb.lb_moe_w4(x, *moe, mixed, top_k=4, workspace=ws[2], stream=s), [mixed]),
        ("norm", x, lambda s: lb.lb_residual_norm(x, x, res, normed, w=norm_w, post_w=norm_w, stream=s), [res, normed]),
        ("rope", x, lambda s: lb.lb_rope(x.view(6, 4, 64), None, pos, freqs, turned, None, stream=s), [turned]),
    ]


@pytest.mark.parametrize("which", range(5))
def test_streams_and_graphs(which):
    """On a stream of its own, and captured and replayed with other inputs: what the eager call gives."""
    name, x, call, outs = calls(which)[which]
    first = x.clone()
    want = []
    for i in range(4):
        x.copy_(first * (1 + i))
        call(None)
        want.append([o.clone() for o in outs])
    side = torch.cuda.Stream()
    x.copy_(first)
    for o in outs:
        o.zero_()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(o, w) for o, w in zip(outs, want[0])), name
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(None)
    for i in range(4):
        x.copy_(first * (1 + i))
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want[i])), (name, i)


def test_graphs_share_a_workspace():
    """Two graphs of one workspace, replayed in turn: what the eager calls give."""
    g = gen(11)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    made = []
    for T, M in ((1, 40), (9, 300)):
        x = torch.randn(T, 256, generator=g).to(BF).cuda()
        big = torch.randn(M, 512, generator=g).to(BF).cuda()
        w, p, _ = weights((), 200, 512, 64, BF, g)
        w, p = w.cuda(), p.cuda()
        wr, up, down = experts(16, 256, 128, 64, BF, g)
        moe = [a.cuda() for a in (wr, up[0], up[1], down[0], down[1])]
        out, many = torch.empty_like(x), torch.empty(M, 200, dtype=BF, device="cuda")

        def call(x=x, moe=moe, out=out, big=big, w=w, p=p, many=many):
            lb.lb_moe_w4(x, *moe, out, top_k=3, workspace=ws)
            lb.lb_linear_w4(big, w, p, many, workspace=ws)

        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        made.append((x, big, out, many, call, graph))
    for i in range(4):
        want = []
        for x, big, out, many, call, _ in made:
            x.mul_(-1.5)
            big.add_(0.25)
            call()
            want.append((out.clone(), many.clone()))
            out.zero_()
            many.zero_()
        for *_, graph in made:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w[0]) and torch.equal(m, w[1]) for (_, _, o, m, _, _), w in zip(made, want)), i


def test_two_streams_at_once():
    """The same weights used on two streams, each with a workspace of its own."""
    g = gen(12)
    wr, up, down = experts(32, 512, 256, 64, BF, g)
    moe = [a.cuda() for a in (wr, up[0], up[1], down[0], down[1])]
    xs = [torch.randn(n, 512, generator=g).to(BF).cuda() for n in (7, 40)]
    want = []
    for x in xs:
        out = torch.empty_like(x)
        lb.lb_moe_w4(x, *moe, out, top_k=4)
        want.append(out)
    streams = [torch.cuda.Stream() for _ in xs]
    ws = [torch.empty(lb.lb_moe_w4_workspace(x.shape[0], 512, 256, 32, 4), dtype=torch.uint8, device="cuda") for x in xs]
    outs = [torch.empty_like(x) for x in xs]
    torch.cuda.synchronize()
    for _ in range(10):
        for x, o, w, s in zip(xs, outs, ws, streams):
            lb.lb_moe_w4(x, *moe, o, top_k=4, workspace=w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
