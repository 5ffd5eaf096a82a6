"""GPU tests of how many digits the decoder layer's 4-bit products keep before their output is rounded.

An output in 16 bits hides what was lost before it.  A bias that cancels all of an output but its rounding shows it (the
rows of x are equal, so that one bias cancels them all); where no bias does, outputs are held against the error that
their rounding alone has."""
import math

import pytest

torch = pytest.importorskip("torch")
import bit_integer_gemm_amd as lb  # noqa: E402
from test_gpu_layer import BF, HF, STEP, check_output, floor_of, gen, half_step, product_bound, weights  # noqa: E402

pytestmark = pytest.mark.gpu


# rows of each kernel: up to 16, and tiles of 64 x 128, 128 x 128 and 128 x 256
MINIMA = [(16, 200, 128), (17, 300, 128), (64, 257, 64), (130, 515, 32), (600, 9000, 128), (601, 8999, 32)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("M,N,group", MINIMA)
def test_minima_of_a_group(dtype, M, N, group):
    """Scales of zero leave the minima: b sum_k x, of one group here."""
    g = gen(M + N)
    x = (torch.rand(1, group, generator=g) + 1).to(dtype)
    b = torch.randn(N, 1, generator=g).to(dtype)
    p = torch.stack([torch.zeros_like(b), b], -1)
    w = torch.randint(0, 256, (N, group // 2), generator=g, dtype=torch.uint8)
    want = x.double().sum() * b.double().flatten()
    bias = (-want).to(dtype)
    out = torch.empty(M, N, dtype=dtype, device="cuda")
    lb.lb_linear_w4(x.cuda().expand(M, group).contiguous(), w.cuda(), p.cuda(), out, bias=bias.cuda())
    left = want + bias.double()
    # half steps: the sum of x, 7 additions of a lane and 4 between lanes; what three parts leave of x's sum and of b, and
    # the products that are not formed; the bias.  Whole ones: a product and its addition, of each of six parts.
    before = (11 + 4 + 1 + 2 * 2 * 6) * STEP * want.abs()
    tol = before + half_step(dtype) * (left.abs() + before) + floor_of(dtype)
    off = (out.cpu().double() - left).abs()
    assert (off <= tol).all(), (off / tol).max()


def roundings(x, u, s, b, group, wide):
    """Sum over all outputs of the expected squares of fp32's roundings: a whole step, evenly spread, of every partial sum
    as its kernel forms it: the minima of 16 groups ahead of their products (wide), or each group's own beside it."""
    xg, ug = x.unflatten(1, (-1, group)), (u + 16).unflatten(1, (-1, group))
    sums, acc, total = xg.sum(-1), torch.zeros(x.shape[0], u.shape[0], dtype=torch.float64), 0.0
    minima = b - 16 * s
    for g in range(sums.shape[1]):
        part = xg[:, g] @ ug[:, g].T * s[:, g]
        total += group / 16 * part.square().sum()
        if not wide:
            total += (acc + part).square().sum()
            acc = acc + sums[:, g, None] * minima[:, g]
        elif g % 16 == 0:
            acc = acc + sums[:, g:g + 16] @ minima[:, g:g + 16].T
            total += 6 * acc.square().sum()
        acc = acc + part
        total += acc.square().sum()
    return float(total) * (2 * STEP) ** 2 / 3


@pytest.mark.parametrize("mean", [0.0, 1.0, 10.0])
@pytest.mark.parametrize("M,N,K,group", [(16, 256, 4096, 128), (17, 256, 4096, 128), (64, 512, 4096, 128), (64, 256, 11008, 32),
                                         (130, 300, 2048, 64), (520, 1024, 4096, 64), (1030, 8200, 1024, 64)])
def test_activations_with_a_mean(M, N, K, group, mean):
    """fp16 outputs are hardly further from the formula than their rounding, whatever the mean of x: minima and products
    are large then, and cancel."""
    g = gen(K + M)
    x = (torch.randn(M, K, generator=g) + mean).to(HF)
    w, p, wd = weights((), N, K, group, HF, g)
    out = torch.empty(M, N, dtype=HF, device="cuda")
    lb.lb_linear_w4(x.cuda(), w.cuda(), p.cuda(), out)
    want = x.double() @ wd.T
    u = torch.stack([w & 15, w >> 4], -1).flatten(-2).double()
    some = slice(0, 256)   # of the columns, for the partial sums
    before = roundings(x.double(), u[some], p[some, :, 0].double(), p[some, :, 1].double(), group, M > 16) * N / min(N, 256)
    least = float((want.to(HF).double() - want).square().sum())
    got = float((out.cpu().double() - want).square().sum())
    # (two sums of squares of M N numbers, neither of which knows of the other)
    assert got <= (least + before) * (1 + 8 / math.sqrt(M * N)), (math.sqrt(got / least), math.sqrt(before / least))


@pytest.mark.parametrize("T", [1, 3, 7, 12, 20])
def test_between_the_experts_products(T):
    """What passes between an expert's products keeps fp32's digits: rows of the second one take the difference of two
    numbers that are nearly equal."""
    group, H, wide = 32, 64, 64
    I = group * wide
    g = gen(T)
    place = torch.randint(0, group, (wide,), generator=g) + torch.arange(wide) * group   # one number in each group, the rest zeros
    gate = (0.2 * (1 + 0.05 * torch.rand(wide, generator=g))).to(HF)
    lift = (0.025 * (1 + 0.1 * torch.rand(wide, generator=g))).to(HF)
    w1 = torch.zeros(1, 2 * I, H // 2, dtype=torch.uint8)
    p1 = torch.zeros(1, 2 * I, H // group, 2, dtype=HF)
    for rows, s in ((place, gate), (I + place, lift)):
        w1[0, rows] = 255
        p1[0, rows, :, 0] = s[:, None]
    a, u = 15 * gate.double(), 15 * lift.double()
    h = a / (1 + torch.exp(-a)) * u
    order = torch.sort(h).indices
    first, second = order[torch.arange(H) % (wide - 1)], order[torch.arange(H) % (wide - 1) + 1]
    p2 = torch.zeros(1, H, wide, 2, dtype=HF)
    p2[0, torch.arange(H), first, 0] = -1.0
    p2[0, torch.arange(H), second, 0] = 1.0
    w2 = torch.full((1, H, I // 2), 255, dtype=torch.uint8)
    x = torch.zeros(T, H, dtype=HF)
    x[torch.arange(T), torch.arange(T)] = 1.0
    out = torch.empty(T, H, dtype=HF, device="cuda")
    lb.lb_moe_w4(x.cuda(), torch.ones(1, H, dtype=HF, device="cuda"), w1.cuda(), p1.cuda(), w2.cuda(), p2.cuda(), out, top_k=1)
    want, both = 15 * (h[second] - h[first]), 15 * (h[second] + h[first])
    # of each number, in half steps: exponential 2, its sum, quotient and product 3, its parts 2; then of 31 and of 16 times
    # it, 15 of which are left: two whole steps of each in products, two in their scaling, and ten of 15 times it in joins
    before = (7 + (31 * 4 + 16 * 4 + 31 * 2) / 15 + 10) * STEP * both
    tol = before + half_step(HF) * (want.abs() + before) + floor_of(HF)
    off = (out.cpu().double() - want).abs()
    assert (off <= tol).all(), (off / tol).max()


@pytest.mark.parametrize("M", [3, 40, 300])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_largest_activations(M, group):
    """bf16 x of 2^116 in magnitude, whole groups of one sign and the largest levels: the sums stay in fp32's range."""
    N, K = 70, 512
    g = gen(M)
    sign = 1 - 2.0 * torch.randint(0, 2, (M, K // group), generator=g)
    x = (2.0 ** 116 * sign.repeat_interleave(group, 1)).to(BF)
    w = torch.full((N, K // 2), 255, dtype=torch.uint8)
    s = 2.0 ** -60 * (1 + torch.rand(N, K // group, generator=g))
    p = torch.stack([s, -7.5 * s], -1).to(BF)
    wd = (15 * p[..., 0].double() + p[..., 1].double()).repeat_interleave(group, 1)
    out = torch.empty(M, N, dtype=BF, device="cuda")
    lb.lb_linear_w4(x.cuda(), w.cuda(), p.cuda(), out)
    assert out.isfinite().all()
    check_output(out, x.double() @ wd.T, product_bound(x, p, K), BF)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("M", [2, 40])
def test_subnormal_activations(dtype, M):
    """Activations below the smallest normal number count as much as others."""
    K, N = 128, 40
    least = torch.finfo(dtype).smallest_normal
    x = torch.zeros(M, K, dtype=torch.float64)
    x[torch.arange(M), torch.arange(M)] = least * torch.linspace(0.25, 0.75, M, dtype=torch.float64)
    x = x.to(dtype)
    assert ((x.double() > 0).sum(1) == 1).all()
    w = torch.full((N, K // 2), 255, dtype=torch.uint8)
    p = torch.tensor([2.0 ** 7, 0.0], dtype=dtype).expand(N, 1, 2).contiguous()
    out = torch.empty(M, N, dtype=dtype, device="cuda")
    lb.lb_linear_w4(x.cuda(), w.cuda(), p.cuda(), out)
    want = 15 * 2.0 ** 7 * x.double().sum(1, keepdim=True).expand(M, N)
    tol = 64 * STEP * want * 3 + half_step(dtype) * want * (1 + 2 ** -12)   # (31 - 16 of them)
    assert ((out.cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("T", [1, 3, 7, 12])
def test_small_beside_large_between_the_products(T):
    """What passes between an expert's products may differ by 2^30 within the 256 numbers that share a power of two."""
    group, H, I = 32, 64, 512
    place = torch.arange(16) * 32 + 5
    size = 2.0 ** -(2.0 * torch.arange(16) % 32)   # of each line's eight: 1, 2^-2 .. 2^-14, and 2^-16 .. 2^-30
    size[8] = 1.0
    w1 = torch.zeros(1, 2 * I, H // 2, dtype=torch.uint8)
    p1 = torch.zeros(1, 2 * I, H // group, 2, dtype=BF)
    w1[0, place] = w1[0, I + place] = 255
    p1[0, place, :, 0] = 0.25
    p1[0, I + place, :, 0] = size[:, None].to(BF)
    gate = torch.tensor(15 * 0.25, dtype=torch.float64)
    h = gate / (1 + torch.exp(-gate)) * 15 * size.double()
    p2 = torch.zeros(1, H, I // group, 2, dtype=BF)
    n = torch.arange(H)
    p2[0, n, n % 16, 0] = 1.0
    w2 = torch.full((1, H, I // 2), 255, dtype=torch.uint8)
    x = torch.zeros(T, H, dtype=BF)
    x[torch.arange(T), torch.arange(T)] = 1.0
    out = torch.empty(T, H, dtype=BF, device="cuda")
    lb.lb_moe_w4(x.cuda(), torch.ones(1, H, dtype=BF, device="cuda"), w1.cuda(), p1.cuda(), w2.cuda(), p2.cuda(), out, top_k=1)
    want = 15 * h[n % 16]
    largest = h.view(2, 8).amax(1)[n % 16 // 8]
    # of the number itself as between nearly equal ones; its parts' last steps: 2^-39 of the largest, 31 and 16 times
    before = (7 + (31 * 4 + 16 * 4 + 31 * 2) / 15 + 10) * STEP * want + 47 * 2.0 ** -39 * largest
    tol = before + half_step(BF) * (want + before)
    off = (out.cpu().double() - want).abs()
    assert (off <= tol).all(), (off / tol).max()
    assert (before[n % 16 == 15] < want[n % 16 == 15] / 8).all()   # (the smallest says something)
