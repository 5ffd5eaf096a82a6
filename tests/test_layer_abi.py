"""CPU tests of the C boundary of the decoder layer's other operators (norms with the residual, rotary positions,
4-bit linear layer, mixture of experts): refusals before any HIP call, workspaces, frequencies, the binding's own
checks.  Nothing is launched here."""
import ctypes
import math

import numpy as np
import pytest

import bit_integer_gemm_amd as lb
from test_serving_abi import NULL, ODD, P, Args, refusals


@pytest.fixture(scope="module")
def lib():
    from bit_integer_gemm_amd import _build
    _build.ensure_built()
    return lb.load()


def test_header_limits_match_binding():
    import os
    import re
    text = open(os.path.join(os.path.dirname(lb.__file__), "..", "include", "lb_gemm.h")).read()
    for name, value in (("LB_W4_K_MAX", lb.W4_K_MAX), ("LB_NORM_H_MAX", lb.NORM_H_MAX),
                        ("LB_MOE_EXPERTS_MAX", lb.MOE_EXPERTS_MAX), ("LB_MOE_TOP_MAX", lb.MOE_TOP_MAX)):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == value


def test_residual_norm_refusals(lib):
    a = Args(Y=P, ldy=64, R=P, ldr=64, post_w=P, gate=P, ldg=0, w=P, R_out=P, ldro=64, X=P, ldx=64, M=3, H=64,
             alpha=1.0, eps=1e-5, ftype=lb.LB_BF16, rtype=lb.LB_F32, stream=NULL)
    refusals(lib.lb_residual_norm, a, [
        (lb.LB_ERR_NULL, dict(Y=NULL, R=NULL)), (lb.LB_ERR_NULL, dict(R_out=NULL, X=NULL)), (lb.LB_ERR_NULL, dict(w=NULL)),
        (lb.LB_ERR_NULL, dict(Y=NULL)), (lb.LB_ERR_NULL, dict(Y=NULL, post_w=NULL)),
        (lb.LB_ERR_SHAPE, dict(M=0)), (lb.LB_ERR_SHAPE, dict(M=2 ** 31)), (lb.LB_ERR_SHAPE, dict(H=0)),
        (lb.LB_ERR_SHAPE, dict(ldy=63)), (lb.LB_ERR_SHAPE, dict(ldr=8)), (lb.LB_ERR_SHAPE, dict(ldg=8)),
        (lb.LB_ERR_SHAPE, dict(ldro=8)), (lb.LB_ERR_SHAPE, dict(ldx=8)),
        (lb.LB_ERR_SHAPE, dict(ldro=72)), (lb.LB_ERR_SHAPE, dict(ldx=72)),   # in place, with another stride
        (lb.LB_ERR_ALIGN, dict(H=60)), (lb.LB_ERR_VARIANT, dict(ftype=3)), (lb.LB_ERR_VARIANT, dict(rtype=lb.LB_F16)),
        (lb.LB_ERR_VARIANT, dict(ftype=lb.LB_F32, rtype=lb.LB_BF16)),
        (lb.LB_ERR_OVERFLOW, dict(H=32776, ldy=32776, ldr=32776, ldro=32776, ldx=32776)),
        (lb.LB_ERR_ALIGN, dict(ldg=68)), (lb.LB_ERR_ALIGN, dict(ldy=68, X=ctypes.c_void_p(0x2000)))])
    refusals(lib.lb_residual_norm, a, [(lb.LB_ERR_ALIGN, {n: ODD}) for n in ("Y", "R", "post_w", "gate", "w", "R_out", "X")])


def test_rope_refusals(lib):
    a = Args(Q=P, ldq=256, K=P, ldk=128, pos=P, freqs=P, Qo=P, ldqo=256, Ko=P, ldko=128, T=3, Hq=4, Hk=2, D=64, R=32,
             layout=0, mult=1.0, ftype=lb.LB_F16, stream=NULL)
    refusals(lib.lb_rope, a, [(lb.LB_ERR_NULL, {n: NULL}) for n in ("Q", "K", "pos", "freqs", "Qo", "Ko")])
    refusals(lib.lb_rope, a, [
        (lb.LB_ERR_SHAPE, dict(T=0)), (lb.LB_ERR_SHAPE, dict(Hq=0)), (lb.LB_ERR_SHAPE, dict(Hk=-1)),
        (lb.LB_ERR_SHAPE, dict(Hq=65536, ldq=2 ** 23, ldqo=2 ** 23)), (lb.LB_ERR_SHAPE, dict(R=80)), (lb.LB_ERR_SHAPE, dict(R=0)),
        (lb.LB_ERR_SHAPE, dict(ldq=255)), (lb.LB_ERR_SHAPE, dict(ldk=64)), (lb.LB_ERR_SHAPE, dict(ldqo=8)),
        (lb.LB_ERR_SHAPE, dict(ldko=8)), (lb.LB_ERR_SHAPE, dict(ldqo=264)), (lb.LB_ERR_SHAPE, dict(ldko=264)),
        (lb.LB_ERR_SHAPE, dict(D=4104, ldq=2 ** 20, ldqo=2 ** 20, ldk=2 ** 20, ldko=2 ** 20)),
        (lb.LB_ERR_ALIGN, dict(R=24)), (lb.LB_ERR_ALIGN, dict(D=60, ldq=264, ldqo=264)),
        (lb.LB_ERR_VARIANT, dict(ftype=5)), (lb.LB_ERR_VARIANT, dict(layout=2)),
        (lb.LB_ERR_ALIGN, dict(ldq=260, Qo=ctypes.c_void_p(0x2000)))])
    refusals(lib.lb_rope, a, [(lb.LB_ERR_ALIGN, {n: ODD}) for n in ("Q", "K", "Qo", "Ko")])


def test_linear_w4_refusals(lib):
    a = Args(X=P, ldx=256, W=P, Wp=P, bias=NULL, out=P, M=4, N=8, K=256, group=128, ftype=lb.LB_BF16,
             ws=NULL, size=0, stream=NULL)
    refusals(lib.lb_linear_w4, a, [(lb.LB_ERR_NULL, {n: NULL}) for n in ("X", "W", "Wp", "out")])
    refusals(lib.lb_linear_w4, a, [(lb.LB_ERR_ALIGN, {n: ODD}) for n in ("X", "W", "Wp", "bias", "out")])
    refusals(lib.lb_linear_w4, a, [
        (lb.LB_ERR_SHAPE, dict(M=0)), (lb.LB_ERR_SHAPE, dict(N=0)), (lb.LB_ERR_SHAPE, dict(N=2 ** 31)),
        (lb.LB_ERR_SHAPE, dict(K=0)), (lb.LB_ERR_SHAPE, dict(group=16)), (lb.LB_ERR_SHAPE, dict(group=256)),
        (lb.LB_ERR_SHAPE, dict(ldx=255)), (lb.LB_ERR_ALIGN, dict(K=192)), (lb.LB_ERR_ALIGN, dict(ldx=260)),
        (lb.LB_ERR_VARIANT, dict(ftype=lb.LB_F32)), (lb.LB_ERR_OVERFLOW, dict(K=2 ** 20 + 128, ldx=2 ** 21)),
        (lb.LB_ERR_ALIGN, dict(M=4, ws=ctypes.c_void_p(0x1010), size=2 ** 30))])
    assert lib.lb_linear_w4_workspace(4, 200, 8, 128) == 0


def test_moe_refusals_and_workspace(lib):
    need = lib.lb_moe_w4_workspace(3, 256, 128, 16, 4)
    assert need % 256 == 0 and need >= 3 * 16 * 4 + 12 * 128 * 4
    # more tokens run 64 at a time
    assert lib.lb_moe_w4_workspace(64, 256, 128, 16, 4) == lib.lb_moe_w4_workspace(1000, 256, 128, 16, 4)
    a = Args(X=P, ldx=256, Wr=P, W1=P, P1=P, W2=P, P2=P, out=P, ids=NULL, weights=NULL, T=3, H=256, I=128, E=16, top_k=4,
             group=64, renorm=1, scale=1.0, ftype=lb.LB_F16, ws=P, size=need, stream=NULL)
    refusals(lib.lb_moe_w4, a, [(lb.LB_ERR_NULL, {n: NULL}) for n in ("X", "Wr", "W1", "P1", "W2", "P2", "out")])
    refusals(lib.lb_moe_w4, a, [(lb.LB_ERR_ALIGN, {n: ODD}) for n in ("X", "Wr", "W1", "P1", "W2", "P2", "out")])
    refusals(lib.lb_moe_w4, a, [
        (lb.LB_ERR_SHAPE, dict(T=0)), (lb.LB_ERR_SHAPE, dict(E=0)), (lb.LB_ERR_SHAPE, dict(E=1025)),
        (lb.LB_ERR_SHAPE, dict(top_k=0)), (lb.LB_ERR_SHAPE, dict(top_k=17)), (lb.LB_ERR_SHAPE, dict(E=128, top_k=65)),
        (lb.LB_ERR_SHAPE, dict(ldx=255)), (lb.LB_ERR_SHAPE, dict(group=48)), (lb.LB_ERR_SHAPE, dict(I=0)),
        (lb.LB_ERR_ALIGN, dict(I=96)), (lb.LB_ERR_ALIGN, dict(H=224)), (lb.LB_ERR_ALIGN, dict(ldx=260)),
        (lb.LB_ERR_VARIANT, dict(ftype=lb.LB_F32)), (lb.LB_ERR_OVERFLOW, dict(H=2 ** 18, I=2 ** 17, ldx=2 ** 18)),
        (lb.LB_ERR_WORKSPACE, dict(ws=NULL)), (lb.LB_ERR_WORKSPACE, dict(size=need - 1)),
        (lb.LB_ERR_ALIGN, dict(ws=ctypes.c_void_p(0x1010)))])
    assert lib.lb_moe_w4_workspace(3, 250, 128, 16, 4) == 0 and lib.lb_moe_w4_workspace(3, 256, 128, 16, 17) == 0


def freqs(R, *args):
    f, m = (ctypes.c_double * (R // 2))(), ctypes.c_float()
    assert lb.load().lb_rope_freqs(f, ctypes.byref(m), R, *args) == lb.LB_OK
    return np.array(f), m.value


@pytest.mark.parametrize("R", [2, 32, 128, 4096])
@pytest.mark.parametrize("base", [10000.0, 5e5])
def test_rope_freqs(lib, R, base):
    """Against the formulas; powers and logarithms are off by some units of 2^-53."""
    i = np.arange(R // 2)
    f = base ** (-2 * i / R)
    near = dict(rtol=1e-13, atol=0)
    np.testing.assert_allclose(freqs(R, base, lb.LB_ROPE_PLAIN, 0.0, 0.0, 0.0, 0.0)[0], f, **near)
    np.testing.assert_allclose(freqs(R, base, lb.LB_ROPE_LINEAR, 4.0, 0.0, 0.0, 0.0)[0], f / 4, **near)
    stretched = (base * 4 ** (R / (R - 2))) ** (-2 * i / R) if R > 2 else f
    np.testing.assert_allclose(freqs(R, base, lb.LB_ROPE_BASE, 4.0, 0.0, 0.0, 0.0)[0], stretched, **near)
    turns = 4096 * f / (2 * math.pi)
    got, m = freqs(R, base, lb.LB_ROPE_BANDS, 8.0, 4096.0, 1.0, 4.0)
    keep = np.clip((turns - 1) / 3, 0, 1)
    np.testing.assert_allclose(got, f / 8 * (1 - keep) + f * keep, rtol=1e-12, atol=0)
    assert m == 1
    got, m = freqs(R, base, lb.LB_ROPE_PARTS, 8.0, 4096.0, 1.0, 32.0)
    assert m == np.float32(0.1 * math.log(8) + 1)
    # pairs that turn often stay, those that hardly turn are stretched, in between neither; falling throughout
    if R > 2:
        assert np.allclose(got[turns >= 40], f[turns >= 40], **near)
        assert np.allclose(got[turns <= 0.5], f[turns <= 0.5] / 8, **near)
        assert (np.diff(got) < 0).all() and (got <= f * (1 + 1e-15)).all() and (got >= f / 8 * (1 - 1e-15)).all()


def test_rope_freqs_refusals(lib):
    f, m = (ctypes.c_double * 8)(), ctypes.byref(ctypes.c_float())
    a = Args(f=f, m=m, R=16, base=1e4, scaling=3, factor=2.0, before=4096.0, low=1.0, high=32.0)
    refusals(lib.lb_rope_freqs, a, [
        (lb.LB_OK, {}), (lb.LB_ERR_NULL, dict(f=None)), (lb.LB_ERR_NULL, dict(m=None)), (lb.LB_ERR_SHAPE, dict(R=0)),
        (lb.LB_ERR_SHAPE, dict(R=15)), (lb.LB_ERR_SHAPE, dict(R=4098)), (lb.LB_ERR_SHAPE, dict(base=1.0)),
        (lb.LB_ERR_VARIANT, dict(scaling=5)), (lb.LB_ERR_VARIANT, dict(scaling=-1)), (lb.LB_ERR_SHAPE, dict(factor=0.0)),
        (lb.LB_ERR_SHAPE, dict(before=0.0)), (lb.LB_ERR_SHAPE, dict(low=0.0)), (lb.LB_ERR_SHAPE, dict(high=1.0)),
        (lb.LB_ERR_SHAPE, dict(base=float("nan"))), (lb.LB_ERR_SHAPE, dict(factor=float("nan")))])


def test_binding_checks_without_a_gpu():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        lb.lb_residual_norm(x, x, x, x, w=x[0])
    with pytest.raises(ValueError, match="None"):
        lb.lb_residual_norm(None, None, x, x, w=x[0])
    q = torch.zeros(4, 2, 64, dtype=torch.float16)
    pos, f = torch.zeros(4, dtype=torch.int64), torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="GPU"):
        lb.lb_rope(q, q, pos, f, q, q)
    with pytest.raises(ValueError, match="layout"):
        lb.lb_rope(q, q, pos, f, q, q, layout="other")
    w, p = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, 2, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        lb.lb_linear_w4(x, w, p, torch.zeros(4, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="divide"):
        lb.lb_linear_w4(x, w, torch.zeros(8, 3, 2, dtype=torch.bfloat16), torch.zeros(4, 8, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="dtype"):
        lb.lb_linear_w4(x.float(), w, p.float(), torch.zeros(4, 8))
    w1, p1 = torch.zeros(2, 64, 32, dtype=torch.uint8), torch.zeros(2, 64, 2, 2, dtype=torch.bfloat16)
    w2, p2 = torch.zeros(2, 64, 16, dtype=torch.uint8), torch.zeros(2, 64, 1, 2, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        lb.lb_moe_w4(x, torch.zeros(2, 64, dtype=torch.bfloat16), w1, p1, w2, p2, torch.zeros_like(x), top_k=1)


def test_sizes_beyond_the_limits(lib):
    """More columns than a launch covers; rows too far apart; the limit itself is the header's."""
    import os
    import re
    text = open(os.path.join(os.path.dirname(lb.__file__), "..", "include", "lb_gemm.h")).read()
    assert int(re.search(r"#define LB_W4_N_MAX (\d+)", text).group(1)) == lb.W4_N_MAX
    a = Args(X=P, ldx=128, W=P, Wp=P, bias=NULL, out=P, M=3, N=64, K=128, group=64, ftype=lb.LB_BF16, ws=NULL, bytes=0, stream=NULL)
    refusals(lib.lb_linear_w4, a, [(lb.LB_ERR_OVERFLOW, dict(N=lb.W4_N_MAX + 1)), (lb.LB_ERR_OVERFLOW, dict(M=40, N=lb.W4_N_MAX + 16)),
                                   (lb.LB_ERR_OVERFLOW, dict(ldx=2 ** 24 + 8))])
    assert lb.lb_linear_w4_workspace(40, 128, lb.W4_N_MAX + 16, 64) == 0
    assert lb.lb_linear_w4_workspace(40, 128, lb.W4_N_MAX, 64) > 0


@pytest.mark.parametrize("before,low,high", [(4.0, 1.0, 32.0), (6.0, 1.0, 4.0), (40.0, 8.0, 32.0), (100.0, 16.0, 17.0), (200.0, 1.0, 32.0)])
@pytest.mark.parametrize("R", [2, 4, 64])
def test_rope_freqs_parts_of_short_contexts(lib, R, before, low, high):
    """A pair that turns at most `low` times is stretched, one that turns `high` times is not, the first pair too."""
    f = 10000.0 ** (-2 * np.arange(R // 2) / R)
    turns = before * f / (2 * math.pi)
    got, _ = freqs(R, 10000.0, lb.LB_ROPE_PARTS, 8.0, before, low, high)
    near = dict(rtol=1e-13, atol=0)
    np.testing.assert_allclose(got[turns <= low * (1 - 1e-9)], f[turns <= low * (1 - 1e-9)] / 8, **near)
    np.testing.assert_allclose(got[turns >= high * (1 + 1e-9)], f[turns >= high * (1 + 1e-9)], **near)
    assert (got <= f * (1 + 1e-15)).all() and (got >= f / 8 * (1 - 1e-15)).all()


def test_rope_freqs_names(lib):
    pytest.importorskip("torch")
    for name, number in (("plain", lb.LB_ROPE_PLAIN), ("linear", lb.LB_ROPE_LINEAR), ("base", lb.LB_ROPE_BASE),
                         ("parts", lb.LB_ROPE_PARTS), ("bands", lb.LB_ROPE_BANDS)):
        args = dict(factor=4.0, before=4096.0, device="cpu")
        (f, m), (g, n) = (lb.lb_rope_freqs(64, scaling=s, **args) for s in (name, number))
        assert (f == g).all() and m == n and len(f) == 32
    for other in ("longer", 5, -1, None):
        with pytest.raises(ValueError, match="scaling"):
            lb.lb_rope_freqs(64, scaling=other, device="cpu")
