"""CPU tests of the serving operators' C boundary: bad arguments get the documented
status before any HIP call, the workspace sizes, and the binding's own checks.
Nothing is launched here."""
import ctypes

import pytest

import bit_integer_gemm_amd as lb

P = ctypes.c_void_p(0x1000)        # never dereferenced: every call below fails validation
ODD = ctypes.c_void_p(0x1008)      # not 16-byte aligned
NULL = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    from bit_integer_gemm_amd import _build
    _build.ensure_built()
    return lb.load()


class Args(dict):
    """Positional arguments by name, in the header's order."""

    def __call__(self, **kw):
        assert set(kw) <= set(self), kw
        return list({**self, **kw}.values())


def refusals(fn, args, cases):
    for want, kw in cases:
        assert fn(*args(**kw)) == want, kw


def test_quant_rows_refusals(lib):
    a = Args(X=P, ldx=64, Q=P, sx=P, M=4, K=64, ftype=lb.LB_BF16, stream=NULL)
    refusals(lib.lb_quant_rows_s8, a, [
        (lb.LB_ERR_NULL, dict(X=NULL)), (lb.LB_ERR_NULL, dict(Q=NULL)), (lb.LB_ERR_NULL, dict(sx=NULL)),
        (lb.LB_ERR_SHAPE, dict(M=0)), (lb.LB_ERR_SHAPE, dict(M=2 ** 31)), (lb.LB_ERR_SHAPE, dict(K=0)),
        (lb.LB_ERR_SHAPE, dict(ldx=48)), (lb.LB_ERR_ALIGN, dict(K=40)), (lb.LB_ERR_ALIGN, dict(ldx=68)),
        (lb.LB_ERR_ALIGN, dict(X=ODD)), (lb.LB_ERR_ALIGN, dict(Q=ODD)), (lb.LB_ERR_VARIANT, dict(ftype=3)),
        (lb.LB_ERR_VARIANT, dict(ftype=-1)), (lb.LB_ERR_OVERFLOW, dict(K=131072, ldx=131072))])


def test_scaled_product_refusals(lib):
    a = Args(X=P, W=P, sx=P, sw=P, bias=NULL, out=P, M=4, N=8, K=64, ftype=lb.LB_F16, stream=NULL)
    refusals(lib.lb_gemm_s8_scaled, a, [
        (lb.LB_ERR_NULL, dict(X=NULL)), (lb.LB_ERR_NULL, dict(W=NULL)), (lb.LB_ERR_NULL, dict(sx=NULL)),
        (lb.LB_ERR_NULL, dict(sw=NULL)), (lb.LB_ERR_NULL, dict(out=NULL)), (lb.LB_ERR_SHAPE, dict(M=-1)),
        (lb.LB_ERR_SHAPE, dict(N=0)), (lb.LB_ERR_SHAPE, dict(N=2 ** 31)), (lb.LB_ERR_ALIGN, dict(K=24)),
        (lb.LB_ERR_VARIANT, dict(ftype=7)), (lb.LB_ERR_OVERFLOW, dict(K=131072)),
        (lb.LB_ERR_ALIGN, dict(bias=ODD)), (lb.LB_ERR_ALIGN, dict(W=ODD)), (lb.LB_ERR_ALIGN, dict(out=ODD))])


def test_linear_refusals_and_workspace(lib):
    need = lib.lb_linear_w8a8_workspace(4, 64, 8)
    assert need >= 4 * 64 + 4 * 4 and need % 256 == 0
    assert lib.lb_linear_w8a8_workspace(4, 65, 8) == 0 and lib.lb_linear_w8a8_workspace(0, 64, 8) == 0
    # 64-bit sizes
    assert lib.lb_linear_w8a8_workspace(2 ** 20, 65536, 8) > 2 ** 36
    a = Args(X=P, ldx=64, W=P, sw=P, bias=NULL, out=P, M=4, N=8, K=64, ftype=lb.LB_F32, ws=P, size=need,
             stream=NULL)
    refusals(lib.lb_linear_w8a8, a, [
        (lb.LB_ERR_NULL, dict(X=NULL)), (lb.LB_ERR_NULL, dict(W=NULL)), (lb.LB_ERR_NULL, dict(sw=NULL)),
        (lb.LB_ERR_NULL, dict(out=NULL)), (lb.LB_ERR_SHAPE, dict(ldx=63)), (lb.LB_ERR_SHAPE, dict(M=0)),
        (lb.LB_ERR_ALIGN, dict(K=56)), (lb.LB_ERR_ALIGN, dict(ldx=65)), (lb.LB_ERR_ALIGN, dict(out=ODD)),
        (lb.LB_ERR_VARIANT, dict(ftype=9)), (lb.LB_ERR_WORKSPACE, dict(ws=NULL)),
        (lb.LB_ERR_WORKSPACE, dict(size=need - 1)), (lb.LB_ERR_ALIGN, dict(ws=ctypes.c_void_p(0x1010)))])


def test_cache_refusals(lib):
    w = Args(K=P, V=P, ldk=256, ldv=256, slots=P, Kc=P, Vc=P, Kp=P, Vp=P, T=3, heads=4, D=64, pages=5, page=16,
             ftype=lb.LB_BF16, stream=NULL)
    r = Args(Kc=P, Vc=P, Kp=P, Vp=P, slots=P, K=P, V=P, T=3, heads=4, D=64, pages=5, page=16, ftype=lb.LB_BF16,
             stream=NULL)
    for fn, a in ((lib.lb_kv4_write, w), (lib.lb_kv4_read, r)):
        refusals(fn, a, [(lb.LB_ERR_NULL, {n: NULL}) for n in ("K", "V", "slots", "Kc", "Vc", "Kp", "Vp")])
        refusals(fn, a, [(lb.LB_ERR_ALIGN, {n: ODD}) for n in ("K", "V", "Kc", "Vc", "Kp", "Vp")])
        refusals(fn, a, [
            (lb.LB_ERR_SHAPE, dict(T=0)), (lb.LB_ERR_SHAPE, dict(heads=0)), (lb.LB_ERR_SHAPE, dict(D=96)),
            (lb.LB_ERR_SHAPE, dict(pages=0)), (lb.LB_ERR_SHAPE, dict(page=-16)),
            (lb.LB_ERR_SHAPE, dict(pages=2 ** 27, page=16)), (lb.LB_ERR_ALIGN, dict(page=24)),
            (lb.LB_ERR_VARIANT, dict(ftype=lb.LB_F32))])
    refusals(lib.lb_kv4_write, w, [(lb.LB_ERR_SHAPE, dict(ldk=255)), (lb.LB_ERR_SHAPE, dict(ldv=128)),
                                   (lb.LB_ERR_ALIGN, dict(ldk=260))])


def attn_args():
    return Args(Q=P, ldq=512, Kc=P, Vc=P, Kp=P, Vp=P, table=P, ldt=8, width=8, q_off=P, lens=P, out=P, ldo=512,
                lse=NULL, B=2, total_q=3, max_q=2, Hq=8, Hkv=2, D=64, pages=5, page=16, max_len=100, scale=0.1,
                window=0, causal=1, ftype=lb.LB_F16, ws=NULL, size=0, stream=NULL)


def test_attention_refusals(lib):
    a = attn_args()
    refusals(lib.lb_attn_kv4, a, [(lb.LB_ERR_NULL, {n: NULL}) for n in
                                  ("Q", "Kc", "Vc", "Kp", "Vp", "table", "q_off", "lens", "out")])
    refusals(lib.lb_attn_kv4, a, [(lb.LB_ERR_ALIGN, {n: ODD}) for n in ("Q", "Kc", "Vc", "Kp", "Vp", "out")])
    refusals(lib.lb_attn_kv4, a, [
        (lb.LB_ERR_SHAPE, dict(B=0)), (lb.LB_ERR_SHAPE, dict(total_q=0)), (lb.LB_ERR_SHAPE, dict(max_q=0)),
        (lb.LB_ERR_SHAPE, dict(Hq=9)), (lb.LB_ERR_SHAPE, dict(Hkv=0)), (lb.LB_ERR_SHAPE, dict(D=80)),
        (lb.LB_ERR_SHAPE, dict(max_len=-1)), (lb.LB_ERR_SHAPE, dict(window=-1)), (lb.LB_ERR_SHAPE, dict(ldq=511)),
        (lb.LB_ERR_SHAPE, dict(ldo=8)), (lb.LB_ERR_SHAPE, dict(ldt=7)), (lb.LB_ERR_SHAPE, dict(width=0)),
        (lb.LB_ERR_SHAPE, dict(pages=0)), (lb.LB_ERR_ALIGN, dict(page=8)), (lb.LB_ERR_ALIGN, dict(ldq=516)),
        (lb.LB_ERR_VARIANT, dict(ftype=lb.LB_F32)), (lb.LB_ERR_ALIGN, dict(ws=ctypes.c_void_p(0x1040), size=4)),
        (lb.LB_ERR_OVERFLOW, dict(width=2 ** 27, ldt=2 ** 27)),
        (lb.LB_ERR_OVERFLOW, dict(total_q=2 ** 30, max_q=2 ** 30))])


def test_attention_workspace(lib):
    """Few rows over many keys are split; many rows are not; refused sizes need nothing."""
    f = lb.lb_attn_kv4_workspace
    one = f(1, 1, 1, 32, 8, 128, 100000, cu_count=256)
    assert one % 256 == 0 and one >= 2 * 32 * (128 + 2) * 4
    assert f(1, 1, 1, 32, 8, 128, 200, cu_count=256) == 0
    assert f(512, 512, 1, 32, 8, 128, 100000, cu_count=256) == 0
    assert f(1, 1, 1, 32, 8, 128, 100000, window=128, cu_count=256) < one
    assert f(1, 1, 1, 33, 8, 128, 100000, cu_count=256) == 0
    assert f(1, 1, 1, 32, 8, 96, 100000, cu_count=256) == 0
    # max_q beyond the batch's queries counts as all of them
    assert f(1, 1, 7, 32, 8, 128, 100000, cu_count=256) == one


def test_binding_checks_without_a_gpu():
    """Shapes, types and devices are refused in Python before any address is taken."""
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(8, 64, dtype=torch.int8)
    sw, out = torch.zeros(8), torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        lb.lb_linear_w8a8(x, w, sw, out)
    with pytest.raises(ValueError, match="GPU"):
        lb.lb_quant_rows_s8(x, torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4))
    k = torch.zeros(3, 2, 64, dtype=torch.float16)
    c = torch.zeros(5, 2, 16, 32, dtype=torch.uint8)
    p = torch.zeros(5, 2, 16, 2, dtype=torch.float16)
    s = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):
        lb.lb_kv4_write(k, k, s, c, c, p, p)
    with pytest.raises(ValueError, match="GPU"):
        lb.lb_kv4_read(c, c, p, p, s, k, k)
    with pytest.raises(ValueError, match="GPU"):
        lb.lb_attn_kv4(k, c, c, p, p, torch.zeros(1, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                       torch.zeros(1, dtype=torch.int32), k)


def test_attention_rows_beyond_one_launch(lib):
    """One sequence is one launch of fewer than 2^32 threads; more than that is refused, not left to the runtime."""
    a = attn_args()
    wide = dict(Hq=32767, Hkv=32767, ldq=32767 * 64, ldo=32767 * 64)
    assert lib.lb_attn_kv4(*a(total_q=2 ** 18, max_q=2 ** 18, **wide)) == lb.LB_ERR_OVERFLOW
    assert lb.lb_attn_kv4_workspace(2, 2 ** 18, 2 ** 18, 32767, 32767, 64, 100, cu_count=256) == 0
