// lb_serve.cpp -- the extern "C" boundary of the serving operators: argument
// checks, planning of the attention's key ranges, launches on the caller's stream.
#include "lb_gemm.h"

#include <hip/hip_runtime.h>

#include <algorithm>

#include "lb_internal.hpp"

namespace {

const int64_t kLim = 0x7FFFFFFF;

bool aligned(const void *p, uintptr_t to = 16) { return (uintptr_t)p % to == 0; }
int64_t elem_of(int ftype) { return ftype == LB_F32 ? 4 : 2; }
bool any_ftype(int t) { return t == LB_BF16 || t == LB_F16 || t == LB_F32; }
bool short_ftype(int t) { return t == LB_BF16 || t == LB_F16; }
int finish(hipError_t e) { return e == hipSuccess ? LB_OK : LB_ERR_HIP; }

// Sizes, K rule, type and K limit of the int8 product, in the documented order.
int check_product(int64_t M, int64_t N, int64_t K, int ftype)
{
    if (M <= 0 || N <= 0 || K <= 0 || M > kLim || N > kLim) return LB_ERR_SHAPE;
    if (K % LB_S8_K_ALIGN != 0) return LB_ERR_ALIGN;
    if (!any_ftype(ftype)) return LB_ERR_VARIANT;
    if (K > LB_S8_K_MAX) return LB_ERR_OVERFLOW;
    return LB_OK;
}

// Compute units of the current device; if it cannot be asked, as on a whole chip.
int cu_count()
{
    int cu = 0;
    return lb::device_cu_count(&cu) == LB_OK ? cu : 256;
}

int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

int scaled(const int8_t *X, const int8_t *W, const float *sx, const float *sw, const void *bias, void *out,
           int64_t M, int64_t N, int64_t K, int ftype, hipStream_t s)
{
    const int cu = cu_count();
    if (lb::linear_is_few(M, N, cu) && !lb::variant_is_forced())
        return finish(lb::launch_linear_few(ftype, X, W, sx, sw, bias, out, M, N, K, cu, s));
    // (4 threads to a row, or a column, of the narrowest tile)
    const int64_t most = lb::LAUNCH_THREADS / 8, elem = elem_of(ftype);
    for (int64_t m0 = 0; m0 < M; m0 += most)
        for (int64_t n0 = 0; n0 < N; n0 += most) {
            const lb::ScaledOut so{bias ? (const char *)bias + n0 * elem : nullptr, ftype};
            const int st = lb::scaled_auto(X + m0 * K, W + n0 * K, sx + m0, sw + n0, (char *)out + (m0 * N + n0) * elem,
                                           std::min(most, M - m0), std::min(most, N - n0), K, N, so, s);
            if (st != LB_OK) return st;
        }
    return LB_OK;
}

// Sizes of the cache.
int check_cache(int64_t heads, int64_t D, int64_t pages, int64_t page, int ftype)
{
    if (heads <= 0 || pages <= 0 || page <= 0 || (D != 64 && D != 128 && D != 256)) return LB_ERR_SHAPE;
    if (heads > 32767 || pages > kLim || page > kLim || (double)pages * (double)page >= 2147483648.0)
        return LB_ERR_SHAPE;
    if (page % LB_KV4_PAGE_ALIGN != 0) return LB_ERR_ALIGN;
    if (!short_ftype(ftype)) return LB_ERR_VARIANT;
    return LB_OK;
}

lb::Kv4Cache cache_of(const uint8_t *Kc, const uint8_t *Vc, const void *Kp, const void *Vp, int64_t heads,
                      int64_t pages, int64_t page)
{
    lb::Kv4Cache c;
    c.k = const_cast<uint8_t *>(Kc);
    c.v = const_cast<uint8_t *>(Vc);
    c.kp = (uint32_t *)const_cast<void *>(Kp);
    c.vp = (uint32_t *)const_cast<void *>(Vp);
    c.pages = pages;
    c.page = (int32_t)page;
    c.heads = (int32_t)heads;
    // slot / page = mulhi(slot, mul) >> shift with 2^shift the power of two below page:
    // mul = ceil(2^(32 + shift) / page) < 2^32, and mul page - 2^(32 + shift) < page
    // <= 2^(shift + 1), so the quotient is exact for slots below 2^31.
    c.page_shift = 31 - (uint32_t)__builtin_clz((uint32_t)page);
    if ((page & (page - 1)) == 0) --c.page_shift;
    c.page_mul = (uint32_t)((((uint64_t)1 << (32 + c.page_shift)) + (uint64_t)page - 1) / (uint64_t)page);
    return c;
}

// One attention call: the kernel, its tiles of rows per key head, the key ranges or
// shares that it makes at most, and the workspace these take.
struct AttnPlan {
    int kernel;
    int64_t tiles, splits, unit, bytes;
};

AttnPlan plan_attn(int64_t B, int64_t total_q, int64_t max_q, int64_t Hq, int64_t Hkv, int64_t D,
                   int64_t max_len, int64_t window, int cu, bool have_workspace, int64_t workspace_bytes)
{
    AttnPlan p{lb::ATTN_ROWS, 0, 1, 1, 0};
    const int64_t rows = max_q * (Hq / Hkv);
    const int64_t keys = window > 0 ? std::min(max_len, window + max_q) : max_len;
    if (rows > 192) {
        // Many rows of a key head share its keys through LDS.  One workgroup to a
        // compute unit; a range costs its rows' partial results in fp32, written and
        // read, about as much as nine tiles of 64 keys: no ranges once there are
        // workgroups for all units, and none below 16 tiles.
        p.kernel = lb::ATTN_CHUNK;
        p.tiles = D == 256 ? (rows + 127) / 128 : (rows + 255) / 256;
        const int64_t blocks = std::max<int64_t>((keys + 63) / 64, 1), per = total_q * Hq * (D + 2) * 4;
        p.splits = std::min((int64_t)cu / (B * Hkv * p.tiles), blocks / 16);
        if (!have_workspace) workspace_bytes = p.splits * per;
        p.splits = std::max<int64_t>(1, std::min({p.splits, (int64_t)64, workspace_bytes / per}));
        p.unit = (blocks + p.splits - 1) / p.splits;
        p.bytes = p.splits > 1 ? p.splits * per : 0;
        return p;
    }
    p.tiles = (rows + 15) / 16;
    const int64_t wgs = B * Hkv * p.tiles, blocks = std::max<int64_t>((keys + 31) / 32, 1), part = 16 * (D + 2) * 4;
    if (wgs <= cu) {
        // Workgroups that fill a compute unit, two blocks to a wave at least before
        // there is a second range (and a launch to join them).  (With more tiles than
        // units they only queue: 384 of D = 64 and 1024 keys 22 us against 16 with four
        // waves each, 320 of D = 128 and 1000 keys 24 against 19.)
        p.kernel = lb::ATTN_WIDE;
        p.splits = std::min((int64_t)cu / wgs, blocks / (2 * lb::attn_wide_waves((int)D)));
        if (!have_workspace) workspace_bytes = p.splits * wgs * part;
        p.splits = std::max<int64_t>(1, std::min({p.splits, (int64_t)64, workspace_bytes / (wgs * part)}));
        p.unit = (blocks + p.splits - 1) / p.splits;
        p.bytes = p.splits > 1 ? p.splits * wgs * part : 0;
    } else if (wgs < 8 * (int64_t)cu && B <= lb::ATTN_FLAT_BATCH && window == 0 && blocks >= 96) {
        // Some tiles to a compute unit, whose lengths may differ: equal shares, as many
        // as run at once.  (Many more tiles even out by themselves, windows make them
        // equal, and short ones are not worth a second launch.)
        const int64_t shares = (D == 256 ? 2 : 3) * (int64_t)cu, bytes = shares * (2 * part + 16);
        if (!have_workspace || workspace_bytes >= bytes) {
            p.kernel = lb::ATTN_FLAT;
            p.splits = shares;
            p.bytes = bytes;
        }
    }
    return p;
}

}  // namespace

extern "C" {

int lb_quant_rows_s8(const void *X, int64_t ldx, int8_t *Q, float *sx, int64_t M, int64_t K, int ftype,
                     void *stream)
{
    if (!X || !Q || !sx) return LB_ERR_NULL;
    if (ldx < K) return LB_ERR_SHAPE;
    const int st = check_product(M, 1, K, ftype);
    if (st != LB_OK) return st;
    if (!aligned(X) || !aligned(Q) || ldx * elem_of(ftype) % 16 != 0) return LB_ERR_ALIGN;
    return finish(lb::launch_quant_rows(ftype, X, ldx, Q, sx, M, K, (hipStream_t)stream));
}

int lb_gemm_s8_scaled(const int8_t *X, const int8_t *W, const float *sx, const float *sw, const void *bias,
                      void *out, int64_t M, int64_t N, int64_t K, int ftype, void *stream)
{
    if (!X || !W || !sx || !sw || !out) return LB_ERR_NULL;
    const int st = check_product(M, N, K, ftype);
    if (st != LB_OK) return st;
    if (!aligned(X) || !aligned(W) || !aligned(out) || !aligned(bias) || !aligned(sw)) return LB_ERR_ALIGN;
    return scaled(X, W, sx, sw, bias, out, M, N, K, ftype, (hipStream_t)stream);
}

int64_t lb_linear_w8a8_workspace(int64_t M, int64_t K, int64_t N)
{
    if (check_product(M, N, K, LB_BF16) != LB_OK) return 0;
    return round_up(M * K, 256) + round_up(M * 4, 256);
}

int lb_linear_w8a8(const void *X, int64_t ldx, const int8_t *W, const float *sw, const void *bias, void *out,
                   int64_t M, int64_t N, int64_t K, int ftype, void *workspace, int64_t workspace_bytes,
                   void *stream)
{
    if (!X || !W || !sw || !out) return LB_ERR_NULL;
    if (ldx < K) return LB_ERR_SHAPE;
    const int st = check_product(M, N, K, ftype);
    if (st != LB_OK) return st;
    if (!aligned(X) || !aligned(W) || !aligned(out) || !aligned(bias) || !aligned(sw) ||
        ldx * elem_of(ftype) % 16 != 0)
        return LB_ERR_ALIGN;
    if (!workspace || workspace_bytes < lb_linear_w8a8_workspace(M, K, N)) return LB_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return LB_ERR_ALIGN;
    const hipStream_t s = (hipStream_t)stream;
    const int cu = cu_count();
    if (lb::linear_fuses(M, N, K, cu) && !lb::variant_is_forced())
        return finish(lb::launch_linear_fused(ftype, X, ldx, W, sw, bias, out, M, N, K, cu, s));
    int8_t *q = (int8_t *)workspace;
    float *sx = (float *)(q + round_up(M * K, 256));
    if (lb::launch_quant_rows(ftype, X, ldx, q, sx, M, K, s) != hipSuccess) return LB_ERR_HIP;
    return scaled(q, W, sx, sw, bias, out, M, N, K, ftype, s);
}

int lb_kv4_write(const void *K, const void *V, int64_t ldk, int64_t ldv, const int64_t *slots, uint8_t *Kc,
                 uint8_t *Vc, void *Kp, void *Vp, int64_t T, int64_t heads, int64_t D, int64_t pages,
                 int64_t page, int ftype, void *stream)
{
    if (!K || !V || !slots || !Kc || !Vc || !Kp || !Vp) return LB_ERR_NULL;
    if (T <= 0 || T > kLim) return LB_ERR_SHAPE;
    const int st = check_cache(heads, D, pages, page, ftype);
    if (st != LB_OK) return st;
    if (ldk < heads * D || ldv < heads * D) return LB_ERR_SHAPE;
    if (!aligned(K) || !aligned(V) || !aligned(Kc) || !aligned(Vc) || !aligned(Kp) || !aligned(Vp) ||
        ldk % 8 != 0 || ldv % 8 != 0)
        return LB_ERR_ALIGN;
    return finish(lb::launch_kv4_write(ftype, K, V, ldk, ldv, slots, cache_of(Kc, Vc, Kp, Vp, heads, pages, page),
                                       T, (int)D, (hipStream_t)stream));
}

int lb_kv4_read(const uint8_t *Kc, const uint8_t *Vc, const void *Kp, const void *Vp, const int64_t *slots,
                void *K, void *V, int64_t T, int64_t heads, int64_t D, int64_t pages, int64_t page, int ftype,
                void *stream)
{
    if (!K || !V || !slots || !Kc || !Vc || !Kp || !Vp) return LB_ERR_NULL;
    if (T <= 0 || T > kLim) return LB_ERR_SHAPE;
    const int st = check_cache(heads, D, pages, page, ftype);
    if (st != LB_OK) return st;
    if (!aligned(K) || !aligned(V) || !aligned(Kc) || !aligned(Vc) || !aligned(Kp) || !aligned(Vp))
        return LB_ERR_ALIGN;
    return finish(lb::launch_kv4_read(ftype, cache_of(Kc, Vc, Kp, Vp, heads, pages, page), slots, K, V, T, (int)D,
                                      (hipStream_t)stream));
}

static int check_attn(int64_t B, int64_t total_q, int64_t max_q, int64_t Hq, int64_t Hkv, int64_t D,
                      int64_t max_len, int64_t window)
{
    if (B <= 0 || total_q <= 0 || max_q <= 0 || Hq <= 0 || Hkv <= 0 || max_len < 0 || window < 0)
        return LB_ERR_SHAPE;
    if (B > kLim || total_q > kLim || max_q > kLim || Hq > 65535 || Hkv > 32767 || max_len > kLim || window > kLim)
        return LB_ERR_SHAPE;
    if (Hq % Hkv != 0 || (D != 64 && D != 128 && D != 256)) return LB_ERR_SHAPE;
    // row numbers of a key head, and of the whole batch's tiles, are 32-bit
    if ((double)max_q * (double)(Hq / Hkv) >= 2147483632.0) return LB_ERR_OVERFLOW;
    if ((double)B * (double)Hkv * (double)((max_q * (Hq / Hkv) + 15) / 16) >= 2147483648.0) return LB_ERR_OVERFLOW;
    // one sequence is one launch
    if (Hkv * ((std::min(max_q, total_q) * (Hq / Hkv) + 127) / 128) * 512 > lb::LAUNCH_THREADS) return LB_ERR_OVERFLOW;
    return LB_OK;
}

int64_t lb_attn_kv4_workspace(int64_t B, int64_t total_q, int64_t max_q, int64_t Hq, int64_t Hkv, int64_t D,
                              int64_t max_len, int64_t window, int cu_count)
{
    if (check_attn(B, total_q, max_q, Hq, Hkv, D, max_len, window) != LB_OK) return 0;
    if (cu_count <= 0 && lb::device_cu_count(&cu_count) != LB_OK) return 0;
    return round_up(plan_attn(B, total_q, std::min(max_q, total_q), Hq, Hkv, D, max_len, window, cu_count, false, 0).bytes,
                    256);
}

int lb_attn_kv4(const void *Q, int64_t ldq, const uint8_t *Kc, const uint8_t *Vc, const void *Kp,
                const void *Vp, const int32_t *table, int64_t ldt, int64_t table_width, const int32_t *q_off,
                const int32_t *lens, void *out, int64_t ldo, float *lse, int64_t B, int64_t total_q,
                int64_t max_q, int64_t Hq, int64_t Hkv, int64_t D, int64_t pages, int64_t page,
                int64_t max_len, float scale, int64_t window, int causal, int ftype, void *workspace,
                int64_t workspace_bytes, void *stream)
{
    if (!Q || !Kc || !Vc || !Kp || !Vp || !table || !q_off || !lens || !out) return LB_ERR_NULL;
    int st = check_attn(B, total_q, max_q, Hq, Hkv, D, max_len, window);
    if (st == LB_ERR_SHAPE) return st;
    if (table_width <= 0 || ldt < table_width || table_width > kLim || ldq < Hq * D || ldo < Hq * D)
        return LB_ERR_SHAPE;
    const int sc = check_cache(Hkv, D, pages, page, ftype);
    if (sc != LB_OK) return sc;
    if (st != LB_OK) return st;
    // key numbers, and those up to three tiles past the last, are 32-bit
    if ((double)table_width * (double)page >= 2147482624.0) return LB_ERR_OVERFLOW;
    if (!aligned(Q) || !aligned(Kc) || !aligned(Vc) || !aligned(Kp) || !aligned(Vp) || !aligned(out) ||
        ldq % 8 != 0 || ldo % 8 != 0 || !aligned(workspace, 256))
        return LB_ERR_ALIGN;
    const int cu = cu_count();
    max_q = std::min(max_q, total_q);
    const AttnPlan p = plan_attn(B, total_q, max_q, Hq, Hkv, D, max_len, window, cu, true,
                                 workspace ? std::max<int64_t>(workspace_bytes, 0) : 0);

    lb::AttnArgs a;
    a.q = Q;
    a.out = out;
    a.lse = lse;
    a.table = table;
    a.q_off = q_off;
    a.lens = lens;
    a.part = (float *)workspace;
    a.c = cache_of(Kc, Vc, Kp, Vp, Hkv, pages, page);
    a.ldq = ldq;
    a.ldo = ldo;
    a.ldt = ldt;
    a.width = table_width;
    a.total_q = total_q;
    a.group = (int32_t)(Hq / Hkv);
    a.batch = (int32_t)B;
    a.window = (int32_t)window;
    a.causal = causal != 0;
    a.splits = (int32_t)p.splits;
    a.unit = (int32_t)p.unit;
    a.kernel = p.kernel;
    a.tiles = (int32_t)p.tiles;
    a.scale2 = scale * 1.44269504088896340736f;
    return finish(lb::launch_attn(ftype, (int)D, a, (hipStream_t)stream));
}

}  // extern "C"
