// lb_layer.cpp -- the extern "C" boundary of the operators that complete a decoder layer around
// the exact products and the attention: argument checks, workspaces, rotary frequencies,
// launches on the caller's stream.
#include "lb_gemm.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "lb_layer.hpp"

namespace {

const int64_t kLim = 0x7FFFFFFF;

bool aligned(const void *p, uintptr_t to = 16) { return (uintptr_t)p % to == 0; }
int64_t elem_of(int ftype) { return ftype == LB_F32 ? 4 : 2; }
bool any_ftype(int t) { return t == LB_BF16 || t == LB_F16 || t == LB_F32; }
bool short_ftype(int t) { return t == LB_BF16 || t == LB_F16; }
int finish(hipError_t e) { return e == hipSuccess ? LB_OK : LB_ERR_HIP; }
bool rows_aligned(int64_t ld, int ftype) { return ld * elem_of(ftype) % 16 == 0; }
int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

int cu_count()
{
    int cu = 0;
    return lb::device_cu_count(&cu) == LB_OK ? cu : 256;
}

// Sizes, group and K rules of a 4-bit product, in the documented order.
int check_w4(int64_t M, int64_t N, int64_t K, int64_t group, int ftype)
{
    if (M <= 0 || N <= 0 || K <= 0 || M > kLim || N > kLim || (group != 32 && group != 64 && group != 128))
        return LB_ERR_SHAPE;
    if (K % group != 0) return LB_ERR_ALIGN;
    if (!short_ftype(ftype)) return LB_ERR_VARIANT;
    if (K > LB_W4_K_MAX || N > LB_W4_N_MAX) return LB_ERR_OVERFLOW;
    return LB_OK;
}
// Byte offsets between 64 rows of x are 32-bit.
const int64_t kLdMax = (int64_t)1 << 24;

int check_moe(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top_k, int64_t group, int ftype)
{
    if (E <= 0 || E > LB_MOE_EXPERTS_MAX || top_k <= 0 || top_k > E || top_k > LB_MOE_TOP_MAX) return LB_ERR_SHAPE;
    int st = check_w4(T, H, I, group, ftype);
    if (st == LB_OK) st = check_w4(T, I, H, group, ftype);
    if (st != LB_OK) return st;
    // experts of up to 4 GiB a matrix; byte offsets and numbers of (token, rank) pairs times columns
    // are 32-bit; one launch covers all experts
    if ((double)(I + 256) * (double)H >= 8589934592.0) return LB_ERR_OVERFLOW;
    const int64_t tokens = std::min<int64_t>(T, lb::MOE_TOKENS);
    if (tokens * top_k * I * 4 >= (int64_t)0xFFFF0000 || tokens * top_k * H >= kLim) return LB_ERR_OVERFLOW;
    if (std::min(tokens * top_k, E) * (std::max(I, H) / 16 + 1) * ((tokens + 15) / 16) * 512 > lb::LAUNCH_THREADS)
        return LB_ERR_OVERFLOW;
    return LB_OK;
}

struct MoeSpace {
    int64_t lists, h, y, bytes;
};
MoeSpace moe_space(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top_k)
{
    const int64_t tokens = std::min<int64_t>(T, lb::MOE_TOKENS);
    MoeSpace m;
    m.lists = round_up(tokens * E * 4, 256);   // (the logits come first)
    m.h = m.lists + round_up((1 + std::min(tokens * top_k, E) * (2 + lb::MOE_TOKENS)) * 4, 256);
    m.y = m.h + round_up(tokens * top_k * I * 4, 256);
    m.bytes = m.y + round_up(tokens * top_k * H * 4, 256);
    return m;
}

}  // namespace

extern "C" {

int lb_residual_norm(const void *Y, int64_t ldy, const void *R, int64_t ldr, const void *post_w, const void *gate,
                     int64_t ldg, const void *w, void *R_out, int64_t ldro, void *X, int64_t ldx, int64_t M,
                     int64_t H, float alpha, float eps, int ftype, int rtype, void *stream)
{
    if ((!Y && !R) || (!R_out && !X) || (X && !w) || (!Y && (post_w || gate))) return LB_ERR_NULL;
    if (M <= 0 || H <= 0 || M > kLim || (Y && ldy < H) || (R && ldr < H) || (gate && ldg != 0 && ldg < H) ||
        (R_out && ldro < H) || (X && ldx < H))
        return LB_ERR_SHAPE;
    // in place: the same rows
    if ((R_out && R_out == R && ldro != ldr) || (X && X == Y && ldx != ldy)) return LB_ERR_SHAPE;
    if (H % 8 != 0) return LB_ERR_ALIGN;
    if (!any_ftype(ftype) || (rtype != ftype && rtype != LB_F32)) return LB_ERR_VARIANT;
    if (H > LB_NORM_H_MAX) return LB_ERR_OVERFLOW;
    if (!aligned(Y) || !aligned(R) || !aligned(post_w) || !aligned(gate) || !aligned(w) || !aligned(R_out) || !aligned(X) ||
        (Y && !rows_aligned(ldy, ftype)) || (R && !rows_aligned(ldr, rtype)) || (gate && !rows_aligned(ldg, ftype)) ||
        (R_out && !rows_aligned(ldro, rtype)) || (X && !rows_aligned(ldx, ftype)))
        return LB_ERR_ALIGN;
    lb::NormArgs a;
    a.y = Y;
    a.r = R;
    a.post_w = post_w;
    a.gate = gate;
    a.w = w;
    a.r_out = R_out;
    a.x = X;
    a.ldy = ldy;
    a.ldr = ldr;
    a.ldg = ldg;
    a.ldro = ldro;
    a.ldx = ldx;
    a.H = (int32_t)H;
    a.alpha = alpha;
    a.eps = eps;
    return finish(lb::launch_residual_norm(ftype, rtype, a, M, (hipStream_t)stream));
}

int lb_rope_freqs(double *freqs, float *mult, int64_t R, double base, int scaling, double factor, double before,
                  double low, double high)
{
    if (!freqs || !mult) return LB_ERR_NULL;
    if (R <= 0 || R % 2 != 0 || R > LB_ROPE_R_MAX || !(base > 1.0)) return LB_ERR_SHAPE;
    if (scaling < LB_ROPE_PLAIN || scaling > LB_ROPE_BANDS) return LB_ERR_VARIANT;
    if (scaling != LB_ROPE_PLAIN && !(factor > 0.0)) return LB_ERR_SHAPE;
    if (scaling >= LB_ROPE_PARTS && (!(before > 0.0) || !(low > 0.0) || !(high > low))) return LB_ERR_SHAPE;
    const double turn = 6.283185307179586477;
    if (scaling == LB_ROPE_BASE && R > 2) base *= std::pow(factor, (double)R / (double)(R - 2));
    *mult = 1.0f;
    double first = 0.0, last = 0.0;
    if (scaling == LB_ROPE_PARTS) {
        // pair (fractional) that turns n times in `before` positions
        auto pair_of = [&](double n) { return (double)R * std::log(before / (n * turn)) / (2.0 * std::log(base)); };
        first = std::max(std::floor(pair_of(high)), 0.0);
        last = std::min(std::ceil(pair_of(low)), (double)(R - 1));
        if (last <= 0.0) first = last = -1.0;   // no pair turns more than `low` times
        if (factor > 1.0) *mult = (float)(0.1 * std::log(factor) + 1.0);
    }
    for (int64_t i = 0; i < R / 2; ++i) {
        const double f = std::pow(base, -2.0 * (double)i / (double)R);
        double keep = 1.0;   // share of the frequency that is not stretched
        if (scaling == LB_ROPE_LINEAR) keep = 0.0;
        if (scaling == LB_ROPE_PARTS)
            keep = 1.0 - std::min(std::max(((double)i - first) / std::max(last - first, 0.001), 0.0), 1.0);
        if (scaling == LB_ROPE_BANDS)
            keep = std::min(std::max((before * f / turn - low) / (high - low), 0.0), 1.0);
        freqs[i] = scaling == LB_ROPE_PLAIN || scaling == LB_ROPE_BASE ? f : f / factor * (1.0 - keep) + f * keep;
    }
    return LB_OK;
}

int lb_rope(const void *Q, int64_t ldq, const void *K, int64_t ldk, const int64_t *pos, const double *freqs,
            void *Q_out, int64_t ldqo, void *K_out, int64_t ldko, int64_t T, int64_t Hq, int64_t Hk, int64_t D,
            int64_t R, int layout, float mult, int ftype, void *stream)
{
    if (!Q || !pos || !freqs || !Q_out || (Hk > 0 && (!K || !K_out))) return LB_ERR_NULL;
    if (T <= 0 || Hq <= 0 || Hk < 0 || D <= 0 || R <= 0 || T > kLim || Hq > 65535 || Hk > 65535 || R > D ||
        D > LB_ROPE_R_MAX || ldq < Hq * D || ldqo < Hq * D || ldk < Hk * D || ldko < Hk * D)
        return LB_ERR_SHAPE;
    // in place: the same rows
    if ((Q == Q_out && ldq != ldqo) || (Hk > 0 && K == K_out && ldk != ldko)) return LB_ERR_SHAPE;
    if (D % 8 != 0 || R % 16 != 0) return LB_ERR_ALIGN;
    if (!any_ftype(ftype) || (layout != LB_ROPE_HALF && layout != LB_ROPE_PAIRS)) return LB_ERR_VARIANT;
    if (!aligned(Q) || !aligned(Q_out) || !rows_aligned(ldq, ftype) || !rows_aligned(ldqo, ftype) ||
        (Hk > 0 && (!aligned(K) || !aligned(K_out) || !rows_aligned(ldk, ftype) || !rows_aligned(ldko, ftype))))
        return LB_ERR_ALIGN;
    lb::RopeArgs a;
    a.q = Q;
    a.k = Hk ? K : nullptr;
    a.qo = Q_out;
    a.ko = Hk ? K_out : nullptr;
    a.pos = pos;
    a.freqs = freqs;
    a.ldq = ldq;
    a.ldk = ldk;
    a.ldqo = ldqo;
    a.ldko = ldko;
    a.T = T;
    a.Hq = (int32_t)Hq;
    a.Hk = (int32_t)Hk;
    a.D = (int32_t)D;
    a.R = (int32_t)R;
    a.mult = mult;
    const bool in_place = Q == Q_out && (Hk == 0 || K == K_out);
    return finish(lb::launch_rope(ftype, a, layout == LB_ROPE_PAIRS, in_place, cu_count(), (hipStream_t)stream));
}

int64_t lb_linear_w4_workspace(int64_t M, int64_t K, int64_t N, int64_t group)
{
    if (check_w4(M, N, K, group, LB_BF16) != LB_OK || M <= lb::W4_FEW_ROWS) return 0;
    return lb::linear_w4_rows_workspace(M, N, K, group, cu_count());
}

int lb_linear_w4(const void *X, int64_t ldx, const uint8_t *W, const void *Wp, const void *bias, void *out, int64_t M,
                 int64_t N, int64_t K, int64_t group, int ftype, void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!X || !W || !Wp || !out) return LB_ERR_NULL;
    if (ldx < K) return LB_ERR_SHAPE;
    const int st = check_w4(M, N, K, group, ftype);
    if (st != LB_OK) return st;
    if (!aligned(X) || !aligned(W) || !aligned(Wp) || !aligned(bias) || !aligned(out) || !rows_aligned(ldx, ftype))
        return LB_ERR_ALIGN;
    if (ldx > kLdMax) return LB_ERR_OVERFLOW;
    const int64_t need = lb_linear_w4_workspace(M, K, N, group);
    if (need > 0 && (!workspace || workspace_bytes < need)) return LB_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return LB_ERR_ALIGN;
    lb::W4Args a;
    a.x = X;
    a.ldx = ldx;
    a.w = W;
    a.p = Wp;
    a.bias = bias;
    a.out = out;
    a.M = M;
    a.N = N;
    a.K = K;
    if (need > 0) return finish(lb::launch_linear_w4_rows(ftype, (int)group, a, cu_count(), workspace, (hipStream_t)stream));
    return finish(lb::launch_linear_w4(ftype, (int)group, a, cu_count(), (hipStream_t)stream));
}

int64_t lb_moe_w4_workspace(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top_k)
{
    if (check_moe(T, H, I, E, top_k, 32, LB_BF16) != LB_OK) return 0;
    return moe_space(T, H, I, E, top_k).bytes;
}

int lb_moe_w4(const void *X, int64_t ldx, const void *Wr, const uint8_t *W1, const void *P1, const uint8_t *W2,
              const void *P2, void *out, int32_t *ids, float *weights, int64_t T, int64_t H, int64_t I, int64_t E,
              int64_t top_k, int64_t group, int renorm, float scale, int ftype, void *workspace,
              int64_t workspace_bytes, void *stream)
{
    if (!X || !Wr || !W1 || !P1 || !W2 || !P2 || !out) return LB_ERR_NULL;
    if (ldx < H) return LB_ERR_SHAPE;
    const int st = check_moe(T, H, I, E, top_k, group, ftype);
    if (st != LB_OK) return st;
    if (!aligned(X) || !aligned(Wr) || !aligned(W1) || !aligned(P1) || !aligned(W2) || !aligned(P2) || !aligned(out) ||
        !rows_aligned(ldx, ftype))
        return LB_ERR_ALIGN;
    if (ldx > kLdMax) return LB_ERR_OVERFLOW;
    const MoeSpace m = moe_space(T, H, I, E, top_k);
    if (!workspace || workspace_bytes < m.bytes) return LB_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return LB_ERR_ALIGN;
    const int cu = cu_count();
    for (int64_t t = 0; t < T; t += lb::MOE_TOKENS) {
        lb::MoeArgs a;
        a.x = (const char *)X + t * ldx * 2;
        a.ldx = ldx;
        a.wr = Wr;
        a.w1 = W1;
        a.w2 = W2;
        a.p1 = P1;
        a.p2 = P2;
        a.out = (char *)out + t * H * 2;
        a.ids = ids ? ids + t * top_k : nullptr;
        a.weights = weights ? weights + t * top_k : nullptr;
        a.T = (int32_t)std::min<int64_t>(T - t, lb::MOE_TOKENS);
        a.E = (int32_t)E;
        a.top_k = (int32_t)top_k;
        a.H = (int32_t)H;
        a.I = (int32_t)I;
        a.renorm = renorm != 0;
        a.scale = scale;
        a.logits = (float *)workspace;
        a.found = (int32_t *)((char *)workspace + m.lists);
        a.lists = a.found + 1;
        a.h = (float *)((char *)workspace + m.h);
        a.y = (float *)((char *)workspace + m.y);
        const hipError_t e = lb::launch_moe_w4(ftype, (int)group, a, cu, (hipStream_t)stream);
        if (e != hipSuccess) return LB_ERR_HIP;
    }
    return LB_OK;
}

}  // extern "C"
