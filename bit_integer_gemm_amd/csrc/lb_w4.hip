// lb_w4.hip -- linear layer with 4-bit weights and group scales on 16-bit activations.
//
//   out[m,n] = round(sum_k x[m,k] (u[n,k] s[n,g] + b[n,g]) + bias[n]),  g = k / G
#include "lb_internal.hpp"
#include "lb_w4.hpp"

namespace lb {

// Few rows: a workgroup takes 16 MT rows of x against some tiles of 16 columns (W4Split).
struct FewArgs {
    const uint8_t *w;
    const uint32_t *p;
    int64_t ldx;
    int32_t M, N, K;
    int32_t kw, each;        // W4Split
    uint32_t tiles_m, tiles_n;   // workgroups
};
template <class T, int MT, int G, bool XLDS, int DEPTH>
__global__ __launch_bounds__(64 * W4_WAVES) void w4_few_kernel(const T *__restrict__ X, const T *__restrict__ bias,
                                                               T *__restrict__ out, FewArgs a)
{
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int32_t lane = (int32_t)(threadIdx.x & 63u);
    const int32_t wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    uint32_t tm, tn;
    tile_of_block(blockIdx.x, a.tiles_m, a.tiles_n, 4u, tm, tn);
    const int32_t m0 = (int32_t)tm * 16 * MT, rows = min(16 * MT, a.M - m0);
    const int32_t per = W4_WAVES / a.kw * a.each, t0 = (int32_t)tn * per;   // the workgroup's tiles
    const int32_t have = min(per, (a.N + 15) / 16 - t0);
    const int32_t lines = (a.K + 255) / 256, share = wave % a.kw, mine = wave / a.kw * a.each;
    const uint32_t stride = w4_x_stride(a.K);
    float *const slots = (float *)(smem + (XLDS ? (uint32_t)rows * stride : 0u));
    const int32_t slot = rows * W4_SLOT_LD;
    uint32_t xat[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const uint32_t row = (uint32_t)min(16 * m + (lane & 15), rows - 1);
        xat[m] = XLDS ? row * stride : row * (uint32_t)a.ldx * 2u;
    }
    const T *const x0 = X + (int64_t)m0 * a.ldx;
    auto row_at = [&](int32_t row) { return x0 + row * a.ldx; };
    W4Stage<decltype(row_at)> stage(smem, a.K, rows, 64 * W4_WAVES, row_at);
    if constexpr (XLDS) stage.first();
    w4_stream<T, T, MT, G, 1, XLDS, DEPTH>(
        a.w, a.p, a.K, share * lines / a.kw, (share + 1) * lines / a.kw, max(0, min(a.each, have - mine)),
        w4_rsrc(x0, 0xFFFFFFF0u), smem, xat, 0u,
        [&](int32_t t) { return W4Tile{(int64_t)(t0 + mine + t) * 16, min(16, a.N - (t0 + mine + t) * 16)}; },
        [&] {
            if constexpr (XLDS) stage.rest();
        },
        [&](int32_t t, const f32x4(&acc)[MT]) { w4_put<MT>(slots + (wave * a.each + t) * slot, rows, acc); });
    __syncthreads();
    for (int32_t i = (int32_t)threadIdx.x; i < rows * have * 16; i += 64 * W4_WAVES) {
        const int32_t m = i / (have * 16), c = i - m * have * 16, t = c / 16, n = t0 * 16 + c;
        if (n >= a.N) continue;
        // tile t: the waves of group t / each, in order
        const float *s = slots + (t / a.each * a.kw * a.each + t % a.each) * slot + m * W4_SLOT_LD + c % 16;
        float v = 0.f;
        for (int32_t k = 0; k < a.kw; ++k)
            if (k * lines / a.kw < (k + 1) * lines / a.kw) v += s[k * a.each * slot];
        if (bias) v += (float)bias[n];
        out[(int64_t)(m0 + m) * a.N + n] = (T)v;
    }
}

enum { FEW_LDS = 160 * 1024 };
template <class T, int MT, int G, bool XLDS>
static hipError_t w4_few_t(const W4Args &a, int64_t rows, const W4Split &sp, hipStream_t s)
{
    const int64_t per = (int64_t)(W4_WAVES / sp.kw) * sp.each, tn = ((a.N + 15) / 16 + per - 1) / per;
    const int64_t most = LAUNCH_THREADS / (64 * W4_WAVES) / tn * 16 * MT;   // rows of one launch
    const uint32_t lds = (uint32_t)((XLDS ? rows * w4_x_stride((int32_t)a.K) : 0) + W4_WAVES * sp.each * rows * W4_SLOT_LD * 4);
    if (most < 16 * MT || lds > FEW_LDS) return hipErrorInvalidValue;
    for (int64_t m = 0; m < a.M; m += most) {
        const int64_t here = a.M - m < most ? a.M - m : most, tm = (here + 16 * MT - 1) / (16 * MT);
        const FewArgs f{a.w, (const uint32_t *)a.p, a.ldx, (int32_t)here, (int32_t)a.N, (int32_t)a.K, sp.kw, sp.each,
                        (uint32_t)tm, (uint32_t)tn};
        hipLaunchKernelGGL((w4_few_kernel<T, MT, G, XLDS, 3>), dim3((uint32_t)(tm * tn)), dim3(64 * W4_WAVES), lds, s,
                           (const T *)a.x + m * a.ldx, (const T *)a.bias, (T *)a.out + m * a.N, f);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class T, int G> static hipError_t w4_g(const W4Args &a, int cu, hipStream_t s)
{
    const int64_t tiles = (a.N + 15) / 16, lines = (a.K + 255) / 256;
    const int mt = a.M <= 16 ? 1 : 2;
    const int64_t rows = a.M < 16 * mt ? a.M : 16 * mt, passes = (a.M + 16 * mt - 1) / (16 * mt);
    int64_t per = (tiles * passes + cu - 1) / cu;
    if (per > 8) per = 8;
    const W4Split sp = w4_split(per, lines);
    const bool xlds = rows * w4_x_stride((int32_t)a.K) + W4_WAVES * sp.each * rows * W4_SLOT_LD * 4 <= FEW_LDS;
    if (mt == 1) return xlds ? w4_few_t<T, 1, G, true>(a, rows, sp, s) : w4_few_t<T, 1, G, false>(a, rows, sp, s);
    return xlds ? w4_few_t<T, 2, G, true>(a, rows, sp, s) : w4_few_t<T, 2, G, false>(a, rows, sp, s);
}

template <class T> static hipError_t w4_t(const W4Args &a, int group, int cu, hipStream_t s)
{
    return group == 32 ? w4_g<T, 32>(a, cu, s) : group == 64 ? w4_g<T, 64>(a, cu, s) : w4_g<T, 128>(a, cu, s);
}

hipError_t launch_linear_w4(int ftype, int group, const W4Args &a, int cu, hipStream_t s)
{
    switch (ftype) {
    case LB_BF16: return w4_t<__bf16>(a, group, cu, s);
    case LB_F16: return w4_t<_Float16>(a, group, cu, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace lb
