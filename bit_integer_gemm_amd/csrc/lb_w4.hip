// lb_w4.hip -- linear layer with 4-bit weights and group scales on 16-bit activations.
//
//   out[m,n] = round(sum_k x[m,k] (u[n,k] s[n,g] + b[n,g]) + bias[n]),  g = k / G
#include "lb_internal.hpp"
#include "lb_w4.hpp"

namespace lb {

// Up to 16 rows: a workgroup takes all of x against some tiles of 16 columns (W4Split).
// EARLY: weights are asked for before x (a row or two of x are there before the first weights).
struct FewArgs {
    const uint8_t *w;
    const uint32_t *p;
    int64_t ldx;
    int32_t M, N, K;
    W4Split sp;
};
template <class T, int G, bool EARLY>
__global__ __launch_bounds__(64 * W4_WAVES) void w4_few_kernel(const T *__restrict__ X, const T *__restrict__ bias,
                                                                  T *__restrict__ out, FewArgs a)
{
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    const int32_t wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), rows = a.M;
    const int32_t kw = a.sp.kw, each = a.sp.each;
    const int32_t per = W4_WAVES / kw * each, t0 = (int32_t)blockIdx.x * per;   // the workgroup's tiles
    const int32_t have = min(per, (a.N + 15) / 16 - t0), mine = wave / kw * each;
    float *const slots = (float *)(smem + W4Lds<G>::x_bytes(rows, a.sp.chunk) + W4Lds<G>::RINGS);
    const int32_t slot = rows * W4_SLOT_LD;
    auto tile_at = [&](int32_t t) { return W4Tile{(int64_t)(t0 + mine + t) * 16, min(16, a.N - (t0 + mine + t) * 16)}; };
    W4Flow<T, T, G, 1, false, decltype(tile_at)> flow(smem, W4Lds<G>::x_bytes(rows, a.sp.chunk), a.w, a.p, a.K, a.sp,
                                               max(0, min(each, have - mine)), tile_at);
    if constexpr (EARLY) flow.start();
    flow.template run<EARLY, false>(
        rows, make_rsrc(X, 0xFFFFFFF0u), [&](int32_t row) { return (uint32_t)row * (uint32_t)a.ldx * 2u; },
        [&](int32_t t, const f32x4 &acc, bool more) { w4_put(slots + (wave * each + t) * slot, rows, acc, more); });
    __syncthreads();
    for (int32_t i = (int32_t)threadIdx.x; i < rows * have * 16; i += 64 * W4_WAVES) {
        const int32_t m = i / (have * 16), c = i - m * have * 16, t = c / 16, n = t0 * 16 + c;
        if (n >= a.N) continue;
        // tile t: the waves of group t / each, in order
        const float *s = slots + (t / each * kw * each + t % each) * slot + m * W4_SLOT_LD + c % 16;
        float v = 0.f;
        for (int32_t k = 0; k < kw; ++k) v += s[k * each * slot];
        if (bias) v += (float)bias[n];
        out[(int64_t)m * a.N + n] = (T)v;
    }
}

enum { FEW_LDS = 160 * 1024 };
template <class T, int G> static hipError_t w4_g(const W4Args &a, int cu, hipStream_t s)
{
    const int64_t tiles = (a.N + 15) / 16, lines = (a.K + 255) / 256;
    // a workgroup to a compute unit, if its sums find room
    int64_t per = (tiles + cu - 1) / cu;
    const int64_t slot = a.M * W4_SLOT_LD * 4, room = 24 * 1024 / (W4_WAVES * slot);
    if (per > room) per = room > 1 ? room : 1;
    const W4Split sp = w4_split(per, lines, a.M, FEW_LDS - 4096 - W4Lds<G>::RINGS - W4_WAVES * per * slot);
    const int64_t wide = (int64_t)(W4_WAVES / sp.kw) * sp.each, wgs = (tiles + wide - 1) / wide;
    const uint32_t lds = W4Lds<G>::x_bytes((int32_t)a.M, sp.chunk) + W4Lds<G>::RINGS + (uint32_t)(W4_WAVES * sp.each * slot);
    if (a.M > W4_FEW_ROWS || wgs * 64 * W4_WAVES > LAUNCH_THREADS || lds > FEW_LDS) return hipErrorInvalidValue;
    const FewArgs f{a.w, (const uint32_t *)a.p, a.ldx, (int32_t)a.M, (int32_t)a.N, (int32_t)a.K, sp};
    const dim3 grid((uint32_t)wgs), block(64 * W4_WAVES);
    const T *x = (const T *)a.x, *bias = (const T *)a.bias;
    if (a.M > 2) hipLaunchKernelGGL((w4_few_kernel<T, G, true>), grid, block, lds, s, x, bias, (T *)a.out, f);
    else hipLaunchKernelGGL((w4_few_kernel<T, G, false>), grid, block, lds, s, x, bias, (T *)a.out, f);
    return hipGetLastError();
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
