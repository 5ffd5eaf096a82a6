// lb_w4.hip -- linear layer with 4-bit weights and group scales on 16-bit activations.
//
//   out[m,n] = round(sum_k x[m,k] (u[n,k] s[n,g] + b[n,g]) + bias[n]),  g = k / G
#include "lb_internal.hpp"
#include "lb_w4.hpp"

namespace lb {

// A tile of 16 NT columns and 16 MT rows to a workgroup, a share of K to each wave.
template <class T, int MT, int NT, int NW, int G>
__global__ __launch_bounds__(64 * NW) void w4_few_kernel(const T *__restrict__ X, int64_t ldx,
                                                         const uint8_t *__restrict__ W, const uint32_t *__restrict__ P,
                                                         const T *__restrict__ bias, T *__restrict__ out, int32_t M,
                                                         int32_t N, int32_t K, uint32_t tiles_m, uint32_t tiles_n)
{
    typedef W4Join<MT, NT, NW> Join;
    __shared__ float sums[Join::FLOATS];
    const int32_t lane = (int32_t)(threadIdx.x & 63u);
    const int32_t wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    uint32_t tm, tn;
    tile_of_block(blockIdx.x, tiles_m, tiles_n, 4u, tm, tn);
    const int32_t m0 = (int32_t)tm * 16 * MT, n0 = (int32_t)tn * 16 * NT;
    const int32_t rows = min(16 * NT, N - n0), lines = (K + 255) / 256;
    const T *xrow[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) xrow[m] = X + (int64_t)min(m0 + 16 * m + (lane & 15), M - 1) * ldx;
    f32x4 acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    w4_product<T, T, MT, NT, G>(W + (int64_t)n0 * (K / 2), (uint64_t)rows * (uint32_t)(K / 2), P + (int64_t)n0 * (K / G),
                             (uint64_t)rows * (uint32_t)(K / G) * 4u, K, 16, wave * lines / NW, (wave + 1) * lines / NW,
                             xrow, 0, acc);
    Join::put(sums, wave, acc);
    __syncthreads();
    for (int32_t i = (int32_t)threadIdx.x; i < 256 * MT * NT; i += 64 * NW) {
        const int32_t m = i / (16 * NT), n = i % (16 * NT);
        if (m0 + m >= M || n0 + n >= N) continue;
        float v = Join::sum(sums, m, n);
        if (bias) v += (float)bias[n0 + n];
        out[(int64_t)(m0 + m) * N + n0 + n] = (T)v;
    }
}

template <class T, int MT, int NT, int NW, int G>
static hipError_t w4_few_t(const W4Args &a, hipStream_t s)
{
    const int64_t tn = (a.N + 16 * NT - 1) / (16 * NT);
    const int64_t most = LAUNCH_THREADS / (64 * NW) / tn * 16 * MT;   // rows of one launch
    if (most < 16 * MT) return hipErrorInvalidValue;
    for (int64_t m = 0; m < a.M; m += most) {
        const int64_t rows = a.M - m < most ? a.M - m : most, tm = (rows + 16 * MT - 1) / (16 * MT);
        hipLaunchKernelGGL((w4_few_kernel<T, MT, NT, NW, G>), dim3((uint32_t)(tm * tn)), dim3(64 * NW), 0, s,
                           (const T *)a.x + m * a.ldx, a.ldx, a.w, (const uint32_t *)a.p, (const T *)a.bias,
                           (T *)a.out + m * a.N, (int32_t)rows, (int32_t)a.N, (int32_t)a.K, (uint32_t)tm, (uint32_t)tn);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class T, int G> static hipError_t w4_g(const W4Args &a, hipStream_t s)
{
    if (a.M <= 16) return w4_few_t<T, 1, 1, 8, G>(a, s);
    if (a.M <= 32) return w4_few_t<T, 2, 1, 8, G>(a, s);
    return w4_few_t<T, 4, 2, 4, G>(a, s);
}

template <class T> static hipError_t w4_t(const W4Args &a, int group, hipStream_t s)
{
    return group == 32 ? w4_g<T, 32>(a, s) : group == 64 ? w4_g<T, 64>(a, s) : w4_g<T, 128>(a, s);
}

hipError_t launch_linear_w4(int ftype, int group, const W4Args &a, hipStream_t s)
{
    switch (ftype) {
    case LB_BF16: return w4_t<__bf16>(a, group, s);
    case LB_F16: return w4_t<_Float16>(a, group, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace lb
