// lb_serve_linear.hip -- int8 linear layer on floating activations: each token's row
// quantised by its own largest magnitude, and the product for few tokens.
//
//   amax[m] = max_k |x[m,k]|,  sx[m] = amax[m] / 127
//   q[m,k]  = round_half_even(127 x[m,k] / amax[m])            (int8)
//   out[m,n] = round((float(sum_k q[m,k] W[n,k]) sx[m]) sw[n] + bias[n])
//
// The sum is exact in int32; the scales, the product and the bias are fp32, and
// there is one rounding to the output type.
#include "lb_float.hpp"
#include "lb_internal.hpp"

namespace lb {

// ---- row quantisation ------------------------------------------------------
// The quotient that decides q is compared with half-integers, so it is formed
// twice: t = x * (127/amax) in fp32 is off by at most 127 * 2^-23 < 2^-16, which
// settles q unless t lies within 2^-13 of a half-integer; there the double
// quotient decides (exact for every 24-bit x and amax: a quotient that is not a
// half-integer differs from one by at least 2^-32 of its size).
__device__ inline int quant_s8(float x, float inv, float amax, bool direct)
{
    const float t = x * inv, n = __builtin_rintf(t);
    if (direct || __builtin_fabsf(t - n) > 0.5f - 0x1p-13f)
        return (int)__builtin_rint((double)x * 127.0 / (double)amax);
    return (int)n;
}

// Row scale of a largest magnitude given as fp32 bits.  direct: 127/amax may
// overflow, every quotient is formed in double.  A row that holds an infinity
// or a NaN gets that as its scale and q = 0, so that its outputs are NaN; a row
// of zeros gets scale 0 and q = 0.
struct RowScale {
    float amax, inv, scale;
    bool zero, direct;
};
__device__ inline RowScale row_scale(uint32_t amax_bits)
{
    RowScale r;
    r.amax = __uint_as_float(amax_bits);
    r.scale = r.amax / 127.0f;
    r.zero = amax_bits == 0 || amax_bits >= 0x7F800000u;
    r.direct = r.amax < 0x1p-100f;
    r.inv = r.zero ? 0.f : 127.0f / r.amax;
    return r;
}

// Magnitude bits of the 16 bytes at a chunk, widened to fp32 (NaN orders above
// infinity above every number, so an integer maximum keeps both).
template <class T> __device__ inline uint32_t chunk_amax(i32x4 c)
{
    if constexpr (sizeof(T) == 4) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, (uint32_t)c[i] & 0x7FFFFFFFu);
        return m;
    } else {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, max((uint32_t)c[i] & 0x7FFFu, ((uint32_t)c[i] >> 16) & 0x7FFFu));
        return m;
    }
}
template <class T> __device__ inline uint32_t widen_bits(uint32_t m)
{
    if constexpr (sizeof(T) == 4) return m;
    else if constexpr (__is_same(T, __bf16)) return m << 16;
    else return __float_as_uint(lo_f32<_Float16>(m));
}

// One workgroup per row; EPT elements per 16-byte chunk.  The row is read once
// if it fits the workgroup's registers (NC chunks per thread), else twice.
template <class T, int NC>
__global__ __launch_bounds__(256) void quant_rows_kernel(const T *__restrict__ X, int64_t ldx,
                                                         int8_t *__restrict__ Q, float *__restrict__ sx,
                                                         int32_t K)
{
    constexpr int EPT = 16 / sizeof(T);
    __shared__ uint32_t red[4];
    const int64_t m = blockIdx.x;
    const T *row = X + m * ldx;
    int8_t *q = Q + m * (int64_t)K;
    const int32_t chunks = K / EPT;
    i32x4 keep[NC];
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int32_t c = (int32_t)threadIdx.x + 256 * i;
        keep[i] = i32x4{0, 0, 0, 0};
        if (c < chunks) keep[i] = *(const i32x4 *)(row + (int64_t)c * EPT);
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) mx = max(mx, chunk_amax<T>(keep[i]));
    for (int32_t c = (int32_t)threadIdx.x + 256 * NC; c < chunks; c += 256)
        mx = max(mx, chunk_amax<T>(*(const i32x4 *)(row + (int64_t)c * EPT)));
#pragma unroll
    for (int d = 32; d; d >>= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, d));
    if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = mx;
    __syncthreads();
    mx = max(max(red[0], red[1]), max(red[2], red[3]));
    const RowScale rs = row_scale(widen_bits<T>(mx));
    if (threadIdx.x == 0) sx[m] = rs.scale;

    auto put = [&](int32_t c, i32x4 v) {
        uint32_t b[EPT / 4];
#pragma unroll
        for (int i = 0; i < EPT / 4; ++i) {
            float x[4];
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = __int_as_float(v[e]);
            } else {
                x[0] = lo_f32<T>((uint32_t)v[2 * i]);
                x[1] = hi_f32<T>((uint32_t)v[2 * i]);
                x[2] = lo_f32<T>((uint32_t)v[2 * i + 1]);
                x[3] = hi_f32<T>((uint32_t)v[2 * i + 1]);
            }
            uint32_t w = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int n = rs.zero ? 0 : quant_s8(x[e], rs.inv, rs.amax, rs.direct);
                w |= ((uint32_t)n & 0xFFu) << (8 * e);
            }
            b[i] = w;
        }
        if constexpr (EPT == 8) *(u32x2 *)(q + (int64_t)c * 8) = u32x2{b[0], b[1]};
        else *(uint32_t *)(q + (int64_t)c * 4) = b[0];
    };
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int32_t c = (int32_t)threadIdx.x + 256 * i;
        if (c < chunks) put(c, keep[i]);
    }
    for (int32_t c = (int32_t)threadIdx.x + 256 * NC; c < chunks; c += 256)
        put(c, *(const i32x4 *)(row + (int64_t)c * EPT));
}

template <class T>
static hipError_t quant_rows_t(const void *X, int64_t ldx, int8_t *Q, float *sx, int64_t M, int64_t K,
                               hipStream_t s)
{
    const int64_t per = 256 * (16 / (int64_t)sizeof(T));  // elements a workgroup holds per chunk
    const dim3 grid((uint32_t)M), block(256);
    if (K <= per)
        hipLaunchKernelGGL((quant_rows_kernel<T, 1>), grid, block, 0, s, (const T *)X, ldx, Q, sx, (int32_t)K);
    else if (K <= 2 * per)
        hipLaunchKernelGGL((quant_rows_kernel<T, 2>), grid, block, 0, s, (const T *)X, ldx, Q, sx, (int32_t)K);
    else
        hipLaunchKernelGGL((quant_rows_kernel<T, 6>), grid, block, 0, s, (const T *)X, ldx, Q, sx, (int32_t)K);
    return hipGetLastError();
}

hipError_t launch_quant_rows(int ftype, const void *X, int64_t ldx, int8_t *Q, float *sx, int64_t M,
                             int64_t K, hipStream_t s)
{
    switch (ftype) {
    case LB_BF16: return quant_rows_t<__bf16>(X, ldx, Q, sx, M, K, s);
    case LB_F16: return quant_rows_t<_Float16>(X, ldx, Q, sx, M, K, s);
    case LB_F32: return quant_rows_t<float>(X, ldx, Q, sx, M, K, s);
    default: return hipErrorInvalidValue;
    }
}

// ---- few tokens ------------------------------------------------------------
// 16 output channels per workgroup, all of K: wave w takes every NW-th block of
// 128 K-bytes, and the waves' exact partial sums meet in LDS.  The weight is the
// MFMA's A operand (lane l: channel l%16, K bytes 32*(l/16) .. +31 of the block,
// so the four lane groups read one whole 128-byte line of each row), the tokens
// its B operand with the same K order; lane l ends with channels 4*(l/16) .. +3
// of token l%16.
template <class T, int MT>
__global__ __launch_bounds__(512) void linear_few_kernel(
    const int8_t *__restrict__ Xq, const int8_t *__restrict__ W, const float *__restrict__ sx,
    const float *__restrict__ sw, const T *__restrict__ bias, T *__restrict__ out, int32_t M, int32_t N,
    int32_t K)
{
    constexpr int NW = 8;
    __shared__ i32x4 part[NW][MT][64];
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int32_t r = (int32_t)(lane & 15u), c = (int32_t)(lane >> 4);
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int8_t *wrow = W + min(n0 + r, (int64_t)N - 1) * K + 32 * c;
    const int8_t *xrow[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) xrow[t] = Xq + (int64_t)min(16 * t + r, M - 1) * K + 32 * c;

    i32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = i32x4{0, 0, 0, 0};
    const int32_t full = K / 128;
    for (int32_t b = (int32_t)wave; b < full; b += NW) {
        const i32x4 w0 = *(const i32x4 *)(wrow + b * 128), w1 = *(const i32x4 *)(wrow + b * 128 + 16);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const i32x4 x0 = *(const i32x4 *)(xrow[t] + b * 128), x1 = *(const i32x4 *)(xrow[t] + b * 128 + 16);
            acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w0, x0, acc[t], 0, 0, 0);
            acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w1, x1, acc[t], 0, 0, 0);
        }
    }
    if (K % 128 != 0 && (int32_t)wave == full % NW) {
        // the last, partial block: 16-byte pieces past K are not read and count as 0
        const i32x4 zero = {0, 0, 0, 0};
        const bool in0 = full * 128 + 32 * c < K, in1 = full * 128 + 32 * c + 16 < K;
        const i32x4 w0 = in0 ? *(const i32x4 *)(wrow + full * 128) : zero;
        const i32x4 w1 = in1 ? *(const i32x4 *)(wrow + full * 128 + 16) : zero;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const i32x4 x0 = in0 ? *(const i32x4 *)(xrow[t] + full * 128) : zero;
            const i32x4 x1 = in1 ? *(const i32x4 *)(xrow[t] + full * 128 + 16) : zero;
            acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w0, x0, acc[t], 0, 0, 0);
            acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w1, x1, acc[t], 0, 0, 0);
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) part[wave][t][lane] = acc[t];
    __syncthreads();
    if (wave >= MT) return;
    i32x4 sum = part[0][wave][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) sum += part[w][wave][lane];
    const int32_t m = 16 * (int32_t)wave + r;
    if (m >= M) return;
    const float scale = sx[m];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int64_t n = n0 + 4 * c + e;
        if (n < N) {
            float y = ((float)sum[e] * scale) * sw[n];
            if (bias) y += (float)bias[n];
            out[m * (int64_t)N + n] = (T)y;
        }
    }
}

template <class T>
static hipError_t linear_few_t(const int8_t *Xq, const int8_t *W, const float *sx, const float *sw,
                               const void *bias, void *out, int64_t M, int64_t N, int64_t K, hipStream_t s)
{
    const dim3 grid((uint32_t)((N + 15) / 16)), block(512);
    if (M <= 16)
        hipLaunchKernelGGL((linear_few_kernel<T, 1>), grid, block, 0, s, Xq, W, sx, sw, (const T *)bias, (T *)out,
                           (int32_t)M, (int32_t)N, (int32_t)K);
    else if (M <= 32)
        hipLaunchKernelGGL((linear_few_kernel<T, 2>), grid, block, 0, s, Xq, W, sx, sw, (const T *)bias, (T *)out,
                           (int32_t)M, (int32_t)N, (int32_t)K);
    else
        hipLaunchKernelGGL((linear_few_kernel<T, 4>), grid, block, 0, s, Xq, W, sx, sw, (const T *)bias, (T *)out,
                           (int32_t)M, (int32_t)N, (int32_t)K);
    return hipGetLastError();
}

hipError_t launch_linear_few(int ftype, const int8_t *Xq, const int8_t *W, const float *sx, const float *sw,
                             const void *bias, void *out, int64_t M, int64_t N, int64_t K, hipStream_t s)
{
    if (M > LINEAR_FEW_MAX) return hipErrorInvalidValue;
    switch (ftype) {
    case LB_BF16: return linear_few_t<__bf16>(Xq, W, sx, sw, bias, out, M, N, K, s);
    case LB_F16: return linear_few_t<_Float16>(Xq, W, sx, sw, bias, out, M, N, K, s);
    case LB_F32: return linear_few_t<float>(Xq, W, sx, sw, bias, out, M, N, K, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace lb
