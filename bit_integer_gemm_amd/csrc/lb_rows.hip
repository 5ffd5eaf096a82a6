// lb_rows.hip -- what stands between the products of a decoder layer, row by row: the norms
// on both sides of a block with its gate and the residual, and rotary positions.
#include "lb_float.hpp"
#include "lb_layer.hpp"

namespace lb {

// Eight elements at a 16-byte aligned address as floats, and back with one rounding each.
template <class T> __device__ inline void load8(const T *p, float *x)
{
    if constexpr (sizeof(T) == 4) {
        const f32x4 a = ((const f32x4 *)p)[0], b = ((const f32x4 *)p)[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = a[i], x[4 + i] = b[i];
    } else {
        const u32x4 v = *(const u32x4 *)p;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = lo_f32<T>(v[i]), x[2 * i + 1] = hi_f32<T>(v[i]);
    }
}
template <class T> __device__ inline void store8(T *p, const float *x)
{
    if constexpr (sizeof(T) == 4) {
        ((f32x4 *)p)[0] = f32x4{x[0], x[1], x[2], x[3]};
        ((f32x4 *)p)[1] = f32x4{x[4], x[5], x[6], x[7]};
    } else {
        *(u32x4 *)p = u32x4{pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7])};
    }
}

// ---- norms, gate and residual ----------------------------------------------
//   z = y, or y rms(y) wp;  r' = r + alpha gate z;  x = r' rms(r') w,
//   rms(v) = 1 / sqrt(mean(v^2) + eps)
// A row to a workgroup, 8 C numbers of it to a thread, which keeps them: every operand is
// read once.  fp32 throughout; r' and x are each rounded once, x from the r' before its
// rounding.  A row may be read and written in place: no thread writes a number that
// another reads.
// Bound by bytes: 8192 x 4096 in 16 bits in 76 us, 5.3 TB/s.  777 x 11008 with a gate and an fp32
// residual takes 31 us (3.9 TB/s): workgroups of 11 waves run two to a compute unit, so that
// 777 rows are one and a half rounds.  As many threads as a row has numbers for: with half as
// many, of twice the numbers, those take 79 and 36 us, and one row of 4096 3.1 in place of 2.4;
// asking for the gate before the first sum changes nothing.

// Sum of v over the workgroup, the same in every thread (partial sums in a fixed order).
__device__ inline float sum_of_row(float v, float *red)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    const int waves = (int)(blockDim.x >> 6);
    if (waves == 1) return v;
    if ((threadIdx.x & 63u) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < waves; ++w) v += red[w];
    return v;
}

template <class T, class RT, int C>
__global__ __launch_bounds__(1024) void residual_norm_kernel(NormArgs a)
{
    __shared__ float red[2][16];
    const int64_t row = blockIdx.x;
    const int32_t chunks = a.H / 8;
    float v[C][8], r[C][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int32_t c = (int32_t)threadIdx.x + i * (int32_t)blockDim.x;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = r[i][e] = 0.f;
        if (c >= chunks) continue;
        if (a.y) load8<T>((const T *)a.y + row * a.ldy + 8 * (int64_t)c, v[i]);
        if (a.r) load8<RT>((const RT *)a.r + row * a.ldr + 8 * (int64_t)c, r[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += v[i][e] * v[i][e];
    }
    float scale = a.alpha;
    if (a.post_w) scale = 1.0f / __builtin_sqrtf(sum_of_row(ss, red[0]) / (float)a.H + a.eps);
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int32_t c = (int32_t)threadIdx.x + i * (int32_t)blockDim.x;
        if (c >= chunks) continue;
        float w[8];
        if (a.y) {
            if (a.post_w) {
                load8<T>((const T *)a.post_w + 8 * (int64_t)c, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] = v[i][e] * scale * w[e] * a.alpha;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] *= a.alpha;
            }
            if (a.gate) {
                load8<T>((const T *)a.gate + row * a.ldg + 8 * (int64_t)c, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] *= w[e];
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            r[i][e] += v[i][e];
            ss += r[i][e] * r[i][e];
        }
        if (a.r_out) store8<RT>((RT *)a.r_out + row * a.ldro + 8 * (int64_t)c, r[i]);
    }
    if (!a.x) return;
    scale = 1.0f / __builtin_sqrtf(sum_of_row(ss, red[1]) / (float)a.H + a.eps);
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int32_t c = (int32_t)threadIdx.x + i * (int32_t)blockDim.x;
        if (c >= chunks) continue;
        float w[8];
        load8<T>((const T *)a.w + 8 * (int64_t)c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = r[i][e] * scale * w[e];
        store8<T>((T *)a.x + row * a.ldx + 8 * (int64_t)c, w);
    }
}

template <class T, class RT> static hipError_t residual_norm_t(const NormArgs &a, int64_t M, hipStream_t s)
{
    const int32_t chunks = a.H / 8;
    static_assert(LB_NORM_H_MAX <= 8 * 4 * 1024, "a row in the registers of 1024 threads");
    const int c = chunks <= 1024 ? 1 : chunks <= 2048 ? 2 : 4;
    const uint32_t threads = (uint32_t)(((chunks + c - 1) / c + 63) / 64 * 64);
    const int64_t most = LAUNCH_THREADS / threads;
    for (int64_t m = 0; m < M; m += most) {
        NormArgs p = a;
        if (p.y) p.y = (const T *)a.y + m * a.ldy;
        if (p.r) p.r = (const RT *)a.r + m * a.ldr;
        if (p.gate) p.gate = (const T *)a.gate + m * a.ldg;
        if (p.r_out) p.r_out = (RT *)a.r_out + m * a.ldro;
        if (p.x) p.x = (T *)a.x + m * a.ldx;
        const dim3 grid((uint32_t)(M - m < most ? M - m : most)), block(threads);
        if (c == 1) hipLaunchKernelGGL((residual_norm_kernel<T, RT, 1>), grid, block, 0, s, p);
        else if (c == 2) hipLaunchKernelGGL((residual_norm_kernel<T, RT, 2>), grid, block, 0, s, p);
        else hipLaunchKernelGGL((residual_norm_kernel<T, RT, 4>), grid, block, 0, s, p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_residual_norm(int ftype, int rtype, const NormArgs &a, int64_t M, hipStream_t s)
{
    const bool wide = rtype == LB_F32;
    switch (ftype) {
    case LB_BF16: return wide ? residual_norm_t<__bf16, float>(a, M, s) : residual_norm_t<__bf16, __bf16>(a, M, s);
    case LB_F16: return wide ? residual_norm_t<_Float16, float>(a, M, s) : residual_norm_t<_Float16, _Float16>(a, M, s);
    case LB_F32: return residual_norm_t<float, float>(a, M, s);
    default: return hipErrorInvalidValue;
    }
}

// ---- rotary positions ------------------------------------------------------
//   (a, b) -> mult (a cos t - b sin t, b cos t + a sin t),  t = pos f_i,
// for pair i of a head's first R numbers: (i, i + R/2), or (2i, 2i + 1).  Angles are formed
// in fp64 and in turns, of which only the fraction counts (in fp32 the angle of position
// 200000 would be off by 2^-7); sine and cosine of the fraction in fp32, once for all heads
// of a workgroup's tokens.  Bound by bytes: 8191 tokens of 40 heads of 128, 32 numbers of each
// turned, in 33 us (5.1 TB/s); 5 tokens in 3.2 us, a launch, three dependent reads and the
// angles.
// An item is the 8 numbers from 8 j on that a thread loads: of a head in halves the first
// R / 16 items are pairs of them, R / 2 apart.
constexpr int32_t ROPE_ANGLES = 2048;   // angles of a workgroup's tokens, at most
static_assert(LB_ROPE_R_MAX / 2 <= ROPE_ANGLES, "one token's at least");

template <class T, bool PAIRS>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a)
{
    __shared__ f32x2 turn[ROPE_ANGLES];
    const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
    const int32_t here = (int32_t)min((int64_t)a.tokens, a.T - t0), half = a.R / 2;
    const int32_t h0 = (int32_t)blockIdx.y * a.heads, heads = min(a.heads, a.Hq + a.Hk - h0);
    const int32_t turned = PAIRS ? a.R / 8 : a.R / 16, items = a.items, all = here * heads * items;
    // item n's numbers, read ahead of the angles that they wait for
    float x[8], b[8];
    T *out;
    int32_t j, t;
    auto read = [&](int32_t n) {
        j = n % items;
        const int32_t rest = n / items, h = h0 + rest % heads;
        t = rest / heads;
        const T *in;
        if (h < a.Hq) {
            in = (const T *)a.q + (t0 + t) * a.ldq + (int64_t)h * a.D;
            out = (T *)a.qo + (t0 + t) * a.ldqo + (int64_t)h * a.D;
        } else {
            in = (const T *)a.k + (t0 + t) * a.ldk + (int64_t)(h - a.Hq) * a.D;
            out = (T *)a.ko + (t0 + t) * a.ldko + (int64_t)(h - a.Hq) * a.D;
        }
        const int32_t at = j < turned ? 8 * j : a.R + 8 * (j - turned);   // (behind R: copied)
        out += at;
        load8<T>(in + at, x);
        if (!PAIRS && j < turned) load8<T>(in + half + at, b);
    };
    int32_t n = (int32_t)threadIdx.x, i = n;
    int64_t pos = a.pos[t0 + min(i / half, here - 1)];
    double freq = a.freqs[i % half];
    if (n < all) read(n);
    for (; i < here * half; i += 256) {
        if (i >= 256) {
            pos = a.pos[t0 + i / half];
            freq = a.freqs[i % half];
        }
        const double turns = (double)pos * (freq * 0.15915494309189533577);
        const float part = (float)(turns - __builtin_rint(turns));
        float sn, cs;
        sincospif(2.0f * part, &sn, &cs);
        turn[i] = f32x2{cs * a.mult, sn * a.mult};
    }
    __syncthreads();
    while (n < all) {
        const f32x2 *tn = turn + t * half;
        if (j < turned) {
            if constexpr (PAIRS) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const f32x2 c = tn[4 * j + e];
                    const float first = x[2 * e];
                    x[2 * e] = first * c.x - x[2 * e + 1] * c.y;
                    x[2 * e + 1] = x[2 * e + 1] * c.x + first * c.y;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const f32x2 c = tn[8 * j + e];
                    const float first = x[e];
                    x[e] = first * c.x - b[e] * c.y;
                    b[e] = b[e] * c.x + first * c.y;
                }
                store8<T>(out + half, b);
            }
        }
        store8<T>(out, x);
        n += 256;
        if (n < all) read(n);
    }
}

template <class T> static hipError_t rope_t(RopeArgs a, bool pairs, bool in_place, int cu, hipStream_t s)
{
    const int32_t heads = a.Hq + a.Hk, turned = pairs ? a.R / 8 : a.R / 16;
    a.items = in_place ? turned : turned + (a.D - a.R) / 8;
    // Few tokens: workgroups of about one item to a thread.  Many: all heads of a token, or of several
    // that give every thread an item (8191 tokens of 40 heads in workgroups of 1, 2, 4 and 8 tokens,
    // each without the reads ahead of the angles, which save 3 us: 37, 38, 39 and 41 us).
    a.tokens = 1;
    a.heads = heads;
    if (a.T >= 4 * (int64_t)cu) a.tokens = max(1, min(256 / (heads * a.items), ROPE_ANGLES / (a.R / 2)));
    else a.heads = max(1, min(heads, (256 + a.items - 1) / a.items));
    if (a.heads < (heads + 65534) / 65535) a.heads = (heads + 65534) / 65535;
    const int64_t most = LAUNCH_THREADS / 256 / ((heads + a.heads - 1) / a.heads) * a.tokens;
    const int64_t T_all = a.T;
    for (int64_t t = 0; t < T_all; t += most) {
        RopeArgs p = a;
        p.T = T_all - t < most ? T_all - t : most;
        p.pos = a.pos + t;
        p.q = (const T *)a.q + t * a.ldq;
        p.qo = (T *)a.qo + t * a.ldqo;
        if (a.Hk) {
            p.k = (const T *)a.k + t * a.ldk;
            p.ko = (T *)a.ko + t * a.ldko;
        }
        const dim3 grid((uint32_t)((p.T + a.tokens - 1) / a.tokens), (uint32_t)((heads + a.heads - 1) / a.heads));
        if (pairs) hipLaunchKernelGGL((rope_kernel<T, true>), grid, dim3(256), 0, s, p);
        else hipLaunchKernelGGL((rope_kernel<T, false>), grid, dim3(256), 0, s, p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_rope(int ftype, const RopeArgs &a, bool pairs, bool in_place, int cu, hipStream_t s)
{
    switch (ftype) {
    case LB_BF16: return rope_t<__bf16>(a, pairs, in_place, cu, s);
    case LB_F16: return rope_t<_Float16>(a, pairs, in_place, cu, s);
    case LB_F32: return rope_t<float>(a, pairs, in_place, cu, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace lb
