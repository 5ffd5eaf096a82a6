// lb_w4_rows.hip -- linear layer with 4-bit weights, many rows of x.
//
// Per group g of G weights, with u' = 16 + u exact in 16 bits and b' = b - 16 s (lb_w4.hpp):
//   out = sum_g b'[n,g] X[m,g] + sum_g s[n,g] sum_{k in g} x[m,k] u'[n,k],  X[m,g] = sum_{k in g} x[m,k].
// The first term is a product of its own with K / G in place of K, from which the accumulators
// start: X and b' in two bf16 parts each (2^-16 of a term).  The second is exact products summed
// in fp32, a group at a time into a second set of accumulators, which are scaled into the
// first: no weight is ever rounded.
//
// A launch of its own puts x in the order in which nibbles come out of a word, rows padded to
// whole stages with zeros, and forms X.
#include <algorithm>

#include "lb_internal.hpp"
#include "lb_w4.hpp"

namespace lb {

// ---- x in order, and its groups' sums --------------------------------------
// 8 numbers to a thread.  x: M x Kp of T; parts: two planes of M x groups16 bf16, X = their sum.
template <class T, int G>
__global__ __launch_bounds__(256) void w4_prepare_kernel(const T *__restrict__ X, int64_t ldx, T *__restrict__ x,
                                                         __bf16 *__restrict__ parts, int32_t M, int32_t K, int32_t Kp,
                                                         int32_t groups16)
{
    const int32_t m = (int32_t)blockIdx.y, at = (int32_t)(blockIdx.x * 256u + threadIdx.x) * 8;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (at < K) v = *(const u32x4 *)(X + m * ldx + at);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) s += lo_f32<T>(v[i]) + hi_f32<T>(v[i]);
#pragma unroll
    for (int d = 1; d < G / 8; d *= 2) s += __shfl_xor(s, d);
    if (at < Kp) *(u32x4 *)(x + (int64_t)m * Kp + at) = w4_order(v);
    const int32_t g = at / G;
    if (at % G == 0 && g < groups16) {
        const __bf16 hi = (__bf16)s, lo = (__bf16)(s - (float)hi);
        parts[(int64_t)m * groups16 + g] = hi;
        parts[((int64_t)M + m) * groups16 + g] = lo;
    }
}

// ---- the product -----------------------------------------------------------
// 128 rows by 256 columns to a workgroup of eight waves, 64 x 64 to a wave (2 x 2 tiles of
// 32 x 32), stages of 128 weights in a ring of three in LDS.  A wave keeps a stage's
// activations in registers and takes its two tiles of columns one after the other, so that
// scaling the one's sums runs beside the other's matrix instructions.
typedef float f32x16 __attribute__((ext_vector_type(16)));
template <class T> __device__ inline f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c)
{
    typedef typename W4Vec<T>::x8 x8;
    if constexpr (__is_same(T, __bf16))
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(x8, a), __builtin_bit_cast(x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(x8, a), __builtin_bit_cast(x8, b), c, 0, 0, 0);
}

struct RowsArgs {
    const void *x;          // M x Kp, in order
    const __bf16 *parts;    // M x groups16, and the second plane `plane` further on
    int64_t plane;
    const uint8_t *w;
    const uint32_t *p;
    const void *bias;
    void *out;
    int64_t ldo;
    int32_t M, N, K, Kp, groups, groups16;
    uint32_t tiles_m, tiles_n;
};

template <int G> struct RowsLds {
    enum : int {
        BM = 128, BN = 256, STAGES = 3,
        X = BM * 256, W = BN * 64, NUMBERS = G == 32 ? 4096 : 2048,
        STAGE = X + W + NUMBERS,
        COPIES = 4 + 2 + (G == 32 ? 2 : 1)   // a wave's copies of a stage
    };
};

template <class T, int G>
__global__ __launch_bounds__(512, 2) void w4_rows_kernel(RowsArgs a)
{
    typedef RowsLds<G> L;
    constexpr int PER = 128 / G;   // groups of a stage
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    const int32_t lane = (int32_t)(threadIdx.x & 63u), r = lane & 31, h = lane >> 5;
    const int32_t wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int32_t wm = wave & 1, wn = wave >> 1;
    uint32_t tm, tn;
    tile_of_block(blockIdx.x, a.tiles_m, a.tiles_n, 4u, tm, tn);
    const int32_t m0 = (int32_t)tm * L::BM, n0 = (int32_t)tn * L::BN;
    const int32_t rows = min((int)L::BM, a.M - m0), cols = min((int)L::BN, a.N - n0);
    const uint32_t kb = (uint32_t)a.K / 2u;

    const i32x4 rx = make_rsrc((const T *)a.x + (int64_t)m0 * a.Kp, (uint64_t)(uint32_t)rows * (uint32_t)a.Kp * 2u);
    const i32x4 rw = make_rsrc(a.w + (int64_t)n0 * kb, (uint64_t)(uint32_t)cols * kb);
    const i32x4 rp = make_rsrc(a.p + (int64_t)n0 * a.groups, (uint64_t)(uint32_t)cols * (uint32_t)a.groups * 4u);
    const uint32_t lds0 = lds_addr(smem);

    // Copies.  x: four rows of 16 pieces at a time, piece p of row i at p ^ i % 8; weights: 16 rows
    // of 4 pieces, piece p of row i at p ^ i / 2 % 4; numbers: word (group, column).
    const uint32_t x_row = 16u * (uint32_t)wave + (uint32_t)(lane >> 4);
    const uint32_t w_row = 32u * (uint32_t)wave + (uint32_t)(lane >> 2);
    const uint32_t w_piece = 16u * (uint32_t)((lane & 3) ^ ((lane >> 3) & 3));
    auto copy = [&](int32_t st, uint32_t base) {
        const bool there = st * 128 < a.Kp;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t row = x_row + 4u * (uint32_t)i, piece = (uint32_t)(lane & 15) ^ (row & 7u);
            dma16(rx, there ? row * (uint32_t)a.Kp * 2u + (uint32_t)st * 256u + 16u * piece : 0xFFFFFFF0u,
                  base + 1024u * (uint32_t)(4 * wave + i));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t at = (uint32_t)st * 64u + w_piece;
            dma16(rw, there && at < kb ? (w_row + 16u * (uint32_t)i) * kb + at : 0xFFFFFFF0u,
                  base + (uint32_t)L::X + 1024u * (uint32_t)(2 * wave + i));
        }
#pragma unroll
        for (int i = 0; i < L::COPIES - 6; ++i) {
            const int32_t word = 64 * ((L::COPIES - 6) * wave + i) + lane, g = st * PER + word / L::BN;
            dma4(rp, there && word / L::BN < PER && g < a.groups ? ((uint32_t)(word % L::BN) * (uint32_t)a.groups + (uint32_t)g) * 4u : 0xFFFFFFF0u,
                 base + (uint32_t)(L::X + L::W) + 256u * (uint32_t)((L::COPIES - 6) * wave + i));
        }
    };
    copy(0, lds0);
    copy(1, lds0 + L::STAGE);

    // The accumulators start from the groups' minima: acc[m][n][i] is row 8 (i / 4) + 4 h + i % 4 of
    // tile m, column lane % 32 of tile n.
    f32x16 acc[2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[m][n][i] = 0.f;
    {
        const __bf16 *xp[2];
        const uint32_t *np[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            xp[t] = a.parts + (int64_t)(m0 + min(64 * wm + 32 * t + r, rows - 1)) * a.groups16 + 8 * h;
            np[t] = a.p + (int64_t)(n0 + min(64 * wn + 32 * t + r, cols - 1)) * a.groups + 8 * h;
        }
        for (int32_t g = 0; g < a.groups16; g += 16) {
            u32x4 xh[2], xl[2];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                xh[m] = *(const u32x4 *)(xp[m] + g);
                xl[m] = *(const u32x4 *)(xp[m] + a.plane + g);
            }
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                u32x4 bh, bl;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float b[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int32_t at = 2 * i + e;
                        const uint32_t w = g + 8 * h + at < a.groups ? np[n][g + at] : 0u;
                        b[e] = hi_f32<T>(w) - 16.0f * lo_f32<T>(w);
                    }
                    bh[i] = pack2<__bf16>(b[0], b[1]);
                    bl[i] = pack2<__bf16>(b[0] - lo_f32<__bf16>(bh[i]), b[1] - hi_f32<__bf16>(bh[i]));
                }
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    acc[m][n] = mfma32<__bf16>(xl[m], bh, acc[m][n]);
                    acc[m][n] = mfma32<__bf16>(xh[m], bl, acc[m][n]);
                    acc[m][n] = mfma32<__bf16>(xh[m], bh, acc[m][n]);
                }
            }
        }
    }

    const W4Const konst = w4_const<T>();
    // What a lane reads of a stage: x piece p of its rows, its columns' pieces, their numbers.
    const uint32_t x_at = (uint32_t)(64 * wm + r) * 256u, w_at = (uint32_t)L::X + (uint32_t)(64 * wn + r) * 64u;
    const uint32_t n_at = (uint32_t)(L::X + L::W) + 4u * (uint32_t)(64 * wn + r);
    const int32_t steps = a.Kp / 128;
    uint32_t at = 0, next = 2 * L::STAGE;
    for (int32_t st = 0; st < steps; ++st) {
        wait_vm_barrier<L::COPIES>();
        copy(st + 2, lds0 + next);
        const char *s0 = smem + at;
        u32x4 x[8][2];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                // instruction j takes 8 weights of piece 2 (j / 4) + h, word j % 4; G = 32: of piece
                // 2 (j / 4) + j / 2 % 2, word 2 (j % 2) + h
                const uint32_t p = G == 32 ? (uint32_t)(4 * (2 * (j / 4) + j / 2 % 2) + 2 * (j % 2)) + (uint32_t)h
                                           : (uint32_t)(8 * (j / 4) + j % 4) + 4u * (uint32_t)h;
                x[j][m] = *(const u32x4 *)(s0 + x_at + 8192u * (uint32_t)m + 16u * (p ^ (uint32_t)(r & 7)));
            }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            u32x4 w[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                w[t] = *(const u32x4 *)(s0 + w_at + 2048u * (uint32_t)n + 16u * ((uint32_t)(2 * t + h) ^ (uint32_t)((r >> 1) & 3)));
                if constexpr (G == 32) {
                    const auto c = __builtin_amdgcn_permlane32_swap(w[t][0], w[t][1], false, false);
                    const auto d = __builtin_amdgcn_permlane32_swap(w[t][2], w[t][3], false, false);
                    w[t] = u32x4{c[0], d[0], c[1], d[1]};
                }
            }
#pragma unroll
            for (int g = 0; g < PER; ++g) {
                f32x16 sum[2];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int i = 0; i < 16; ++i) sum[m][i] = 0.f;
#pragma unroll
                for (int j = g * 8 / PER; j < (g + 1) * 8 / PER; ++j) {
                    const u32x4 lv = w4_levels<T>(w[j / 4][j % 4], konst);
#pragma unroll
                    for (int m = 0; m < 2; ++m) sum[m] = mfma32<T>(x[j][m], lv, sum[m]);
                }
                const float s = lo_f32<T>(*(const uint32_t *)(s0 + n_at + 128u * (uint32_t)n + 4u * (uint32_t)(L::BN * g)));
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[m][n][i] = __builtin_fmaf(s, sum[m][i], acc[m][n][i]);
            }
        }
        at = at == 2 * L::STAGE ? 0 : at + L::STAGE;
        next = next == 2 * L::STAGE ? 0 : next + L::STAGE;
    }
    wait_vm_all();   // (the last two copies brought nothing)

#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const int32_t col = 64 * wn + 32 * n + r;
        if (col >= cols) continue;
        const float bias = a.bias ? (float)((const T *)a.bias)[n0 + col] : 0.f;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int32_t row = 64 * wm + 32 * m + 8 * (i / 4) + 4 * h + i % 4;
                if (row < rows) ((T *)a.out)[(int64_t)(m0 + row) * a.ldo + n0 + col] = (T)(acc[m][n][i] + bias);
            }
    }
}

struct RowsSpace {
    int64_t Kp, groups16, parts, bytes;
};
static RowsSpace rows_space(int64_t M, int64_t K, int64_t group)
{
    RowsSpace s;
    s.Kp = (K + 127) / 128 * 128;
    s.groups16 = (K / group + 15) / 16 * 16;
    s.parts = (M * s.Kp * 2 + 255) / 256 * 256;
    s.bytes = s.parts + (2 * M * s.groups16 * 2 + 255) / 256 * 256;
    return s;
}
int64_t linear_w4_rows_workspace(int64_t M, int64_t K, int64_t group) { return rows_space(M, K, group).bytes; }

template <class T, int G> static hipError_t rows_t(const W4Args &a, void *workspace, hipStream_t s)
{
    const RowsSpace sp = rows_space(a.M, a.K, G);
    T *x = (T *)workspace;
    __bf16 *parts = (__bf16 *)((char *)workspace + sp.parts);
    // (a thread for every 8 numbers, up to the last padded group's first)
    const int64_t across = std::max(sp.Kp, sp.groups16 * G), wide = (across / 8 + 255) / 256;
    const int64_t most = std::min<int64_t>(65535, LAUNCH_THREADS / (256 * wide));
    for (int64_t m = 0; m < a.M; m += most)
        hipLaunchKernelGGL((w4_prepare_kernel<T, G>), dim3((uint32_t)wide, (uint32_t)std::min(most, a.M - m)), dim3(256), 0, s,
                           (const T *)a.x + m * a.ldx, a.ldx, x + m * sp.Kp, parts + m * sp.groups16, (int32_t)a.M, (int32_t)a.K,
                           (int32_t)sp.Kp, (int32_t)sp.groups16);
    typedef RowsLds<G> L;
    const int64_t tn = (a.N + L::BN - 1) / L::BN, rows = LAUNCH_THREADS / 512 / tn * L::BM;
    if (rows < L::BM) return hipErrorInvalidValue;
    for (int64_t m = 0; m < a.M; m += rows) {
        RowsArgs r;
        r.x = x + m * sp.Kp;
        r.parts = parts + m * sp.groups16;
        r.plane = a.M * sp.groups16;
        r.w = a.w;
        r.p = (const uint32_t *)a.p;
        r.bias = a.bias;
        r.out = (T *)a.out + m * a.N;
        r.ldo = a.N;
        r.M = (int32_t)std::min(rows, a.M - m);
        r.N = (int32_t)a.N;
        r.K = (int32_t)a.K;
        r.Kp = (int32_t)sp.Kp;
        r.groups = (int32_t)(a.K / G);
        r.groups16 = (int32_t)sp.groups16;
        r.tiles_m = (uint32_t)((r.M + L::BM - 1) / L::BM);
        r.tiles_n = (uint32_t)tn;
        hipLaunchKernelGGL((w4_rows_kernel<T, G>), dim3(r.tiles_m * r.tiles_n), dim3(512), (uint32_t)(L::STAGES * L::STAGE), s, r);
    }
    return hipGetLastError();
}

hipError_t launch_linear_w4_rows(int ftype, int group, const W4Args &a, void *workspace, hipStream_t s)
{
    if (ftype == LB_BF16)
        return group == 32 ? rows_t<__bf16, 32>(a, workspace, s) : group == 64 ? rows_t<__bf16, 64>(a, workspace, s) : rows_t<__bf16, 128>(a, workspace, s);
    if (ftype == LB_F16)
        return group == 32 ? rows_t<_Float16, 32>(a, workspace, s) : group == 64 ? rows_t<_Float16, 64>(a, workspace, s) : rows_t<_Float16, 128>(a, workspace, s);
    return hipErrorInvalidValue;
}

}  // namespace lb
