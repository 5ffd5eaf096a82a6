// lb_w4.hpp -- products of 16-bit activations with 4-bit weights in registers, shared by the
// linear layer and the mixture of experts.
//
// A row of weights holds levels u in 0..15, and a scale s and a minimum b for each group of G
// of them; the weight is u s + b.  Per group
//   sum_k x (u s + b) = s sum_k x (16 + u) + (b - 16 s) sum_k x,
// where 16 + u is exact in bf16 and fp16 and made of a nibble by one shift and one AND-OR for
// two weights (the nibble is written into the mantissa of 16.0), and both sums come from the
// matrix cores in fp32: every product is exact, nothing is rounded to 16 bits on the way.
//
// A wave takes 16 rows of weights a line (256 weights, 128 bytes) at a time, two loads of 8
// rows by 128 bytes: whole lines of memory, straight to registers.  With lane = 16 q + 8 h + r,
// load i delivers piece 4 h + q (16 bytes) of row 8 i + r; exchanging halves of 8 lanes
// between the two gives pieces q and 4 + q of row 8 h + r, the rows where a 16x16x32 matrix
// instruction expects them.  Then the four pieces of the same row are transposed between
// the lane rows q, so that word j of a lane is word q of piece j: one instruction
// covers 32 consecutive weights, whatever G.  Eight nibbles of a word come out in the order
// 0 4 1 5 2 6 3 7, and x is put in the same order.
#pragma once

#include "lb_float.hpp"

namespace lb {

template <class T> struct W4Vec;
template <> struct W4Vec<__bf16> {
    typedef bf16x8 x8;
    enum : uint32_t { MASK = 0x00780078u, BASE = 0x41804180u };
    enum : int { AT = 3 };   // bit of the mantissa that stands for 1 in [16, 32)
};
template <> struct W4Vec<_Float16> {
    typedef f16x8 x8;
    enum : uint32_t { MASK = 0x03C003C0u, BASE = 0x4C004C00u };
    enum : int { AT = 6 };
};

template <class T> __device__ inline f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c)
{
    typedef typename W4Vec<T>::x8 x8;
    if constexpr (__is_same(T, __bf16))
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(x8, a), __builtin_bit_cast(x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(x8, a), __builtin_bit_cast(x8, b), c, 0, 0, 0);
}

// 16 + u of a word's eight levels, in the order 0 4, 1 5, 2 6, 3 7.
template <class T> __device__ inline u32x4 w4_levels(uint32_t w)
{
    constexpr uint32_t M = W4Vec<T>::MASK, B = W4Vec<T>::BASE;
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int up = W4Vec<T>::AT - 4 * i;
        r[i] = ((up >= 0 ? w << (up >= 0 ? up : 0) : w >> (up < 0 ? -up : 0)) & M) | B;
    }
    return r;
}
// Eight activations in that order.
__device__ inline u32x4 w4_order(u32x4 x)
{
    u32x4 r;
    r[0] = __builtin_amdgcn_perm(x[2], x[0], 0x05040100u);
    r[1] = __builtin_amdgcn_perm(x[2], x[0], 0x07060302u);
    r[2] = __builtin_amdgcn_perm(x[3], x[1], 0x05040100u);
    r[3] = __builtin_amdgcn_perm(x[3], x[1], 0x07060302u);
    return r;
}
template <class T> __device__ inline uint32_t one_pair() { return __is_same(T, __bf16) ? 0x3F803F80u : 0x3C003C00u; }

// The two loads of a line, exchanged: pieces q (p0) and 4 + q (p1) of row lane % 16.
__device__ inline void w4_rows(u32x4 &p0, u32x4 &p1)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int a = (int)p0[i], b = (int)p1[i];
        p0[i] = (uint32_t)__builtin_amdgcn_update_dpp(a, b, 0x128, 0xF, 0xC, false);   // lanes 8..15: b of lane - 8
        p1[i] = (uint32_t)__builtin_amdgcn_update_dpp(b, a, 0x128, 0xF, 0x3, false);   // lanes 0..7: a of lane + 8
    }
}
// Word j of lane row q becomes word q of lane row j.
__device__ inline void w4_transpose(u32x4 &p)
{
    const auto a = __builtin_amdgcn_permlane32_swap(p[0], p[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(p[1], p[3], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    p[0] = c[0];
    p[1] = c[1];
    p[2] = d[0];
    p[3] = d[1];
}

// A tile of 16 NT rows of weights against 16 MT rows of x, lines `first` to `last` of K.
//   w, wbytes: the tile's first row and the bytes from there to the operand's end (rows
//     past it read as zeros); prm likewise, the groups' (scale, minimum) words.
//   xrow[m]: this lane's row (16 m + lane % 16) of x, any valid row where there is none;
//     PLANES 2: x is the sum of two planes, `plane` elements apart.
//   tile_rows: rows between the first rows of two tiles of weights.
//   T: the type of x as the matrix cores take it; PT: of the groups' numbers.
//   acc[m][n][i]: row 4 (lane / 16) + i of tile m of x, row lane % 16 of tile n of weights.
template <class T, class PT, int MT, int NT, int G, int PLANES = 1>
__device__ inline void w4_product(const uint8_t *w, uint64_t wbytes, const uint32_t *prm, uint64_t pbytes, int32_t K,
                                  int32_t tile_rows, int32_t first, int32_t last, const T *const (&xrow)[MT], int64_t plane,
                                  f32x4 (&acc)[MT][NT])
{
    constexpr int GROUPS = 256 / G, STEPS = G / 32;
    const int32_t lane = (int32_t)(threadIdx.x & 63u), q = lane >> 4, r = lane & 15;
    const i32x4 rw = make_rsrc(w, wbytes), rp = make_rsrc(prm, pbytes);
    const uint32_t kb = (uint32_t)K / 2u, groups = (uint32_t)K / G;
    const uint32_t piece = (uint32_t)(16 * (4 * ((lane >> 3) & 1) + q));
    const uint32_t row_at = (uint32_t)(lane & 7) * kb;
    u32x4 wv[NT][2];
    uint32_t pv[NT][GROUPS];
    auto load_line = [&](int32_t line) {
        const uint32_t at = (uint32_t)line * 128u + piece;
        const bool in = line < last && at < kb;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                wv[n][i] = __builtin_bit_cast(u32x4, load16(rw, in ? row_at + (uint32_t)(tile_rows * n + 8 * i) * kb + at : 0xFFFFFFF0u));
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                const uint32_t gi = (uint32_t)(line * GROUPS + g);
                const uint64_t b = (uint64_t)(uint32_t)rp.x | ((uint64_t)((uint32_t)rp.y & 0xFFFFu) << 32);
                const __amdgpu_buffer_rsrc_t br = __builtin_amdgcn_make_buffer_rsrc((void *)(uintptr_t)b, (short)0, rp.z, rp.w);
                pv[n][g] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(
                    br, (int)(line < last && gi < groups ? ((uint32_t)(tile_rows * n + r) * groups + gi) * 4u : 0xFFFFFFFCu), 0, 0);
            }
    };
    load_line(first);
    for (int32_t line = first; line < last; ++line) {
        u32x4 cw[NT][2];
        uint32_t cp[NT][GROUPS];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            cw[n][0] = wv[n][0];
            cw[n][1] = wv[n][1];
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) cp[n][g] = pv[n][g];
        }
        load_line(line + 1);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            w4_rows(cw[n][0], cw[n][1]);
            w4_transpose(cw[n][0]);
            w4_transpose(cw[n][1]);
        }
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            f32x4 sum[MT][NT], xs[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                xs[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int n = 0; n < NT; ++n) sum[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
#pragma unroll
            for (int st = 0; st < STEPS; ++st) {
                const int j = g * STEPS + st;   // 32 weights of the line
                const int32_t k = line * 256 + 32 * j + 8 * q;
                u32x4 lv[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) lv[n] = w4_levels<T>(cw[n][j / 4][j % 4]);
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int pl = 0; pl < PLANES; ++pl) {
                        u32x4 x = {0u, 0u, 0u, 0u};
                        if (k < K) x = w4_order(*(const u32x4 *)(xrow[m] + pl * plane + k));
                        const uint32_t one = one_pair<T>();
                        xs[m] = mfma16<T>(x, u32x4{one, one, one, one}, xs[m]);
#pragma unroll
                        for (int n = 0; n < NT; ++n) sum[m][n] = mfma16<T>(x, lv[n], sum[m][n]);
                    }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float s = lo_f32<PT>(cp[n][g]), c = hi_f32<PT>(cp[n][g]) - 16.0f * s;
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        acc[m][n][i] = __builtin_fmaf(s, sum[m][n][i], acc[m][n][i]);
                        acc[m][n][i] = __builtin_fmaf(c, xs[m][i], acc[m][n][i]);
                    }
            }
        }
    }
}

// Sums of the waves' tiles, in a fixed order, into LDS: NW tiles of 16 MT x 16 NT floats there,
// rows of x of 16 NT + 4 (so that a lane's four rows lie on other banks).  Afterwards
// w4_sum(lds, m, n) is the total; a barrier has passed.
template <int MT, int NT, int NW>
struct W4Join {
    enum : int { LD = 16 * NT + 4, TILE = 16 * MT * LD, FLOATS = NW * TILE };
    static __device__ inline void put(float *lds, int wave, const f32x4 (&acc)[MT][NT])
    {
        const int lane = (int)(threadIdx.x & 63u), q = lane >> 4, r = lane & 15;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) lds[wave * TILE + (16 * m + 4 * q + i) * LD + 16 * n + r] = acc[m][n][i];
    }
    static __device__ inline float sum(const float *lds, int m, int n)
    {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) v += lds[w * TILE + m * LD + n];
        return v;
    }
};

}  // namespace lb
