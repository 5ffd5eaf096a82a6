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

// One row tile's numbers of a line: GROUPS words (scale, minimum) of row lane % 16.
template <int GROUPS> __device__ inline void w4_numbers(const __amdgpu_buffer_rsrc_t &rsrc, uint32_t at, int32_t left, uint32_t (&v)[GROUPS])
{
    if (left >= GROUPS) {
        if constexpr (GROUPS == 2) {
            const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rsrc, (int)at, 0, 0));
            v[0] = a[0], v[1] = a[1];
        } else {
#pragma unroll
            for (int g = 0; g < GROUPS; g += 4) {
                const u32x4 a = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, (int)(at + 4u * g), 0, 0));
#pragma unroll
                for (int i = 0; i < 4; ++i) v[g + i] = a[i];
            }
        }
    } else {
#pragma unroll
        for (int g = 0; g < GROUPS; ++g)
            v[g] = g < left ? (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rsrc, (int)(at + 4u * g), 0, 0) : 0u;
    }
}

__device__ inline __amdgpu_buffer_rsrc_t w4_rsrc(const void *base, uint64_t bytes)
{
    const i32x4 r = make_rsrc(base, bytes);
    const uint64_t b = (uint64_t)(uint32_t)r.x | ((uint64_t)((uint32_t)r.y & 0xFFFFu) << 32);
    return __builtin_amdgcn_make_buffer_rsrc((void *)(uintptr_t)b, (short)0, r.z, r.w);
}
__device__ inline u32x4 w4_load(const __amdgpu_buffer_rsrc_t &rsrc, uint32_t at)
{
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, (int)at, 0, 0));
}

// The sixteen rows of weights of a tile, at row `row` of the operand; rows from `rows` on do not
// exist and read as zeros.
struct W4Tile {
    int64_t row;
    int32_t rows;
};

// Activations in LDS: rows of w4_x_stride(K) bytes (K up to whole lines, the rest zeros; 16
// bytes more, so that 16 rows' pieces lie on all banks once), in the order of the levels.
// first() takes what a batch of loads covers (8 of 16 bytes a thread) to registers, rest()
// writes it to LDS and brings whatever is left: between the two a wave asks for its first
// weights, whose latency then runs beside the copy.
__host__ __device__ inline uint32_t w4_x_stride(int32_t K) { return (uint32_t)((K + 255) / 256) * 512u + 16u; }

template <class RowAt> struct W4Stage {
    enum : int { BATCH = 8 };
    char *lds;
    int32_t K, pieces, all, threads;   // pieces of 16 bytes of a row, and of all rows
    RowAt row_at;                      // (row) -> its first element
    u32x4 v[BATCH];
    __device__ inline W4Stage(char *l, int32_t k, int32_t rows, int32_t n, const RowAt &at)
        : lds(l), K(k), pieces((k + 255) / 256 * 32), all((k + 255) / 256 * 32 * rows), threads(n), row_at(at)
    {
    }
    __device__ inline void fetch(int32_t i0)
    {
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int32_t i = i0 + b * threads;
            v[b] = u32x4{0u, 0u, 0u, 0u};
            if (i < all) {
                const int32_t row = i / pieces, at = i - row * pieces;
                if (8 * at < K) v[b] = ((const u32x4 *)row_at(row))[at];
            }
        }
    }
    __device__ inline void write(int32_t i0)
    {
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int32_t i = i0 + b * threads;
            if (i < all) {
                const int32_t row = i / pieces, at = i - row * pieces;
                *(u32x4 *)(lds + (uint32_t)row * w4_x_stride(K) + 16u * (uint32_t)at) = w4_order(v[b]);
            }
        }
    }
    __device__ inline void first() { fetch((int32_t)threadIdx.x); }
    __device__ inline void rest()
    {
        write((int32_t)threadIdx.x);
        for (int32_t i = (int32_t)threadIdx.x + BATCH * threads; i < all; i += BATCH * threads) {
            fetch(i);
            write(i);
        }
        __syncthreads();
    }
};

// The stream of a wave: lines `first` to `last` of K of its tiles, one tile after another,
// DEPTH lines of weights on their way.
//   tile_at(t): the W4Tile of tile t of `tiles`.
//   ready(): called by every wave once its first loads are under way.
//   done(t, acc): its sums; acc[m][i] is row 4 (lane / 16) + i of tile m of x, column lane % 16.
// x: XLDS: in LDS as W4Stage leaves it, row 16 m + lane % 16 at xat[m], PLANES 2: the sum of two
// planes, `plane` bytes apart.  Otherwise in memory, xat and plane byte offsets in rx, loaded
// half a line ahead.
//   T: the type of x as the matrix cores take it; PT: of the groups' numbers.
template <class T, class PT, int MT, int G, int PLANES, bool XLDS, int DEPTH, class TileAt, class Ready, class Done>
__device__ inline void w4_stream(const uint8_t *W, const uint32_t *P, int32_t K, int32_t first, int32_t last, int32_t tiles,
                                 const __amdgpu_buffer_rsrc_t &rx, const char *xlds, const uint32_t (&xat)[MT],
                                 uint32_t plane, TileAt &&tile_at, Ready &&ready, Done &&done)
{
    constexpr int GROUPS = 256 / G, HALF = GROUPS / 2, STEPS = G / 32;
    const int32_t share = last - first, items = share * tiles;
    if (items <= 0) {
        ready();
        return;
    }
    const int32_t lane = (int32_t)(threadIdx.x & 63u), q = lane >> 4, r = lane & 15;
    const uint32_t kb = (uint32_t)K / 2u, groups = (uint32_t)K / G;
    const uint32_t piece = (uint32_t)(16 * (4 * ((lane >> 3) & 1) + q));
    const uint32_t row_at = (uint32_t)(lane & 7) * kb + piece, p_at = (uint32_t)r * groups * 4u;

    u32x4 wv[DEPTH][2];
    uint32_t pv[DEPTH][GROUPS];
    int32_t load_tile = 0, load_line = first;   // what is loaded next
    auto load = [&](u32x4 (&w)[2], uint32_t (&p)[GROUPS]) {
        if (load_tile >= tiles) return;
        const W4Tile t = tile_at(load_tile);
        const __amdgpu_buffer_rsrc_t rw = w4_rsrc(W + t.row * kb, (uint64_t)(uint32_t)t.rows * kb);
        const __amdgpu_buffer_rsrc_t rp = w4_rsrc(P + t.row * groups, (uint64_t)(uint32_t)t.rows * groups * 4u);
        const uint32_t at = (uint32_t)load_line * 128u;
        const bool in = at + piece < kb;
#pragma unroll
        for (int i = 0; i < 2; ++i) w[i] = w4_load(rw, in ? row_at + (uint32_t)(8 * i) * kb + at : 0xFFFFFFF0u);
        w4_numbers<GROUPS>(rp, p_at + (uint32_t)(load_line * GROUPS) * 4u, (int32_t)groups - load_line * GROUPS, p);
        if (++load_line == last) {
            load_line = first;
            ++load_tile;
        }
    };
    u32x4 xv[2][MT][4][PLANES];
    auto load_x = [&](int h, int32_t line) {
#pragma unroll
        for (int st = 0; st < 4; ++st)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int pl = 0; pl < PLANES; ++pl) {
                    const int32_t k = line * 256 + 128 * h + 32 * st + 8 * q;
                    if constexpr (XLDS)
                        xv[h][m][st][pl] = *(const u32x4 *)(xlds + xat[m] + pl * plane + (uint32_t)(2 * k));
                    else
                        xv[h][m][st][pl] = w4_load(rx, k < K ? xat[m] + pl * plane + (uint32_t)(2 * k) : 0xFFFFFFF0u);
                }
    };

    f32x4 acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto half = [&](int h, const u32x4 &w, const uint32_t (&p)[GROUPS]) {   // 128 weights
#pragma unroll
        for (int g = 0; g < HALF; ++g) {
            f32x4 sum[MT], xs[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) sum[m] = xs[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int st = 0; st < STEPS; ++st) {
                const int j = g * STEPS + st;   // 32 weights of the half
                const u32x4 lv = w4_levels<T>(w[j]);
                const uint32_t one = one_pair<T>();
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int pl = 0; pl < PLANES; ++pl) {
                        const u32x4 x = XLDS ? xv[h][m][j][pl] : w4_order(xv[h][m][j][pl]);
                        xs[m] = mfma16<T>(x, u32x4{one, one, one, one}, xs[m]);
                        sum[m] = mfma16<T>(x, lv, sum[m]);
                    }
            }
            const float s = lo_f32<PT>(p[h * HALF + g]), c = hi_f32<PT>(p[h * HALF + g]) - 16.0f * s;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[m][i] = __builtin_fmaf(s, sum[m][i], acc[m][i]);
                    acc[m][i] = __builtin_fmaf(c, xs[m][i], acc[m][i]);
                }
        }
    };

#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(wv[d], pv[d]);
    ready();
    load_x(0, first);
    int32_t tile = 0, line = first;
    for (int32_t i = 0; i < items; i += DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            if (i + d >= items) break;
            u32x4 w0 = wv[d][0], w1 = wv[d][1];
            uint32_t p[GROUPS];
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) p[g] = pv[d][g];
            w4_rows(w0, w1);
            w4_transpose(w0);
            w4_transpose(w1);
            load(wv[d], pv[d]);
            load_x(1, line);
            half(0, w0, p);
            const int32_t now = tile;
            const bool end = ++line == last;
            if (end) {
                line = first;
                ++tile;
            }
            load_x(0, line);
            half(1, w1, p);
            if (end) {
                done(now, acc);
#pragma unroll
                for (int m = 0; m < MT; ++m) acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
        }
    }
}

// Waves' sums in LDS: `rows` rows of x by 16 columns, rows 20 floats apart (a lane's four rows lie
// on other banks).
enum { W4_SLOT_LD = 20 };
template <int MT> __device__ inline void w4_put(float *slot, int32_t rows, const f32x4 (&acc)[MT])
{
    const int lane = (int)(threadIdx.x & 63u), q = lane >> 4, r = lane & 15;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (16 * m + 4 * q + i < rows) slot[(16 * m + 4 * q + i) * W4_SLOT_LD + r] = acc[m][i];
}

// How a workgroup of eight waves shares its tiles: kw waves take a share of K each, of `each`
// tiles, the next kw waves of the next ones.
constexpr int W4_WAVES = 8;
struct W4Split {
    int32_t kw, each;
};
// For `tiles` tiles of `lines` lines: the fewest lines for the busiest wave, and of equals the
// fewest shares.
inline W4Split w4_split(int64_t tiles, int64_t lines)
{
    W4Split best{1, (int32_t)((tiles + W4_WAVES - 1) / W4_WAVES)};
    for (int kw = 2; kw <= W4_WAVES; kw *= 2) {
        const W4Split s{kw, (int32_t)((tiles + W4_WAVES / kw - 1) / (W4_WAVES / kw))};
        if ((lines + kw - 1) / kw * s.each < (lines + best.kw - 1) / best.kw * best.each) best = s;
    }
    return best;
}

}  // namespace lb
