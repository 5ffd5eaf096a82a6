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
// A wave takes 16 rows of weights a line (256 weights, 128 bytes) at a time, copied straight
// into a ring of its own in LDS, whole lines of memory 8 rows at a time.  A lane reads two
// pieces of 16 bytes of a row there.  For G = 128 the four pieces of a group, one in each 16
// lanes, make four matrix instructions word by word; for shorter groups they are first
// transposed between the 16-lane rows, so that each instruction covers 32 consecutive
// weights.  Eight nibbles of a word come out in the order 0 4 1 5 2 6 3 7, and x is put in
// the same order, once, in LDS.
//
// What bounds it: a line costs a wave some 100 vector instructions (G = 128; 170 for G = 32,
// whose eight groups are each scaled) beside 16 matrix instructions, which eight waves hide
// under 5 TB/s of weights, except for G = 32 (about 4 TB/s).  Beyond that a launch is latencies:
// about 2 us until a kernel runs, 1 to 2 for x, 2 for the first weights, 1 for the join: 9 us
// for the first product of 5 tokens where there is hardly a weight to read.  Rings of two, three
// and four lines, and 16 waves in place of eight, are within 2% of each other; two workgroups
// to a compute unit are slower.
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

// 16 + u of a word's eight levels, in the order 0 4, 1 5, 2 6, 3 7.  (The constants are kept in
// registers: two literals would make two instructions of the AND and the OR.)
struct W4Const {
    uint32_t mask, base;
};
template <class T> __device__ inline W4Const w4_const()
{
    W4Const c{W4Vec<T>::MASK, W4Vec<T>::BASE};
    asm("" : "+v"(c.mask), "+s"(c.base));
    return c;
}
template <class T> __device__ inline u32x4 w4_levels(uint32_t w, const W4Const &c)
{
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int up = W4Vec<T>::AT - 4 * i;
        r[i] = ((up >= 0 ? w << (up >= 0 ? up : 0) : w >> (up < 0 ? -up : 0)) & c.mask) | c.base;
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

// The largest of 32 lanes' numbers, those of a line of x: of 16 by rotations, of both by a swap.
__device__ inline uint32_t w4_most_of_line(uint32_t v)
{
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x128, 0xF, 0xF, true));   // row_ror:8, then 4, 2 and 1
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x124, 0xF, 0xF, true));
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x122, 0xF, 0xF, true));
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x121, 0xF, 0xF, true));
    const auto both = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return max((uint32_t)both[0], (uint32_t)both[1]);
}

// The sixteen rows of weights of a tile, from row `row` of the operand; rows from `rows` on do not
// exist and read as zeros.
struct W4Tile {
    int64_t row;
    int32_t rows;
};

// How a workgroup shares its work.  K is taken in chunks of lines whose activations are in LDS
// together; a chunk's lines of all the workgroup's tiles, one tile's after the other's, are cut
// into eight equal parts, one to a wave.  A wave has parts of tiles tiles w / 8 and following.
constexpr int W4_WAVES = 8;
__host__ __device__ inline int32_t w4_first(int32_t tiles, int32_t wave) { return tiles * wave / W4_WAVES; }

// LDS of a workgroup: x (two planes: the second behind the first, then a scale for each line of
// each row), the rings, and what the caller puts behind.
template <int G> struct W4Lds {
    enum : int {
        GROUPS = 256 / G,
        NUMBERS = G == 32 ? 512 : 256,          // (scale, minimum) words of a line's 16 rows, group by group
        STAGE = 2048 + NUMBERS,
        DEPTH = 3,
        COPIES = G == 32 ? 4 : 3,               // copies of a stage
        RING = DEPTH * STAGE,
        RINGS = W4_WAVES * RING
    };
    // (a copy fills 1 KiB)
    static __host__ __device__ inline uint32_t plane_bytes(int32_t rows, int32_t lines) { return (uint32_t)(rows * lines + 1) / 2u * 1024u; }
    static __host__ __device__ inline uint32_t x_bytes(int planes, int32_t rows, int32_t chunk)
    {
        return planes * plane_bytes(rows, chunk) + (planes > 1 ? (uint32_t)(rows * chunk + 255) / 256u * 1024u : 0u);
    }
};

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// dma16 and dma4 with a second offset that is the same for all lanes.
__device__ inline void w4_copy16(i32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %3\n\t"
                 "s_nop 0\n\t"
                 "buffer_load_dwordx4 %0, %1, %2 offen lds"
                 :
                 : "v"(voff), "s"(rsrc), "s"(soff), "s"(lds)
                 : "memory", "m0");
}
__device__ inline void w4_copy4(i32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %3\n\t"
                 "s_nop 0\n\t"
                 "buffer_load_dword %0, %1, %2 offen lds"
                 :
                 : "v"(voff), "s"(rsrc), "s"(soff), "s"(lds)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

template <int N> __device__ inline void w4_wait() { asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory"); }

// The products of a wave's tiles: 16 rows of x at most by 16 columns each.
//   lds: x (x_bytes of it), then the rings.  Copies of two lines are under way while a third is
//     worked on; each wave waits for its own by count.
//   PLANES 2: x is fp32, in order in memory.  In LDS it is two planes of fp16 under a power of two
//     for each line, which puts the line's largest number into [2^14, 2^15): off by 2^-23 of a number,
//     and 2^-39 of the line's largest where that is more.
//   tiles: the workgroup's; tile_at(t): a W4Tile.
//   T: the type of x as the matrix cores take it; PT: of the groups' numbers.
// Every wave of a workgroup makes the same calls, also one without lines (x is copied by all).
template <class T, class PT, int G, int PLANES, class TileAt>
struct W4Flow {
    typedef W4Lds<G> L;
    enum : int { GROUPS = L::GROUPS, STEPS = G / 32 };
    char *const lds;
    const uint8_t *const W;
    const uint32_t *const P;
    const int32_t K, lines, chunk;
    const TileAt tile_at;
    const int32_t lane, wave;
    int32_t tiles;
    const uint32_t kb, groups;
    char *const ring;
    // what is copied next
    int32_t c_chunk, c_tile, c_line, c_hi;
    bool left;
    i32x4 rw, rp;
    uint32_t c_at, c_slot;
    uint32_t w_at[2], p_at[L::COPIES - 2];   // of a lane in a line of 16 rows of weights, of their numbers

    __device__ inline W4Flow(char *lds_, uint32_t x_bytes, const uint8_t *W_, const uint32_t *P_, int32_t K_, int32_t chunk_,
                             const TileAt &at_)
        : lds(lds_), W(W_), P(P_), K(K_), lines((K_ + 255) / 256), chunk(chunk_), tile_at(at_), lane((int32_t)(threadIdx.x & 63u)),
          wave(__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6))), tiles(0), kb((uint32_t)K_ / 2u), groups((uint32_t)K_ / G),
          ring(lds_ + x_bytes + wave * L::RING)
    {
    }

    __device__ inline int32_t first() const { return w4_first(tiles, wave); }
    __device__ inline int32_t end() const { return (tiles * (wave + 1) + W4_WAVES - 1) / W4_WAVES; }
    // Lines of the chunk from line c on, for a tile, that are this wave's.
    __device__ inline void bounds(int32_t c, int32_t tile, int32_t &lo, int32_t &hi) const
    {
        const int32_t n = min(chunk, lines - c), all = tiles * n, before = tile * n;
        lo = c + min(max(all * wave / W4_WAVES - before, 0), n);
        hi = c + min(max(all * (wave + 1) / W4_WAVES - before, 0), n);
    }
    // The tile that is copied next: the first from c_tile on of which this wave has lines.  Behind the
    // last one nothing is read: size 0, and no scalar offset, which the range check subtracts from
    // the size (0 less an offset would let everything pass, and the line behind the weights be read).
    __device__ inline void next_tile()
    {
        for (left = false;; ++c_tile) {
            if (c_tile >= end()) {
                c_chunk += chunk;
                c_tile = first();
                if (c_chunk >= lines) {
                    rw.z = rp.z = c_line = 0;
                    return;
                }
            }
            bounds(c_chunk, c_tile, c_line, c_hi);
            left = c_line < c_hi;
            if (left) break;
        }
        const W4Tile t = tile_at(c_tile);
        rw = make_rsrc(W + t.row * kb, (uint64_t)(uint32_t)t.rows * kb);
        rp = make_rsrc(P + t.row * groups, (uint64_t)(uint32_t)t.rows * groups * 4u);
    }
    // The next line into the ring: piece p of row i lies at p ^ i / 2 (the rows' pieces that 16 lanes
    // read together then lie on all 64 banks).  Past the last line nothing is read, nor past the end
    // of a row: no copy relies on how a range check counts the scalar offset.
    __device__ inline void copy()
    {
        const int32_t have = (int32_t)groups - c_line * GROUPS;
        uint32_t at[2] = {w_at[0], w_at[1]};
        if (have < GROUPS)   // the row ends in this line
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if ((uint32_t)c_line * 128u + 16u * (uint32_t)((lane & 7) ^ (4 * i + (lane >> 4))) >= kb) at[i] = 0xFFFFFFF0u;
#pragma unroll
        for (int i = 0; i < 2; ++i) w4_copy16(rw, at[i], (uint32_t)c_line * 128u, c_at + 1024u * (uint32_t)i);
#pragma unroll
        for (int i = 0; i < L::COPIES - 2; ++i) {
            uint32_t at = p_at[i];
            if (have < GROUPS && 4 * i + (lane >> 4) >= have) at = 0xFFFFFFF0u;
            w4_copy4(rp, at, (uint32_t)(c_line * GROUPS) * 4u, c_at + 2048u + 256u * (uint32_t)i);
        }
        c_at += L::STAGE;
        if (++c_slot == L::DEPTH) {
            c_slot = 0;
            c_at -= L::RING;
        }
        if (left && ++c_line == c_hi) {
            ++c_tile;
            next_tile();
        }
    }
    // Asks for the first lines of tiles_ tiles.
    __device__ inline void start(int32_t tiles_)
    {
        tiles = tiles_;
        c_chunk = c_line = 0;
        c_tile = first();
        rw = rp = make_rsrc(W, 0);
        next_tile();
        c_at = lds_addr(ring);
        c_slot = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) w_at[i] = (uint32_t)(8 * i + (lane >> 3)) * kb + 16u * (uint32_t)((lane & 7) ^ (4 * i + (lane >> 4)));
#pragma unroll
        for (int i = 0; i < L::COPIES - 2; ++i) {
            const uint32_t g = (uint32_t)(4 * i + (lane >> 4));
            p_at[i] = g < GROUPS ? ((uint32_t)(lane & 15) * groups + g) * 4u : 0xFFFFFFF0u;
        }
#pragma unroll
        for (int d = 0; d < L::DEPTH - 1; ++d) copy();
    }

    // x of the chunk from line c on: piece p of row i lies at p ^ i % 16 of the row.  fp32: the halves of
    // a piece's numbers in the two planes, of which the second has piece p at p ^ i % 16 ^ 8 in the end (both
    // planes of 8 rows then lie on all 64 banks).
    template <class XAt> __device__ inline void ask_x(int32_t c, int32_t rows, const i32x4 rx, XAt &&x_at)
    {
        const int32_t per = min(chunk, lines - c) * 32, all = per * rows;
        const uint32_t plane = L::plane_bytes(rows, per / 32);
        int32_t row = (wave * 64 + lane) / per, at = wave * 64 + lane - row * per;
        for (int32_t i0 = wave * 64; i0 < all; i0 += 64 * W4_WAVES) {
            const int32_t k = c * 256 + 8 * (at ^ (row & 15));
            const bool there = i0 + lane < all && k < K;
            const uint32_t from = x_at(min(row, rows - 1)) + 2u * PLANES * (uint32_t)k;
#pragma unroll
            for (int pl = 0; pl < PLANES; ++pl)
                dma16(rx, there ? from + 16u * (uint32_t)pl : 0xFFFFFFF0u, lds_addr(lds) + plane * (uint32_t)pl + 16u * (uint32_t)i0);
            for (at += 64 * W4_WAVES; at >= per; at -= per) ++row;
        }
    }
    // Each lane what it copied itself: numbers in order; fp32 into two planes.
    __device__ inline void order_x(int32_t c, int32_t rows)
    {
        const int32_t all = min(chunk, lines - c) * 32 * rows;
        u32x4 *const p = (u32x4 *)lds;
        if constexpr (PLANES == 2) {
            const uint32_t plane = L::plane_bytes(rows, min(chunk, lines - c));
            u32x4 *const p1 = (u32x4 *)(lds + plane);
            float *const scale = (float *)(lds + 2 * plane);
            constexpr int AT_ONCE = 2;
            for (int32_t i0 = (int32_t)threadIdx.x; i0 < all; i0 += 64 * W4_WAVES * AT_ONCE) {
                u32x4 v[AT_ONCE][2];
#pragma unroll
                for (int u = 0; u < AT_ONCE; ++u) {
                    const int32_t i = min(i0 + 64 * W4_WAVES * u, all - 1);
                    v[u][0] = p[i];
                    v[u][1] = p1[i];
                }
#pragma unroll
                for (int u = 0; u < AT_ONCE; ++u) {
                    const int32_t i = i0 + 64 * W4_WAVES * u;
                    if (i >= all) break;   // (for whole lines: half a wave has one)
                    uint32_t most = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) most = max(most, v[u][e / 4][e % 4] & 0x7FFFFFFFu);
                    // infinities and NaN are above all, and stay so
                    const uint32_t up = min(268u - (w4_most_of_line(most) >> 23), 253u);   // the power's exponent
                    u32x4 hi, lo;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float a = __uint_as_float(v[u][e / 2][e % 2 * 2]) * __uint_as_float(up << 23);
                        const float b = __uint_as_float(v[u][e / 2][e % 2 * 2 + 1]) * __uint_as_float(up << 23);
                        hi[e] = pack2<_Float16>(a, b);
                        lo[e] = pack2<_Float16>(a - lo_f32<_Float16>(hi[e]), b - hi_f32<_Float16>(hi[e]));
                    }
                    p[i] = hi;
                    p1[i ^ 8] = lo;   // (a lane of this wave's, which has read what lay there)
                    if (i % 32 == 0) scale[i / 32] = __uint_as_float((254u - up) << 23);
                }
            }
        } else {
            constexpr int AT_ONCE = 4;
            for (int32_t i = (int32_t)threadIdx.x; i < all; i += 64 * W4_WAVES * AT_ONCE) {
                u32x4 v[AT_ONCE];
#pragma unroll
                for (int u = 0; u < AT_ONCE; ++u) v[u] = p[min(i + 64 * W4_WAVES * u, all - 1)];
#pragma unroll
                for (int u = 0; u < AT_ONCE; ++u)
                    if (i + 64 * W4_WAVES * u < all) p[i + 64 * W4_WAVES * u] = w4_order(v[u]);
            }
        }
        __syncthreads();
    }

    // `rows` rows of x through rx, row i's first byte at x_at(i).  STARTED: start() has been called, and
    // the weights' latency runs beside the copy of x; else start(tiles_) comes after it, and beside
    // the putting in order.
    //   done(t, acc, more): sums of tile t over this wave's lines; acc[i] is row 4 i + lane / 16, column
    //     lane % 16 of the tile.  Called for each chunk (more: not the first) and each of the
    //     wave's tiles, also one without lines.
    template <bool STARTED, class XAt, class Done>
    __device__ inline void run(int32_t tiles_, int32_t rows, const i32x4 rx, XAt &&x_at, Done &&done)
    {
        auto none = [](int32_t) { return 0; };
        if (rows <= 4) run_n<1, STARTED, false>(tiles_, rows, rx, x_at, done, none);
        else if (rows <= 8) run_n<2, STARTED, false>(tiles_, rows, rx, x_at, done, none);
        else run_n<4, STARTED, false>(tiles_, rows, rx, x_at, done, none);
    }
    // RO: at most 4 RO rows.  A matrix instruction's row 4 q + i, whose sums are in lanes q of register
    // i, takes row 4 i + q, so that few rows need few registers scaled.  Two planes of at most 8 rows
    // are rows of one instruction, the second plane's sums RO registers behind the first's.
    // OWN_ROW: a tile has one row of x, row_of(tile).
    template <int RO, bool STARTED, bool OWN_ROW, class XAt, class Done, class RowOf>
    __device__ inline void run_n(int32_t tiles_, int32_t rows, const i32x4 rx, XAt &&x_at, Done &&done, RowOf &&row_of)
    {
        constexpr bool STACK = PLANES == 2 && RO < 4;
        constexpr int PL = STACK ? 1 : PLANES, RI = STACK ? 2 * RO : RO;
        const int32_t q = lane >> 4, r = lane & 15;
        ask_x(0, rows, rx, x_at);
        if constexpr (!STARTED) start(tiles_);
        if constexpr (STARTED) w4_wait<0>();
        else w4_wait<(L::DEPTH - 1) * L::COPIES>();
        order_x(0, rows);

        const W4Const konst = w4_const<T>();
        uint32_t at = 0, slot = 0;   // of the ring
        for (int32_t c = 0; c < lines; c += chunk) {
            if (c) {
                __syncthreads();
                ask_x(c, rows, rx, x_at);
                w4_wait<0>();
                order_x(c, rows);
            }
            // what a lane reads of x: its row's pieces j of a line's first half, any row's where it has none;
            // and, of two planes, the scales of the rows whose sums it has
            const int32_t here = min(chunk, lines - c);
            const uint32_t plane = L::plane_bytes(rows, here);
            uint32_t xa[4][PL], sa[RO];
            auto aim_x = [&](int32_t first) {
#pragma unroll
                for (int pl = 0; pl < PL; ++pl) {
                    const uint32_t second = (uint32_t)(STACK ? min((r & 3) / RO, 1) : pl);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        xa[j][pl] = second * plane + (uint32_t)(first * here) * 512u +
                                    16u * ((uint32_t)(G == 128 ? 4 * q + j : 4 * j + q) ^ (uint32_t)(first & 15) ^ (8u * second));
                }
#pragma unroll
                for (int i = 0; i < RO; ++i) sa[i] = 2 * plane + 4u * (uint32_t)((OWN_ROW ? first : min(4 * i + q, rows - 1)) * here);
            };
            if constexpr (!OWN_ROW) aim_x(min((STACK ? (r & 3) % RO : r & 3) * 4 + (r >> 2), rows - 1));
            const int32_t last = end();
            for (int32_t tile = first(); tile < last; ++tile) {
                if constexpr (OWN_ROW) aim_x(row_of(tile));
                int32_t lo, hi;
                bounds(c, tile, lo, hi);
                f32x4 acc = {0.f, 0.f, 0.f, 0.f};
                for (int32_t line = lo; line < hi; ++line) {
                    copy();
                    w4_wait<(L::DEPTH - 1) * L::COPIES>();
                    // everything that the line needs from LDS at once: one latency
                    const char *st = ring + at;
                    u32x4 w[2], x[8][PL];
                    uint32_t num[GROUPS];
                    float scale[RO];
#pragma unroll
                    for (int h = 0; h < 2; ++h) w[h] = *(const u32x4 *)(st + 128 * r + 16 * ((4 * h + q) ^ (r >> 1)));
#pragma unroll
                    for (int g = 0; g < GROUPS; ++g) num[g] = *(const uint32_t *)(st + 2048 + 64 * g + 4 * r);
                    const char *xl = lds + (uint32_t)(line - c) * 512u;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
#pragma unroll
                        for (int pl = 0; pl < PL; ++pl) x[j][pl] = *(const u32x4 *)(xl + xa[j % 4][pl] + 256 * (j / 4));
                    if constexpr (PLANES == 2)
#pragma unroll
                        for (int i = 0; i < RO; ++i) scale[i] = *(const float *)(lds + sa[i] + 4u * (uint32_t)(line - c));
                    __builtin_amdgcn_sched_barrier(0);
                    if constexpr (G != 128) {
                        w4_transpose(w[0]);
                        w4_transpose(w[1]);
                    }
                    f32x4 of_line = {0.f, 0.f, 0.f, 0.f};
                    f32x4 &to = PLANES == 2 ? of_line : acc;
#pragma unroll
                    for (int g = 0; g < GROUPS; ++g) {
                        f32x4 sum = {0.f, 0.f, 0.f, 0.f}, xs = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int j = g * STEPS; j < (g + 1) * STEPS; ++j) {   // 32 weights
                            const u32x4 lv = w4_levels<T>(w[j / 4][j % 4], konst);
                            const uint32_t one = one_pair<T>();
#pragma unroll
                            for (int pl = 0; pl < PL; ++pl) {
                                // (x's own sum too: forming it beside the ordering of x takes longer)
                                xs = mfma16<T>(x[j][pl], u32x4{one, one, one, one}, xs);
                                sum = mfma16<T>(x[j][pl], lv, sum);
                            }
                        }
                        const float s = lo_f32<PT>(num[g]), b = hi_f32<PT>(num[g]) - 16.0f * s;
#pragma unroll
                        for (int i = 0; i < RI; ++i) {
                            to[i] = __builtin_fmaf(s, sum[i], to[i]);
                            to[i] = __builtin_fmaf(b, xs[i], to[i]);
                        }
                    }
                    if constexpr (PLANES == 2)
#pragma unroll
                        for (int i = 0; i < RO; ++i) acc[i] = __builtin_fmaf(scale[i], STACK ? of_line[i] + of_line[RO + i] : of_line[i], acc[i]);
                    // the next copies overwrite what has been read here
                    asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
                    at += L::STAGE;
                    if (++slot == L::DEPTH) slot = at = 0;
                }
                done(tile, acc, c > 0);
            }
        }
        finish();
    }
    // No copy outlives the workgroup's use of the LDS.
    __device__ inline void finish() { w4_wait<0>(); }
};

// f(i, row, column) for the numbers acc[i] that a lane has of `rows` rows of x by 16 columns.
enum { W4_SLOT_LD = 16 };
template <class F> __device__ inline void w4_rows(int32_t rows, F &&f)
{
    const int lane = (int)(threadIdx.x & 63u), q = lane >> 4, r = lane & 15;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (4 * i + q < rows) f(i, 4 * i + q, r);
}
// A wave's sums into LDS, or (more) onto what it left there.
__device__ inline void w4_put(float *slot, int32_t rows, const f32x4 &acc, bool more)
{
    w4_rows(rows, [&](int32_t i, int32_t row, int32_t column) {
        float *s = slot + row * W4_SLOT_LD + column;
        *s = more ? *s + acc[i] : acc[i];
    });
}
// Sums of a workgroup's tiles, in units of `per` tiles that belong together, `rows` rows each.
// EDGES (one chunk): a unit that is a wave's alone stays in its registers, and only a wave's
// first and last unit, which others may have parts of, need LDS.  Else all units do.
template <bool EDGES> struct W4Sums {
    float *const slots;
    const int32_t units, per, rows, most;
    __device__ inline W4Sums(char *lds, int32_t units_, int32_t per_, int32_t rows_)
        : slots((float *)lds), units(units_), per(per_), rows(rows_), most(EDGES ? 2 : units_ / W4_WAVES + 2)
    {
    }
    __device__ inline bool whole(int32_t wave, int32_t u) const
    {
        return EDGES && wave * units <= W4_WAVES * u && W4_WAVES * (u + 1) <= (wave + 1) * units;
    }
    __device__ inline float *at(int32_t wave, int32_t u, int32_t i) const   // tile i of unit u
    {
        const int32_t n = u - w4_first(units, wave);
        return slots + ((wave * most + (EDGES ? min(n, 1) : n)) * per + i) * rows * W4_SLOT_LD;
    }
    // From all waves that have a part, in their order.
    __device__ inline float sum(int32_t u, int32_t i, int32_t row, int32_t column) const
    {
        const int32_t t = u * per + i, tiles = units * per, last = (W4_WAVES * (t + 1) + tiles - 1) / tiles;
        float v = 0.f;
        for (int32_t w = W4_WAVES * t / tiles; w < last; ++w) v += at(w, u, i)[row * W4_SLOT_LD + column];
        return v;
    }
    // f(u, row, column) for what lies in LDS.
    template <class F> __device__ inline void each(F &&f) const
    {
        const int32_t n = rows * W4_SLOT_LD;
        for (int32_t i = (int32_t)threadIdx.x; i < (EDGES ? W4_WAVES - 1 : units) * n; i += 64 * W4_WAVES) {
            int32_t u = i / n;
            const int32_t rest = i - u * n;
            if constexpr (EDGES) {   // the unit in which wave u + 1 begins, unless it begins there or another did
                const int32_t at = (u + 1) * units, before = u * units;
                if (at % W4_WAVES == 0 || (before % W4_WAVES && before / W4_WAVES == at / W4_WAVES)) continue;
                u = at / W4_WAVES;
            }
            f(u, rest / W4_SLOT_LD, rest % W4_SLOT_LD);
        }
    }
};
inline int64_t w4_sums_bytes(bool edges, int64_t units, int64_t per, int64_t rows)
{
    return W4_WAVES * (edges ? 2 : units / W4_WAVES + 2) * per * rows * W4_SLOT_LD * 4;
}

// Lines whose x, xrows of it, finds room in x_bytes.
inline int32_t w4_chunk(int64_t lines, int64_t xrows, int64_t x_bytes)
{
    const int64_t chunk = x_bytes / (512 * xrows);
    return (int32_t)(chunk >= lines ? lines : chunk > 0 ? chunk : 1);
}

}  // namespace lb
