// lb_w4_rows.hip -- linear layer with 4-bit weights, many rows of x.
//
// Per group g of G weights, with u' = 16 + u exact in 16 bits and b' = b - 16 s (lb_w4.hpp):
//   out = sum_g b'[n,g] X[m,g] + sum_g s[n,g] sum_{k in g} x[m,k] u'[n,k],  X[m,g] = sum_{k in g} x[m,k].
// The first term is a product of its own with K / G in place of K: X and b' in three bf16 parts
// each (2^-23 of a term; with two, 2^-16, the error of fp16 outputs was up to 1.3 times that of their
// rounding where activations have a mean).  The second is exact products summed in fp32, a group at a time into a
// second set of accumulators, which are scaled into the first: no weight is ever rounded.  The
// terms have opposite signs, so that they enter the accumulators 16 groups of the one before the
// same groups of the other: with all of the first ahead of the second, fp32's roundings of what
// cancels later are as large as those of two parts (11008 weights in groups of 32).
//
// 4096 x 11008 x 4096 (G = 128): 346 us for five whole rounds of 128 x 256 tiles and 42 for the
// columns that are left, 950 TFLOP/s; the matrix cores are busy 47% of the time at the 2 GHz that
// the card allows (a large library product in bf16, without levels to make, reaches 1217): nine
// vector instructions, which make levels and scale sums, go with every matrix instruction.
//
// A launch of its own puts x in the order in which nibbles come out of a word, rows padded to
// whole stages with zeros, and forms X.
#include <algorithm>

#include "lb_layer.hpp"
#include "lb_w4.hpp"

namespace lb {

// ---- x in order, and its groups' sums --------------------------------------
// 8 numbers to a thread.  x: M x Kp of T; parts: three planes of M x groups16 bf16, X = their sum.
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
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const __bf16 part = (__bf16)s;
            parts[((int64_t)i * M + m) * groups16 + g] = part;
            s -= (float)part;
        }
    }
}

// ---- the product -----------------------------------------------------------
// 64 WM rows by 128 WN columns to a workgroup of eight waves (2 x 4), 32 WM x 32 WN to a wave,
// stages of 128 weights in a ring of three in LDS.  A wave keeps a stage's activations in
// registers; the sums of one tile of 32 columns are scaled beside the other's matrix
// instructions.  Or a part of K to a workgroup, whose fp32 sums a second launch adds up.
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
    const __bf16 *parts;    // M x groups16, and two more planes, each `plane` further on
    int64_t plane;
    const uint8_t *w;
    const uint32_t *p;
    const void *bias;
    void *out;              // or, with more than one part of K, parts of M x N fp32
    int64_t ldo;
    int32_t M, N, K, Kp, groups, groups16, splits;
    uint32_t tiles_m, tiles_n;
};

// Numbers from one part of K's sums to the next one's.
__host__ __device__ inline int64_t rows_apart(int64_t M, int64_t N) { return (M * N + 3) / 4 * 4; }

template <int G, int WM, int WN> struct RowsLds {
    enum : int {
        BM = 64 * WM, BN = 128 * WN, STAGES = 3,
        X = BM * 256, W = BN * 64, WORDS = BN * 128 / G,
        XC = 2 * WM, WC = WN,                                  // a wave's copies of a stage: x, weights,
        NC = WORDS > 512 ? WORDS / 512 : 1,                    // numbers
        NUMBERS = NC * 2048, STAGE = X + W + NUMBERS, COPIES = XC + WC + NC,
        UNITS = WN * 128 / G,                                  // (32 columns, group) of a stage
        BLOCK = 16 * G / 128,                                  // stages whose minima enter together
        // How the loop over stages is written, by registers and by times.  NEST: a loop for each block, and
        // the pipelined sums end with it; FRESH: addresses of the minima are formed for each block.  Groups of
        // 64 in one tile of columns: 34.6 us for 128 x 11008 x 4096 with one loop and fresh addresses, 38.3 with
        // nested ones.  Two tiles: without both, groups of 32 and 64 spill (800 and 690 us for 4096 x 11008 x
        // 4096 in place of 680 and 505); groups of 128 take 400 us with fresh addresses, 392 without.
        NEST = WN == 2 || G != 64, FRESH = G == 64 || (G == 32 && WN == 2),
        OUT_LD = BN + 8                                        // the tile on its way out, 16-bit
    };
    static_assert(BM * OUT_LD * 2 <= STAGES * STAGE, "the tile over the ring");
};

template <class T, int G, int WM, int WN>
__global__ __launch_bounds__(512, 2) void w4_rows_kernel(RowsArgs a)
{
    typedef RowsLds<G, WM, WN> L;
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
    const int32_t stages = a.Kp / 128, part = (int32_t)blockIdx.y;
    const int32_t first = part * stages / a.splits, last = (part + 1) * stages / a.splits;

    const i32x4 rx = make_rsrc((const T *)a.x + (int64_t)m0 * a.Kp, (uint64_t)(uint32_t)rows * (uint32_t)a.Kp * 2u);
    const i32x4 rw = make_rsrc(a.w + (int64_t)n0 * kb, (uint64_t)(uint32_t)cols * kb);
    const i32x4 rp = make_rsrc(a.p + (int64_t)n0 * a.groups, (uint64_t)(uint32_t)cols * (uint32_t)a.groups * 4u);
    const uint32_t lds0 = lds_addr(smem);

    // Copies.  x: four rows of 16 pieces at a time, piece p of row i at p ^ i % 16; weights: 16
    // rows of 4 pieces, piece p of row i at p ^ i / 4 % 4 (16 lanes' reads then lie on all 64
    // banks); numbers: word (group, column).
    const uint32_t x_row = 4u * (uint32_t)(L::XC * wave) + (uint32_t)(lane >> 4);
    const uint32_t w_row = 16u * (uint32_t)(L::WC * wave) + (uint32_t)(lane >> 2);
    const uint32_t w_piece = 16u * (uint32_t)((lane & 3) ^ ((lane >> 4) & 3));
    auto copy = [&](int i, int32_t st, uint32_t base) {   // number i of a wave's copies of stage st
        const bool there = st < last;
        if (i < L::XC) {
            const uint32_t row = x_row + 4u * (uint32_t)i, piece = (uint32_t)(lane & 15) ^ (row & 15u);
            dma16(rx, there ? row * (uint32_t)a.Kp * 2u + (uint32_t)st * 256u + 16u * piece : 0xFFFFFFF0u,
                  base + 1024u * (uint32_t)(L::XC * wave + i));
        } else if (i < L::XC + L::WC) {
            const uint32_t at = (uint32_t)st * 64u + w_piece;
            dma16(rw, there && at < kb ? (w_row + 16u * (uint32_t)(i - L::XC)) * kb + at : 0xFFFFFFF0u,
                  base + (uint32_t)L::X + 1024u * (uint32_t)(L::WC * wave + i - L::XC));
        } else {
            const int32_t c = L::NC * wave + i - L::XC - L::WC, word = 64 * c + lane, g = st * PER + word / L::BN;
            dma4(rp, there && word < L::WORDS && g < a.groups ? ((uint32_t)(word % L::BN) * (uint32_t)a.groups + (uint32_t)g) * 4u : 0xFFFFFFF0u,
                 base + (uint32_t)(L::X + L::W) + 256u * (uint32_t)c);
        }
    };
#pragma unroll
    for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int i = 0; i < L::COPIES; ++i) copy(i, first + st, lds0 + (uint32_t)(st * L::STAGE));

    f32x16 acc[WM][WN];
#pragma unroll
    for (int m = 0; m < WM; ++m)
#pragma unroll
        for (int n = 0; n < WN; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[m][n][i] = 0.f;
    const __bf16 *xp[WM];
    const uint32_t *np[WN];
    auto aim = [&](int32_t at) {
#pragma unroll
        for (int m = 0; m < WM; ++m) xp[m] = a.parts + (int64_t)(m0 + min(32 * (WM * wm + m) + (at & 31), rows - 1)) * a.groups16 + 8 * (at >> 5);
#pragma unroll
        for (int n = 0; n < WN; ++n) np[n] = a.p + (int64_t)(n0 + min(32 * (WN * wn + n) + (at & 31), cols - 1)) * a.groups + 8 * (at >> 5);
    };
    if constexpr (!L::FRESH) aim(lane);
    // The minima of groups lo .. hi, of the 16 from g on, into the accumulators: acc[m][n][i] is row
    // 8 (i / 4) + 4 h + i % 4 of tile m, column lane % 32 of tile n.  Of the nine products of X's parts
    // and b''s, the six down to 2^-16 of the first, smallest first.
    auto minima = [&](int32_t g, int32_t lo, int32_t hi) {
        if constexpr (L::FRESH) {
            int32_t at = lane;
            asm volatile("" : "+v"(at));
            aim(at);
        }
        u32x4 xv[WM][3];
        uint32_t nv[WN][8];
#pragma unroll
        for (int m = 0; m < WM; ++m)
#pragma unroll
            for (int i = 0; i < 3; ++i) xv[m][i] = *(const u32x4 *)(xp[m] + i * a.plane + g);
#pragma unroll
        for (int n = 0; n < WN; ++n)
#pragma unroll
            for (int i = 0; i < 8; ++i) nv[n][i] = np[n][min(g + i, a.groups - 1 - 8 * h)];
#pragma unroll
        for (int n = 0; n < WN; ++n) {
            u32x4 b[3];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float v[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int32_t k = g + 8 * h + 2 * i + e;
                    const uint32_t w = k >= lo && k < hi ? nv[n][2 * i + e] : 0u;
                    v[e] = hi_f32<T>(w) - 16.0f * lo_f32<T>(w);
                }
#pragma unroll
                for (int part = 0; part < 3; ++part) {
                    b[part][i] = pack2<__bf16>(v[0], v[1]);
                    v[0] -= lo_f32<__bf16>(b[part][i]);
                    v[1] -= hi_f32<__bf16>(b[part][i]);
                }
            }
#pragma unroll
            for (int m = 0; m < WM; ++m)
#pragma unroll
                for (int both = 2; both >= 0; --both)   // part i of X with part both - i of b'
#pragma unroll
                    for (int i = both; i >= 0; --i) acc[m][n] = mfma32<__bf16>(xv[m][i], b[both - i], acc[m][n]);
        }
    };

    const W4Const konst = w4_const<T>();
    // What a lane reads of a stage: x piece p of its rows, its columns' pieces, their numbers.
    const uint32_t x_at = (uint32_t)(32 * WM * wm + r) * 256u, w_at = (uint32_t)L::X + (uint32_t)(32 * WN * wn + r) * 64u;
    const uint32_t n_at = (uint32_t)(L::X + L::W) + 4u * (uint32_t)(32 * WN * wn + r);
    uint32_t at = 0, next = 2 * L::STAGE;
    constexpr bool PIPE = L::UNITS % 2 == 0;
    f32x16 sum[2][WM];
    float pending = 0.f;
#pragma unroll
    for (int m = 0; m < WM; ++m)
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[1][m][i] = 0.f;
    auto stage = [&](int32_t st) {
        wait_vm_barrier<L::COPIES>();
        const char *s0 = smem + at;
        // the columns' pieces and numbers first, then the rows in the order of their use: the first
        // matrix instructions need not wait for the last reads
        u32x4 wv[WN][2], x[8][WM];
        float scale[WN][PER];
#pragma unroll
        for (int n = 0; n < WN; ++n)
#pragma unroll
            for (int t = 0; t < 2; ++t)
                wv[n][t] = *(const u32x4 *)(s0 + w_at + 2048u * (uint32_t)n + 16u * ((uint32_t)(2 * t + h) ^ (uint32_t)((r >> 2) & 3)));
#pragma unroll
        for (int n = 0; n < WN; ++n)
#pragma unroll
            for (int g = 0; g < PER; ++g)
                scale[n][g] = lo_f32<T>(*(const uint32_t *)(s0 + n_at + 128u * (uint32_t)n + 4u * (uint32_t)(L::BN * g)));
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int m = 0; m < WM; ++m) {
                // instruction j takes 8 weights of piece 2 (j / 4) + h, word j % 4; G = 32: of piece
                // 2 (j / 4) + j / 2 % 2, word 2 (j % 2) + h
                const uint32_t p = G == 32 ? (uint32_t)(4 * (2 * (j / 4) + j / 2 % 2) + 2 * (j % 2)) + (uint32_t)h
                                           : (uint32_t)(8 * (j / 4) + j % 4) + 4u * (uint32_t)h;
                x[j][m] = *(const u32x4 *)(s0 + x_at + 8192u * (uint32_t)m + 16u * (p ^ (uint32_t)(r & 15)));
            }
#pragma unroll
        for (int n = 0; n < WN; ++n) {
            u32x4 w[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                w[t] = wv[n][t];
                if constexpr (G == 32) {
                    const auto c = __builtin_amdgcn_permlane32_swap(w[t][0], w[t][1], false, false);
                    const auto d = __builtin_amdgcn_permlane32_swap(w[t][2], w[t][3], false, false);
                    w[t] = u32x4{c[0], d[0], c[1], d[1]};
                }
            }
#pragma unroll
            for (int g = 0; g < PER; ++g) {
                constexpr int STEPS = 8 / PER;
                constexpr int CHAINS = WM == 1 && STEPS > 2 ? 2 : 1;   // one tile of rows: sums in two, or each instruction waits for the last
                // PIPE: the sums of the unit (columns, group) before are scaled step by step beside this
                // one's matrix instructions, the last unit's in the next stage or behind the loop
                const int now = PIPE ? (n * PER + g) % 2 : 0, was = 1 - now;
                const int wn_ = (n * PER + g + L::UNITS - 1) % L::UNITS / PER;   // whose columns they are
#pragma unroll
                for (int m = 0; m < WM; ++m)
#pragma unroll
                    for (int i = 0; i < 16; ++i) sum[now][m][i] = 0.f;
                f32x16 other;
#pragma unroll
                for (int i = 0; i < 16; ++i) other[i] = 0.f;
#pragma unroll
                for (int j = g * STEPS; j < (g + 1) * STEPS; ++j) {
                    const u32x4 lv = w4_levels<T>(w[j / 4][j % 4], konst);
#pragma unroll
                    for (int m = 0; m < WM; ++m) {
                        if (CHAINS == 2 && j % 2) other = mfma32<T>(x[j][m], lv, other);
                        else sum[now][m] = mfma32<T>(x[j][m], lv, sum[now][m]);
                        if constexpr (PIPE)
#pragma unroll
                            for (int i = 16 / STEPS * (j % STEPS); i < 16 / STEPS * (j % STEPS + 1); ++i)
                                acc[m][wn_][i] = __builtin_fmaf(pending, sum[was][m][i], acc[m][wn_][i]);
                    }
                    // a copy of the stage after next now and then: all at once they would hold up
                    // every wave at the start of a stage
                    if (WN == 1) {
                        if (j < L::COPIES) copy(j, st + 2, lds0 + next);
                    } else if (j % 2 == 0 && 4 * n + j / 2 < L::COPIES) {
                        copy(4 * n + j / 2, st + 2, lds0 + next);
                    }
                }
                if constexpr (CHAINS == 2)
#pragma unroll
                    for (int i = 0; i < 16; ++i) sum[now][0][i] += other[i];
                if constexpr (PIPE) {
                    pending = scale[n][g];
                } else {
#pragma unroll
                    for (int m = 0; m < WM; ++m)
#pragma unroll
                        for (int i = 0; i < 16; ++i) acc[m][n][i] = __builtin_fmaf(scale[n][g], sum[now][m][i], acc[m][n][i]);
                }
            }
        }
        static_assert(L::COPIES <= 8, "all copies are made");
        at = at == 2 * L::STAGE ? 0 : at + L::STAGE;
        next = next == 2 * L::STAGE ? 0 : next + L::STAGE;
    };
    auto flush = [&] {   // the last unit's sums
        if constexpr (PIPE)
#pragma unroll
            for (int m = 0; m < WM; ++m)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    acc[m][WN - 1][i] = __builtin_fmaf(pending, sum[1][m][i], acc[m][WN - 1][i]);
                    sum[1][m][i] = 0.f;
                }
    };
    auto block_end = [&](int32_t st) { return min((st / L::BLOCK + 1) * L::BLOCK, last); };
    auto enter = [&](int32_t st, int32_t end) { minima(16 * (st / L::BLOCK), st * PER, min(end * PER, a.groups)); };
    if constexpr (L::NEST) {
        for (int32_t st = first; st < last;) {
            const int32_t end = block_end(st);
            enter(st, end);
            for (; st < end; ++st) stage(st);
            flush();
        }
    } else {
        for (int32_t st = first, end = first; st < last; ++st) {
            if (st == end) {
                end = block_end(st);
                enter(st, end);
            }
            stage(st);
        }
        flush();
    }
    wait_vm_all();   // (the last two stages' copies brought nothing)
    if (a.splits > 1) {
        float *out = (float *)a.out + (int64_t)part * rows_apart(a.M, a.ldo) + (int64_t)m0 * a.ldo + n0;
#pragma unroll
        for (int n = 0; n < WN; ++n) {
            const int32_t col = 32 * (WN * wn + n) + r;
            if (col >= cols) continue;
#pragma unroll
            for (int m = 0; m < WM; ++m)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int32_t row = 32 * (WM * wm + m) + 8 * (i / 4) + 4 * h + i % 4;
                    if (row < rows) out[row * a.ldo + col] = acc[m][n][i];
                }
        }
        return;
    }
    // Out through LDS, so that rows are written in pieces of 16 bytes (directly, 2 bytes a lane, the
    // stores took 19 us more at 4096 x 11008 x 4096).
    __syncthreads();
    T *const tile = (T *)smem;
#pragma unroll
    for (int n = 0; n < WN; ++n) {
        const int32_t col = 32 * (WN * wn + n) + r;
        const float bias = a.bias && col < cols ? (float)((const T *)a.bias)[n0 + col] : 0.f;
#pragma unroll
        for (int m = 0; m < WM; ++m)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                tile[(32 * (WM * wm + m) + 8 * (i / 4) + 4 * h + i % 4) * L::OUT_LD + col] = (T)(acc[m][n][i] + bias);
    }
    __syncthreads();
    T *const out = (T *)a.out + (int64_t)m0 * a.ldo + n0;
    if (a.ldo % 8 == 0 && cols % 8 == 0) {
        for (int32_t i = (int32_t)threadIdx.x; i < rows * (L::BN / 8); i += 512) {
            const int32_t row = i / (L::BN / 8), c = i % (L::BN / 8) * 8;
            if (c < cols) *(u32x4 *)(out + row * a.ldo + c) = *(const u32x4 *)(tile + row * L::OUT_LD + c);
        }
    } else {
        for (int32_t i = (int32_t)threadIdx.x; i < rows * L::BN; i += 512) {
            const int32_t row = i / L::BN, c = i % L::BN;
            if (c < cols) out[row * a.ldo + c] = tile[row * L::OUT_LD + c];
        }
    }
}

// Parts of K added up, in their order: four numbers to a thread, whatever their columns (parts
// are a multiple of four numbers apart).
template <class T>
__global__ __launch_bounds__(256) void w4_join_kernel(const float *__restrict__ parts, const T *__restrict__ bias, T *__restrict__ out,
                                                      int64_t n, int64_t apart, int32_t N, int32_t splits)
{
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    for (int32_t s0 = 0; s0 < splits; s0 += 4) {
        f32x4 p[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) p[u] = *(const f32x4 *)(parts + min(s0 + u, splits - 1) * apart + i);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (s0 + u < splits)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] += p[u][e];
    }
    if (bias) {
        int32_t c = (int32_t)(i % N);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] += (float)bias[c];
            c = c + 1 == N ? 0 : c + 1;
        }
    }
    if (i + 4 <= n) *(u32x2 *)(out + i) = u32x2{pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3])};
    else
        for (int e = 0; i + e < n; ++e) out[i + e] = (T)v[e];
}

// ---- planning --------------------------------------------------------------
// A band of columns: its tiles and parts of K.
struct RowsBand {
    int tile;            // 0: 128 x 256, 1: 128 x 128, 2: 64 x 128
    int64_t n0, cols, splits;
};
struct RowsPlan {
    int bands;
    RowsBand band[2];
    double us;
};
static const int64_t kBM[3] = {128, 128, 64}, kBN[3] = {256, 128, 128};
// Time of a band, us: rounds of workgroups of a stage's time in each tile, as measured, and what a
// workgroup takes besides.  (Two workgroups of the smallest tile share a compute unit, which
// gains them about a tenth.)
static double band_us(const RowsBand &b, int64_t M, int64_t stages, int cu)
{
    static const double per_stage[3] = {1.75, 1.05, 0.75}, rest[3] = {9, 7.5, 6.5};
    const int64_t wgs = ((M + kBM[b.tile] - 1) / kBM[b.tile]) * ((b.cols + kBN[b.tile] - 1) / kBN[b.tile]) * b.splits;
    const double each = rest[b.tile] + (double)((stages + b.splits - 1) / b.splits) * per_stage[b.tile];
    const double rounds = b.tile < 2 || wgs <= cu ? (double)((wgs + cu - 1) / cu) : 0.9 * (double)((2 * wgs + cu - 1) / cu) / 2;
    double us = 2.5 + rounds * each;
    if (b.splits > 1) us += 3.5 + (double)(M * b.cols) * (double)(4 * b.splits) / 4.5e6;
    return us;
}
static RowsPlan rows_plan(int64_t M, int64_t N, int64_t K, int cu)
{
    const int64_t stages = (K + 127) / 128;
    RowsPlan best{};
    auto offer = [&](const RowsPlan &p) {
        if (best.bands == 0 || p.us < best.us) best = p;
    };
    for (int t = 0; t < 3; ++t) {
        RowsPlan p{1, {{t, 0, N, 1}, {}}, 0};
        p.us = band_us(p.band[0], M, stages, cu);
        offer(p);
        // parts of K where there are too few tiles
        const int64_t tiles = ((M + kBM[t] - 1) / kBM[t]) * ((N + kBN[t] - 1) / kBN[t]);
        for (int64_t s = 2; s <= 16 && s * 2 <= stages && tiles * (s - 1) < cu; ++s) {
            p.band[0].splits = s;
            p.us = band_us(p.band[0], M, stages, cu);
            offer(p);
        }
    }
    // whole rounds of the largest tiles, and the columns that are left in smaller ones
    const int64_t tm = (M + 127) / 128, full = (tm * (N / 256)) / cu * cu / tm * 256;
    if (full > 0 && full < N)
        for (int t = 1; t < 3; ++t) {
            RowsPlan p{2, {{0, 0, full, 1}, {t, full, N - full, 1}}, 0};
            p.us = band_us(p.band[0], M, stages, cu) + band_us(p.band[1], M, stages, cu);
            offer(p);
        }
    return best;
}

struct RowsSpace {
    int64_t Kp, groups16, parts, sums, bytes;
};
static RowsSpace rows_space(int64_t M, int64_t N, int64_t K, int64_t group, const RowsPlan &p)
{
    RowsSpace s;
    s.Kp = (K + 127) / 128 * 128;
    s.groups16 = (K / group + 15) / 16 * 16;
    s.parts = (M * s.Kp * 2 + 255) / 256 * 256;
    s.sums = s.parts + (3 * M * s.groups16 * 2 + 255) / 256 * 256;
    s.bytes = s.sums + (p.band[0].splits > 1 ? p.band[0].splits * rows_apart(M, N) * 4 : 0);
    return s;
}
int64_t linear_w4_rows_workspace(int64_t M, int64_t N, int64_t K, int64_t group, int cu)
{
    return rows_space(M, N, K, group, rows_plan(M, N, K, cu)).bytes;
}

template <class T, int G, int WM, int WN> static hipError_t rows_launch(RowsArgs r, hipStream_t s)
{
    typedef RowsLds<G, WM, WN> L;
    // (N is bounded, and parts of K are made only of products of few tiles: one launch)
    const int64_t tn = (r.N + L::BN - 1) / L::BN, M = r.M, most = LAUNCH_THREADS / 512 / tn / r.splits * L::BM;
    if (most < (r.splits > 1 ? M : L::BM)) return hipErrorInvalidValue;
    for (int64_t m = 0; m < M; m += most) {
        RowsArgs q = r;
        q.x = (const T *)r.x + m * r.Kp;
        q.parts = r.parts + m * r.groups16;
        q.out = (T *)r.out + m * r.ldo;   // (with parts of K, m is 0)
        q.M = (int32_t)std::min(most, M - m);
        q.tiles_m = (uint32_t)((q.M + L::BM - 1) / L::BM);
        q.tiles_n = (uint32_t)tn;
        hipLaunchKernelGGL((w4_rows_kernel<T, G, WM, WN>), dim3(q.tiles_m * q.tiles_n, (uint32_t)r.splits), dim3(512),
                           (uint32_t)(L::STAGES * L::STAGE), s, q);
    }
    return hipGetLastError();
}

template <class T, int G> static hipError_t rows_t(const W4Args &a, int cu, void *workspace, hipStream_t s)
{
    const RowsPlan plan = rows_plan(a.M, a.N, a.K, cu);
    const RowsSpace sp = rows_space(a.M, a.N, a.K, G, plan);
    T *x = (T *)workspace;
    __bf16 *parts = (__bf16 *)((char *)workspace + sp.parts);
    // (a thread for every 8 numbers, up to the last padded group's first)
    const int64_t across = std::max(sp.Kp, sp.groups16 * G), wide = (across / 8 + 255) / 256;
    const int64_t most = std::min<int64_t>(65535, LAUNCH_THREADS / (256 * wide));
    for (int64_t m = 0; m < a.M; m += most)
        hipLaunchKernelGGL((w4_prepare_kernel<T, G>), dim3((uint32_t)wide, (uint32_t)std::min(most, a.M - m)), dim3(256), 0, s,
                           (const T *)a.x + m * a.ldx, a.ldx, x + m * sp.Kp, parts + m * sp.groups16, (int32_t)a.M, (int32_t)a.K,
                           (int32_t)sp.Kp, (int32_t)sp.groups16);
    for (int i = 0; i < plan.bands; ++i) {
        const RowsBand &b = plan.band[i];
        RowsArgs r;
        r.x = x;
        r.parts = parts;
        r.plane = a.M * sp.groups16;
        r.w = a.w + b.n0 * (a.K / 2);
        r.p = (const uint32_t *)a.p + b.n0 * (a.K / G);
        r.bias = a.bias ? (const T *)a.bias + b.n0 : nullptr;
        r.out = b.splits > 1 ? (void *)((char *)workspace + sp.sums) : (void *)((T *)a.out + b.n0);
        r.ldo = a.N;
        r.M = (int32_t)a.M;
        r.N = (int32_t)b.cols;
        r.K = (int32_t)a.K;
        r.Kp = (int32_t)sp.Kp;
        r.groups = (int32_t)(a.K / G);
        r.groups16 = (int32_t)sp.groups16;
        r.splits = (int32_t)b.splits;
        const hipError_t e = b.tile == 0 ? rows_launch<T, G, 2, 2>(r, s) : b.tile == 1 ? rows_launch<T, G, 2, 1>(r, s) : rows_launch<T, G, 1, 1>(r, s);
        if (e != hipSuccess) return e;
        if (b.splits > 1) {
            const int64_t n = a.M * a.N;
            hipLaunchKernelGGL((w4_join_kernel<T>), dim3((uint32_t)((n + 1023) / 1024)), dim3(256), 0, s,
                               (const float *)((char *)workspace + sp.sums), (const T *)a.bias, (T *)a.out, n, rows_apart(a.M, a.N),
                               (int32_t)a.N, (int32_t)b.splits);
        }
    }
    return hipGetLastError();
}

hipError_t launch_linear_w4_rows(int ftype, int group, const W4Args &a, int cu, void *workspace, hipStream_t s)
{
    if (ftype == LB_BF16)
        return group == 32 ? rows_t<__bf16, 32>(a, cu, workspace, s) : group == 64 ? rows_t<__bf16, 64>(a, cu, workspace, s)
                                                                                  : rows_t<__bf16, 128>(a, cu, workspace, s);
    if (ftype == LB_F16)
        return group == 32 ? rows_t<_Float16, 32>(a, cu, workspace, s) : group == 64 ? rows_t<_Float16, 64>(a, cu, workspace, s)
                                                                                    : rows_t<_Float16, 128>(a, cu, workspace, s);
    return hipErrorInvalidValue;
}

}  // namespace lb
