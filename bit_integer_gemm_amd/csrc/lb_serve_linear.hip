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

// The 16 bytes of a chunk quantised to q.
template <class T> __device__ inline void put_chunk(int8_t *q, i32x4 v, const RowScale &rs)
{
    constexpr int EPT = 16 / sizeof(T);
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
    if constexpr (EPT == 8) *(u32x2 *)q = u32x2{b[0], b[1]};
    else *(uint32_t *)q = b[0];
}

// One workgroup per row; EPT elements per 16-byte chunk.  The row is read once
// if it fits the workgroup's registers (NC chunks per thread), else twice.  Bound by
// memory: 8192 rows of 4096 bf16 in 25.0 us, 4.0 TB/s where a copy reaches 5.0; few
// rows by latency, 16 of them 3.6 us.
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

#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int32_t c = (int32_t)threadIdx.x + 256 * i;
        if (c < chunks) put_chunk<T>(q + (int64_t)c * EPT, keep[i], rs);
    }
    for (int32_t c = (int32_t)threadIdx.x + 256 * NC; c < chunks; c += 256)
        put_chunk<T>(q + (int64_t)c * EPT, *(const i32x4 *)(row + (int64_t)c * EPT), rs);
}

template <class T>
static hipError_t quant_rows_part(const void *X, int64_t ldx, int8_t *Q, float *sx, int64_t M, int64_t K,
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

template <class T>
static hipError_t quant_rows_t(const void *X, int64_t ldx, int8_t *Q, float *sx, int64_t M, int64_t K,
                               hipStream_t s)
{
    const int64_t most = LAUNCH_THREADS / 256;
    for (int64_t m = 0; m < M; m += most) {
        const hipError_t e = quant_rows_part<T>((const T *)X + m * ldx, ldx, Q + m * K, sx + m,
                                                M - m < most ? M - m : most, K, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
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

// ---- few rows --------------------------------------------------------------
// A tile of 16 MT rows of X by 16 NT rows of W (output columns) per workgroup, and
// all of K: eight (four) waves each take their share of K for the whole tile, through
// rings of LDS of their own, and their exact sums meet in LDS by integer adds
// (whose order does not matter).  Every operand byte is read once per workgroup,
// but no wave waits for another before the end, and DEPTH - 1 stages of copies are
// under way in each: what bounds these products is the latency and number of bytes
// on their way, not the matrix cores.
//   A stage of a wave is S x 64 bytes of each row.  A copy fills 16 / S rows, 4 S
//   lanes to a row, whose bytes come in one piece (straight to registers in fragment
//   order, 16 rows to a load, delivers half as much: 18.1 us at 16 x 11008 x 4096).
//   Piece p of row n lies at p ^ n % 8 (S = 1: p ^ (n / 2) % 4), which keeps the
//   fragment reads off each other's banks.
//   Kernel times, weights from HBM: 1 x 4096 x 4096 6.8 us (2.5 TB/s; the launch, the
//   row's quantisation and one latency of HBM are most of it), 16 x 11008 x 4096 9.4 us
//   (4.8 TB/s of weights, about what a copy reaches).
//   W is the MFMA's A operand (lane l: row l % 16, piece l / 16), X its B operand;
//   lane l ends with columns 4 (l / 16) .. + 3 of row l % 16.
// FUSED (MT = 1, few rows): X is the layer's floating activations; while the first
// weights are on their way every workgroup quantises the rows for itself into LDS,
// which saves the launch that would do it once.
template <int MT, int NT, int S, int DEPTH, bool FUSED> struct FewTile {
    // waves; of the largest tiles four, which leaves room for whole lines (eight with
    // half a line each: 14.8 against 13.9 us at 256 x 4096 x 4096), and the sums lie
    // over their rings
    static constexpr bool OVER = MT > 3 && S == 2;
    static constexpr int NW = OVER ? 4 : 8;
    static constexpr int BLOCKS = (FUSED ? 0 : MT) + NT;      // 1 KiB blocks of a 64-byte step
    static constexpr int STAGE = S * BLOCKS * 1024, RING = DEPTH * STAGE;
    static constexpr int TM = 16 * MT, TN = 16 * NT, LD = TM + 4;   // a column of sums: TM and 4, so that 16 rows x 4 columns hit all banks once
    static constexpr int SUMS_AT = OVER ? 0 : NW * RING;
    static constexpr int SCALE_AT = OVER ? NW * RING : SUMS_AT + TN * LD * 4, RED_AT = SCALE_AT + TM * 4;
    static constexpr int X_AT = RED_AT + (FUSED ? NW * 16 : 0);   // FUSED: M x K int8
    static_assert((DEPTH - 1) * S * BLOCKS < 64, "vmcnt is 6 bits");
    static_assert(!OVER || TN * LD * 4 <= NW * RING, "sums over the rings");
};

template <int N> __device__ inline void wait_copies() { asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory"); }

template <class T, int MT, int NT, int S, int DEPTH, bool FUSED>
__global__ __launch_bounds__((64 * FewTile<MT, NT, S, DEPTH, FUSED>::NW)) void linear_few_kernel(
    const void *__restrict__ X, int64_t ldx, const int8_t *__restrict__ W, const float *__restrict__ sx,
    const float *__restrict__ sw, const T *__restrict__ bias, T *__restrict__ out, int32_t M, int32_t N,
    int32_t K, uint32_t tiles_m, uint32_t tiles_n)
{
    using FT = FewTile<MT, NT, S, DEPTH, FUSED>;
    constexpr int NW = FT::NW, THREADS = 64 * NW, TM = FT::TM, TN = FT::TN, LD = FT::LD;
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    int32_t *const sums = (int32_t *)(smem + FT::SUMS_AT);
    float *const row_scales = (float *)(smem + FT::SCALE_AT);
    const int32_t lane = (int32_t)(threadIdx.x & 63u);
    const int32_t wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int32_t r = lane & 15, c = lane >> 4;
    uint32_t tm, tn;
    tile_of_block(blockIdx.x, tiles_m, tiles_n, 4u, tm, tn);
    const int32_t m0 = (int32_t)tm * TM, n0 = (int32_t)tn * TN;

    // Copies: lane i takes piece (i % 8) ^ (i / 8) of row i / 8 (S = 1: piece
    // (i % 4) ^ (i / 8) % 4 of row i / 4).  Rows past the operand, pieces past K and
    // steps past this wave's share lie beyond the buffer's range and read as zeros.
    const i32x4 rw = make_rsrc(W + (int64_t)n0 * K, (uint64_t)min(TN, N - n0) * (uint32_t)K);
    const i32x4 rx = FUSED ? rw : make_rsrc((const int8_t *)X + (int64_t)m0 * K, (uint64_t)min(TM, M - m0) * (uint32_t)K);
    const uint32_t row_at = (uint32_t)(S == 1 ? lane >> 2 : lane >> 3) * (uint32_t)K;
    const int32_t piece = 16 * (S == 1 ? (lane & 3) ^ ((lane >> 3) & 3) : (lane & 7) ^ (lane >> 3));
    const uint32_t ring = lds_addr(smem) + (uint32_t)(wave * FT::RING);
    // Shares of K: whole 128-byte lines.  With one 64-byte step to a stage, two waves
    // take a share together, the left and the right halves of its lines, so that a
    // line is asked for twice at about one time and comes once.
    constexpr int PAIR = S == 1 ? 2 : 1;
    const int32_t lines = (K + 127) / 128, share = wave / PAIR, shares = NW / PAIR;
    const int32_t half = wave % PAIR;
    const int32_t first = 2 / PAIR * (share * lines / shares), last = 2 / PAIR * ((share + 1) * lines / shares);
    auto byte_of = [&](int32_t st) { return 64 * (PAIR * st + half); };
    auto copy = [&](int d, int32_t st) {
        const int32_t k = byte_of(st) + piece;
        const bool in = st < last && k < K;
        const uint32_t dst = ring + (uint32_t)(d * FT::STAGE);
#pragma unroll
        for (int t = 0; t < S * NT; ++t)
            dma16(rw, in ? row_at + (uint32_t)(16 / S * t) * (uint32_t)K + (uint32_t)k : 0xFFFFFFF0u, dst + t * 1024);
        if constexpr (!FUSED)
#pragma unroll
            for (int t = 0; t < S * MT; ++t)
                dma16(rx, in ? row_at + (uint32_t)(16 / S * t) * (uint32_t)K + (uint32_t)k : 0xFFFFFFF0u,
                      dst + (S * NT + t) * 1024);
    };
#pragma unroll
    for (int d = 0; d < DEPTH - 1; ++d) copy(d, first + S * d);
    auto clear_sums = [&] {
        for (int32_t i = (int32_t)threadIdx.x; i < TN * LD; i += THREADS) sums[i] = 0;
    };
    if constexpr (!FT::OVER) clear_sums();

    const int8_t *xq = nullptr;
    if constexpr (FUSED) {
        constexpr int EPT = 16 / sizeof(T);
        const int32_t chunks = K / EPT;
        uint32_t(*red)[4] = (uint32_t(*)[4])(smem + FT::RED_AT);
        for (int32_t m = 0; m < M; ++m) {
            const T *x = (const T *)X + m * ldx;
            uint32_t mx = 0;
            for (int32_t q = (int32_t)threadIdx.x; q < chunks; q += THREADS)
                mx = max(mx, chunk_amax<T>(*(const i32x4 *)(x + (int64_t)q * EPT)));
#pragma unroll
            for (int d = 32; d; d >>= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, d));
            if (lane == 0) red[wave][m] = mx;
        }
        __syncthreads();
        for (int32_t m = 0; m < M; ++m) {
            const T *x = (const T *)X + m * ldx;
            uint32_t mx = 0;
#pragma unroll
            for (int w = 0; w < NW; ++w) mx = max(mx, red[w][m]);
            const RowScale rs = row_scale(widen_bits<T>(mx));
            if (threadIdx.x == 0) row_scales[m] = rs.scale;
            for (int32_t q = (int32_t)threadIdx.x; q < chunks; q += THREADS)
                put_chunk<T>((int8_t *)(smem + FT::X_AT) + (int64_t)m * K + q * EPT, *(const i32x4 *)(x + (int64_t)q * EPT), rs);
        }
        xq = (const int8_t *)(smem + FT::X_AT) + (int64_t)min(r, M - 1) * K + 16 * c;
    } else {
        if (threadIdx.x < TM) row_scales[threadIdx.x] = sx[min(m0 + (int32_t)threadIdx.x, M - 1)];
    }
    __syncthreads();

    i32x4 acc[MT][NT];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int u = 0; u < NT; ++u) acc[t][u] = i32x4{0, 0, 0, 0};
    const char *frag[S];
#pragma unroll
    for (int s = 0; s < S; ++s)
        frag[s] = smem + wave * FT::RING + (S == 1 ? 4 * r + (c ^ ((r >> 1) & 3)) : 8 * r + ((4 * s + c) ^ (r & 7))) * 16;
    for (int32_t st = first; st < last; st += S * DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            // Stage d: copied DEPTH - 1 stages ago.  (Stages past the wave's share
            // hold zeros.)
            const int32_t at = st + S * d;
            copy((d + DEPTH - 1) % DEPTH, at + S * (DEPTH - 1));
            wait_copies<(DEPTH - 1) * S * FT::BLOCKS>();
            i32x4 wf[S][NT], xf[S][MT];
#pragma unroll
            for (int s = 0; s < S; ++s) {
#pragma unroll
                for (int t = 0; t < NT; ++t) wf[s][t] = *(const i32x4 *)(frag[s] + d * FT::STAGE + S * t * 1024);
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    if constexpr (FUSED) xf[s][t] = *(const i32x4 *)(xq + min(byte_of(at + s), K - 16 - 16 * c));
                    else xf[s][t] = *(const i32x4 *)(frag[s] + d * FT::STAGE + S * (NT + t) * 1024);
                }
            }
            // the next copies overwrite what has been read here
            asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int u = 0; u < NT; ++u)
                        acc[t][u] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[s][u], xf[s][t], acc[t][u], 0, 0, 0);
        }
    }
    wait_copies<0>();
    if constexpr (FT::OVER) {
        __syncthreads();
        clear_sums();
        __syncthreads();
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) atomicAdd(&sums[(16 * u + 4 * c + e) * LD + 16 * t + r], acc[t][u][e]);
    __syncthreads();
    const bool vec = N % 4 == 0;
    for (int32_t i = (int32_t)threadIdx.x; i < TM * TN / 4; i += THREADS) {
        const int32_t m = i / (TN / 4), n = i % (TN / 4) * 4;
        if (m0 + m >= M || n0 + n >= N) continue;
        const int32_t *v = sums + n * LD + m;
        const float scale = row_scales[m];
        f32x4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = vec || n0 + n + e < N ? ((float)v[e * LD] * scale) * sw[n0 + n + e] : 0.f;
        store_scaled<T>(bias, out, (m0 + m) * (int64_t)N + n0 + n, n0 + n, N - n0 - n, vec, y);
    }
}

// Rows that every workgroup quantises for itself, and the LDS for them: four rows
// of 4096 take a workgroup about a us, a launch of their own about three.
enum { FUSED_ROWS = 4, FUSED_BYTES = 64 * 1024 };

template <class T, int MT, int NT, int S, int DEPTH, bool FUSED>
static hipError_t few_t(const void *X, int64_t ldx, const int8_t *W, const float *sx, const float *sw,
                        const void *bias, void *out, int64_t M, int64_t N, int64_t K, hipStream_t s)
{
    using FT = FewTile<MT, NT, S, DEPTH, FUSED>;
    const uint64_t tm = (uint64_t)((M + FT::TM - 1) / FT::TM), tn = (uint64_t)((N + FT::TN - 1) / FT::TN);
    if (tm * tn > 0x7FFFFFFFull) return hipErrorInvalidValue;
    static_assert(FT::X_AT + (FUSED ? FUSED_BYTES : 0) <= 160 * 1024, "LDS");
    hipLaunchKernelGGL((linear_few_kernel<T, MT, NT, S, DEPTH, FUSED>), dim3((uint32_t)(tm * tn)), dim3(64 * FT::NW),
                       (uint32_t)(FT::X_AT + (FUSED ? M * K : 0)), s, X, ldx, W, sx, sw, (const T *)bias, (T *)out,
                       (int32_t)M, (int32_t)N, (int32_t)K, (uint32_t)tm, (uint32_t)tn);
    return hipGetLastError();
}

// Which tile a product takes; 0 rows: none of these, the LDS-tiled kernels of
// lb_gemm_s8_linear.  A workgroup takes about as long whatever its tile (latency,
// and some 50 KB a us of copies to a compute unit), so the narrowest tile whose
// workgroups run at once, and the other kernels where none does.  Measured, bf16,
// weights from HBM, us here and there: 1 x 4096 x 4096 6.3 / 18.7, 16 x 8000 x 2048
// 6.0 / 10.9, 16 x 11008 x 4096 12.0 / 14.0, 32 x 6000 x 4096 10.2 / 13.8, 32 x 11008
// x 4096 13.7 / 14.7, 64 x 4096 x 4096 (16 columns) 10.9 / 28, 100 x 4096 x 4096 (32) 10.8
// / 28, 64 x 11008 x 4096 (48) 15.2 / 16.3, 256 x 4096 x 4096 (64) 13.9 / 17.7; past the
// rule 16 x 16384 x 4096 (64) 18.1 / 17.3, 128 x 8192 x 4096 (64) 15.7 / 15.4, 331 x 4097
// x 5504 (64) 32.0 / 25.2, 200 x 11008 x 4096 (64) 37.1 / 23.8.
struct FewShape {
    int tm, tn;
};
static FewShape few_shape(int64_t M, int64_t N, int cu)
{
    const int tm = M <= 16 ? 16 : M <= 32 ? 32 : 64;
    for (int tn = 16; tn <= (M > 128 ? 64 : 48); tn += 16)
        if (((M + tm - 1) / tm) * ((N + tn - 1) / tn) <= cu) return {tm, tn};
    return {0, 0};
}
bool linear_is_few(int64_t M, int64_t N, int cu) { return few_shape(M, N, cu).tm != 0; }
bool linear_few_tile(int64_t M, int64_t N, int cu, int *tm, int *tn)
{
    const FewShape f = few_shape(M, N, cu);
    *tm = f.tm;
    *tn = f.tn;
    return f.tm != 0;
}

template <class T>
static hipError_t linear_few_t(const int8_t *Xq, const int8_t *W, const float *sx, const float *sw,
                               const void *bias, void *out, int64_t M, int64_t N, int64_t K, int cu, hipStream_t s)
{
    const FewShape f = few_shape(M, N, cu);
#define LB_FEW(...) few_t<T, __VA_ARGS__, false>(Xq, K, W, sx, sw, bias, out, M, N, K, s)
    if (f.tm == 16) return f.tn == 16 ? LB_FEW(1, 1, 2, 2) : f.tn == 32 ? LB_FEW(1, 2, 1, 3) : LB_FEW(1, 3, 2, 2);
    if (f.tm == 32) return f.tn == 16 ? LB_FEW(2, 1, 2, 2) : f.tn == 32 ? LB_FEW(2, 2, 1, 3) : LB_FEW(2, 3, 1, 2);
    if (f.tm == 64 && f.tn <= 32) return f.tn == 16 ? LB_FEW(4, 1, 1, 3) : LB_FEW(4, 2, 1, 2);
    if (f.tm == 64) return f.tn == 48 ? LB_FEW(4, 3, 2, 2) : LB_FEW(4, 4, 2, 2);
#undef LB_FEW
    return hipErrorInvalidValue;
}

hipError_t launch_linear_few(int ftype, const int8_t *Xq, const int8_t *W, const float *sx, const float *sw,
                             const void *bias, void *out, int64_t M, int64_t N, int64_t K, int cu,
                             hipStream_t s)
{
    switch (ftype) {
    case LB_BF16: return linear_few_t<__bf16>(Xq, W, sx, sw, bias, out, M, N, K, cu, s);
    case LB_F16: return linear_few_t<_Float16>(Xq, W, sx, sw, bias, out, M, N, K, cu, s);
    case LB_F32: return linear_few_t<float>(Xq, W, sx, sw, bias, out, M, N, K, cu, s);
    default: return hipErrorInvalidValue;
    }
}

bool linear_fuses(int64_t M, int64_t N, int64_t K, int cu)
{
    return M <= FUSED_ROWS && M * K <= FUSED_BYTES && linear_is_few(M, N, cu);
}

template <class T>
static hipError_t linear_fused_t(const void *X, int64_t ldx, const int8_t *W, const float *sw, const void *bias,
                                 void *out, int64_t M, int64_t N, int64_t K, int cu, hipStream_t s)
{
#define LB_FUSED(...) few_t<T, __VA_ARGS__, true>(X, ldx, W, nullptr, sw, bias, out, M, N, K, s)
    switch (few_shape(M, N, cu).tn) {
    case 16: return LB_FUSED(1, 1, 2, 3);
    case 32: return LB_FUSED(1, 2, 1, 3);
    case 48: return LB_FUSED(1, 3, 1, 3);
    default: return hipErrorInvalidValue;
    }
#undef LB_FUSED
}

hipError_t launch_linear_fused(int ftype, const void *X, int64_t ldx, const int8_t *W, const float *sw,
                               const void *bias, void *out, int64_t M, int64_t N, int64_t K, int cu, hipStream_t s)
{
    if (!linear_fuses(M, N, K, cu)) return hipErrorInvalidValue;
    switch (ftype) {
    case LB_BF16: return linear_fused_t<__bf16>(X, ldx, W, sw, bias, out, M, N, K, cu, s);
    case LB_F16: return linear_fused_t<_Float16>(X, ldx, W, sw, bias, out, M, N, K, cu, s);
    case LB_F32: return linear_fused_t<float>(X, ldx, W, sw, bias, out, M, N, K, cu, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace lb
