// lb_serve_kv4.hip -- a paged cache of keys and values in 4 bits: written, read back
// and attended over.
//
// A vector x (the D numbers of one token and head) is held as levels u[d] in
// 0..15, a scale s and a minimum m, both in the type T of x:
//   m = min_d x[d],  s = T((max_d x[d] - m) / 15), or T's number before that where
//                        15 s + m would round to infinity,
//   u[d] = clamp(round_half_even((x[d] - m) / s), 0, 15)   (0 where s = 0),
// and stands for u[d] s + m.  A vector that holds an infinity or a NaN, or whose
// range is beyond fp32, stands for NaN.
#include "lb_float.hpp"
#include "lb_internal.hpp"

namespace lb {

// ---- write -----------------------------------------------------------------
// Both kernels: D/8 lanes per vector, eight numbers (16 bytes) and one word of levels
// each, of a key and its value; a workgroup takes neighbouring tokens of one head,
// whose levels lie next to each other in the cache where their slots do, and the
// next workgroup the next head of the same tokens, whose numbers lie next to theirs.
// 32768 tokens of 8 heads of 128 in bf16 are written in 53 us, 3.2 TB/s, bound by its
// vector instructions (2.95e7, 450 a wave; at 4 cycles each on 1024 SIMDs of 2.1 GHz
// 55 us); 40000 are read back in 40.0 us, 5.1 TB/s, what a copy reaches.  A few tokens
// take the latency of a launch, 3.5 and 2.8 us.

// slot / page by a multiplication (page_mul is 2^(32 + page_shift) / page rounded up).
__device__ inline int32_t slot_page(const Kv4Cache &c, int64_t slot) { return (int32_t)(__umulhi((uint32_t)slot, c.page_mul) >> c.page_shift); }

// Least (most) of x over the N lanes (8, 16 or 32) of a vector, in all of them.
template <int CTRL> __device__ inline float lane_dpp(float x)
{
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xF, 0xF, true));
}
template <int N, class F> __device__ inline float over_lanes(float x, F f)
{
    x = f(x, lane_dpp<0xB1>(x));     // lane ^ 1
    x = f(x, lane_dpp<0x4E>(x));     // lane ^ 2
    x = f(x, lane_dpp<0x141>(x));    // the other four of eight, mirrored
    if constexpr (N >= 16) x = f(x, lane_dpp<0x140>(x));   // the other eight of sixteen
    if constexpr (N >= 32) x = f(x, __shfl_xor(x, 16));
    return x;
}

// (x - m) / s decides between levels at half-integers.  The product with 1/s (one
// step off at most) is off by less than 2^-18 (15 * 4 * 2^-24), so it settles the
// levels unless one lies within 2^-16 of a half-integer; then the correctly rounded
// quotients decide (a division for every number made the kernel's time that of its
// vector instructions).  So they do for subnormal scales, whose rounding may put the
// largest number past 15.5; a normal one puts it below 15.2.  A slot outside the
// cache is not written.
template <class T, int D>
__device__ inline void write_vector(const Kv4Cache &c, i32x4 w, int64_t slot, int32_t h, uint32_t sub, uint8_t *levels,
                                    uint32_t *params)
{
    constexpr int LPV = D / 8;
    float x[8];
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = lo_f32<T>((uint32_t)w[i]);
        x[2 * i + 1] = hi_f32<T>((uint32_t)w[i]);
        odd |= __builtin_isunordered(x[2 * i], x[2 * i + 1]);
    }
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
    }
    lo = over_lanes<LPV>(lo, [](float p, float q) { return fminf(p, q); });
    hi = over_lanes<LPV>(hi, [](float p, float q) { return fmaxf(p, q); });
    float s = (float)(T)((hi - lo) / 15.0f);
    // where T's rounding of 15 s + lo becomes infinite (the quotient was rounded up)
    if (__builtin_fmaf(15.f, s, lo) >= (__is_same(T, __bf16) ? 0x1.FFp127f : 65520.f) && s < __builtin_inff()) {
        if constexpr (__is_same(T, __bf16)) s = __uint_as_float(__float_as_uint(s) - 0x10000u);
        else s = lo_f32<T>(pack2<T>(s, 0.f) - 1u);
    }
    // a NaN, or a range that is not finite
    const uint64_t odds = __ballot(odd) >> ((threadIdx.x & 63u) / LPV * LPV);
    const bool bad = (odds & (((uint64_t)1 << LPV) - 1)) != 0 || !(s < __builtin_inff());
    uint32_t word = 0;
    if (s > 0.f && !bad) {
        const float inv = __builtin_amdgcn_rcpf(s);
        float n[8], far = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = (x[i] - lo) * inv;
            n[i] = __builtin_rintf(q);
            far = fmaxf(far, __builtin_fabsf(q - n[i]));
        }
        if (far > 0.5f - 0x1p-16f || s < (__is_same(T, __bf16) ? 0x1p-100f : 0x1p-14f)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) n[i] = fminf(__builtin_rintf((x[i] - lo) / s), 15.f);
        }
        uint32_t even = 0, odd_levels = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            even = __builtin_amdgcn_cvt_pk_u8_f32(n[2 * i], (uint32_t)i, even);
            odd_levels = __builtin_amdgcn_cvt_pk_u8_f32(n[2 * i + 1], (uint32_t)i, odd_levels);
        }
        word = even | odd_levels << 4;
    }
    if ((uint64_t)slot >= (uint64_t)(c.pages * c.page)) return;
    const int32_t p = slot_page(c, slot);
    const int64_t at = ((int64_t)p * c.heads + h) * c.page + ((int32_t)slot - p * c.page);
    ((uint32_t *)levels)[at * LPV + sub] = word;
    if (sub == 0) {
        const float nan = __uint_as_float(0x7FC00000u);
        params[at] = bad ? pack2<T>(nan, nan) : pack2<T>(s, lo);
    }
}

template <class T, int D>
__global__ __launch_bounds__(256) void kv4_write_kernel(const T *__restrict__ K, const T *__restrict__ V,
                                                        int64_t ldk, int64_t ldv,
                                                        const int64_t *__restrict__ slots, Kv4Cache c,
                                                        int64_t tokens)
{
    constexpr int LPV = D / 8;
    const uint32_t group = blockIdx.x / (uint32_t)c.heads;
    const int32_t h = (int32_t)(blockIdx.x - group * (uint32_t)c.heads);
    const int64_t t = (int64_t)group * (256 / LPV) + threadIdx.x / LPV;
    const uint32_t sub = threadIdx.x % LPV;
    if (t >= tokens) return;  // whole vectors
    const int64_t slot = slots[t];
    const i32x4 k = *(const i32x4 *)(K + t * ldk + h * D + sub * 8);
    const i32x4 v = *(const i32x4 *)(V + t * ldv + h * D + sub * 8);
    write_vector<T, D>(c, k, slot, h, sub, c.k, c.kp);
    write_vector<T, D>(c, v, slot, h, sub, c.v, c.vp);
}

// ---- read back -------------------------------------------------------------
// One rounding, of u s + m (u s is exact in fp32).  A slot outside the cache
// reads as zeros.
template <class T, int D>
__global__ __launch_bounds__(256) void kv4_read_kernel(Kv4Cache c, const int64_t *__restrict__ slots,
                                                       T *__restrict__ K, T *__restrict__ V, int64_t tokens)
{
    constexpr int LPV = D / 8;
    const uint32_t group = blockIdx.x / (uint32_t)c.heads;
    const int32_t h = (int32_t)(blockIdx.x - group * (uint32_t)c.heads);
    const int64_t t = (int64_t)group * (256 / LPV) + threadIdx.x / LPV;
    const uint32_t sub = threadIdx.x % LPV;
    if (t >= tokens) return;
    const int64_t slot = slots[t];
    i32x4 o[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    if ((uint64_t)slot < (uint64_t)(c.pages * c.page)) {
        const int32_t p = slot_page(c, slot);
        const int64_t at = ((int64_t)p * c.heads + h) * c.page + ((int32_t)slot - p * c.page);
        const uint32_t w[2] = {((const uint32_t *)c.k)[at * LPV + sub], ((const uint32_t *)c.v)[at * LPV + sub]};
        const uint32_t prm[2] = {c.kp[at], c.vp[at]};
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const float s = lo_f32<T>(prm[x]), m = hi_f32<T>(prm[x]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[x][i] = (int)pack2<T>((float)((w[x] >> (8 * i)) & 15u) * s + m,
                                        (float)((w[x] >> (8 * i + 4)) & 15u) * s + m);
        }
    }
    const int64_t to = (t * c.heads + h) * D + sub * 8;
    *(i32x4 *)(K + to) = o[0];
    *(i32x4 *)(V + to) = o[1];
}

template <class T, int D>
static hipError_t write_t(const void *K, const void *V, int64_t ldk, int64_t ldv, const int64_t *slots,
                          const Kv4Cache &c, int64_t T_, hipStream_t s)
{
    const int64_t most = LAUNCH_THREADS / 256 / c.heads * (2048 / D);   // tokens of a launch
    for (int64_t t = 0; t < T_; t += most) {
        const int64_t n = T_ - t < most ? T_ - t : most, blocks = (n + 2048 / D - 1) / (2048 / D) * c.heads;
        hipLaunchKernelGGL((kv4_write_kernel<T, D>), dim3((uint32_t)blocks), dim3(256), 0, s,
                           (const T *)K + t * ldk, (const T *)V + t * ldv, ldk, ldv, slots + t, c, n);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}
template <class T, int D>
static hipError_t read_t(const Kv4Cache &c, const int64_t *slots, void *K, void *V, int64_t T_, hipStream_t s)
{
    const int64_t most = LAUNCH_THREADS / 256 / c.heads * (2048 / D), row = (int64_t)c.heads * D;
    for (int64_t t = 0; t < T_; t += most) {
        const int64_t n = T_ - t < most ? T_ - t : most, blocks = (n + 2048 / D - 1) / (2048 / D) * c.heads;
        hipLaunchKernelGGL((kv4_read_kernel<T, D>), dim3((uint32_t)blocks), dim3(256), 0, s, c,
                           slots + t, (T *)K + t * row, (T *)V + t * row, n);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

#define LB_KV4_BY_TYPE(CALL)                                   \
    if (ftype == LB_BF16) {                                    \
        if (D == 64) return CALL(__bf16, 64);                  \
        if (D == 128) return CALL(__bf16, 128);                \
        if (D == 256) return CALL(__bf16, 256);                \
    } else if (ftype == LB_F16) {                              \
        if (D == 64) return CALL(_Float16, 64);                \
        if (D == 128) return CALL(_Float16, 128);              \
        if (D == 256) return CALL(_Float16, 256);              \
    }                                                          \
    return hipErrorInvalidValue;

hipError_t launch_kv4_write(int ftype, const void *K, const void *V, int64_t ldk, int64_t ldv,
                            const int64_t *slots, const Kv4Cache &c, int64_t T, int D, hipStream_t s)
{
#define CALL(TY, DD) write_t<TY, DD>(K, V, ldk, ldv, slots, c, T, s)
    LB_KV4_BY_TYPE(CALL)
#undef CALL
}
hipError_t launch_kv4_read(int ftype, const Kv4Cache &c, const int64_t *slots, void *K, void *V, int64_t T,
                           int D, hipStream_t s)
{
#define CALL(TY, DD) read_t<TY, DD>(c, slots, K, V, T, s)
    LB_KV4_BY_TYPE(CALL)
#undef CALL
}

// ---- attention -------------------------------------------------------------
// The rows of one sequence and key head: query i and head j of the group is row
// i * group + j; query i stands at position len - nq + i and sees the keys
// [lo, hi) with hi = position + 1 (causal) or len, lo = position - window + 1
// (window > 0) or 0.
//
// Scores without ever scaling a key: u s + m is linear in u, so
//   q . k = s (sum_d q[d] u[d]) + m (sum_d q[d]),
// and the first sum runs on the matrix cores with the levels exact in T.  A
// nibble becomes a T by writing it into the mantissa of a power of two,
// B + u (bf16: B = 128, fp16: B = 64): one AND-OR for two nibbles, and a
// constant to take off, -B sum_d q[d], which is the accumulator's start.  (The fp32 sums
// are then of numbers up to 10 times the levels', and so are their roundings: 7e-6 of
// a score at most in 65536 ordinary keys, where the plain sum's are 1e-6.)
// The values are summed the same way with the weights carrying the scale:
//   sum_t p[t] v[t,d] = sum_t (p[t] s[t]) u[t,d] + sum_t p[t] m[t].
// The weight p s goes in two bf16 parts (16 bits in all, off by 2^-17, with fp32's
// range, which fp16 scales or weights would not have; over 131072 keys outputs are
// off by 5e-5 before their rounding, a tenth of fp16's half step), and the sum of both parts, by one more
// product with ones, takes off what the nibbles' power of two adds.
template <class T> struct Mfma;
// A constant kept in a vector register: AND-OR takes one scalar operand, and with
// mask and magic both scalar the compiler makes two instructions of it.
__device__ inline uint32_t in_vgpr(uint32_t x)
{
    asm volatile("" : "+v"(x));
    return x;
}
// The low halves, and the high halves, of two words.
__device__ inline uint32_t low_halves(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
__device__ inline uint32_t high_halves(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }
template <> struct Mfma<__bf16> {
    typedef bf16x8 frag;
    static constexpr float base = 128.f;
    static constexpr uint32_t magic = 0x43004300u, mask = 0x000F000Fu;
    static __device__ inline f32x4 mul(i32x4 a, i32x4 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(frag, a), __builtin_bit_cast(frag, b), c,
                                                       0, 0, 0);
    }
    // nibbles i and i+4 of w as a pair; mg is in_vgpr(magic)
    static __device__ inline uint32_t pair(uint32_t w, int i, uint32_t mg) { return ((w >> (4 * i)) & mask) | mg; }
};
template <> struct Mfma<_Float16> {
    typedef f16x8 frag;
    static constexpr float base = 64.f;
    static constexpr uint32_t magic = 0x54005400u, mask = 0x00F000F0u;
    static __device__ inline f32x4 mul(i32x4 a, i32x4 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(frag, a), __builtin_bit_cast(frag, b), c,
                                                      0, 0, 0);
    }
    static __device__ inline uint32_t pair(uint32_t w, int i, uint32_t mg)
    {
        return ((i == 0 ? w << 4 : w >> (4 * i - 4)) & mask) | mg;
    }
};
using MfmaV = Mfma<__bf16>;  // the values' product, whatever T is

// Eight numbers of a query in the order of a word's nibble pairs: element 2i is
// number i, element 2i+1 number i+4.
__device__ inline i32x4 query_order(i32x4 w)
{
    const uint32_t w0 = (uint32_t)w.x, w1 = (uint32_t)w.y, w2 = (uint32_t)w.z, w3 = (uint32_t)w.w;
    return i32x4{(int)((w0 & 0xFFFFu) | (w2 << 16)), (int)((w0 >> 16) | (w2 & 0xFFFF0000u)),
                 (int)((w1 & 0xFFFFu) | (w3 << 16)), (int)((w1 >> 16) | (w3 & 0xFFFF0000u))};
}

// What one workgroup of an attention kernel works on.
struct Span {
    int32_t n, nq, rows;   // keys and queries of the sequence, rows of its key head
    int64_t q0;            // first query
};
__device__ inline Span lane_span_of(const AttnArgs &a, int32_t b)   // b may differ between lanes
{
    Span s;
    const int64_t cap = a.width * a.c.page;
    const int64_t n = a.lens[b];
    s.n = (int32_t)(n < 0 ? 0 : n > cap ? cap : n);
    int64_t q0 = a.q_off[b], q1 = a.q_off[b + 1];
    q0 = q0 < 0 ? 0 : q0 > a.total_q ? a.total_q : q0;
    q1 = q1 < q0 ? q0 : q1 > a.total_q ? a.total_q : q1;
    s.q0 = q0;
    s.nq = (int32_t)(q1 - q0);
    s.rows = s.nq * a.group;
    return s;
}
__device__ inline Span span_of(const AttnArgs &a, int32_t b)        // b is the same in all
{
    Span s = lane_span_of(a, b);
    s.n = __builtin_amdgcn_readfirstlane(s.n);
    s.nq = __builtin_amdgcn_readfirstlane(s.nq);
    s.q0 = __builtin_amdgcn_readfirstlane((int32_t)s.q0);
    s.rows = s.nq * a.group;
    return s;
}
__device__ inline int32_t page_of(const AttnArgs &a, int32_t key) { return slot_page(a.c, key); }
// A page number of the table, by a scalar load.
__device__ inline int32_t page_number(const AttnArgs &a, int32_t b, int32_t key)
{
    typedef const __attribute__((address_space(4))) int32_t *const_ptr;
    return ((const_ptr)(uintptr_t)(a.table + (int64_t)b * a.ldt))[page_of(a, key)];
}

__device__ inline int32_t key_hi(const AttnArgs &a, const Span &s, int32_t qi)
{
    return a.causal ? max(0, min(s.n, s.n - s.nq + qi + 1)) : s.n;
}
__device__ inline int32_t key_lo(const AttnArgs &a, const Span &s, int32_t qi)
{
    // (a position before the first key counts as the first, or the largest windows would overflow)
    return a.window > 0 ? max(0, max(0, s.n - s.nq + qi + 1) - a.window) : 0;
}

// Keys that some row of r0 .. r0 + n - 1 sees.
__device__ inline void tile_keys(const AttnArgs &a, const Span &sp, int32_t r0, int32_t n, int32_t &lo, int32_t &hi)
{
    lo = key_lo(a, sp, r0 / a.group);
    hi = key_hi(a, sp, min(r0 + n - 1, sp.rows - 1) / a.group);
}

// Row `row` of key head h, dims oc D/16 .. of it: o / l, and m + log2(l).
template <class T, int D>
__device__ inline void rows_out(const AttnArgs &a, const Span &sp, int32_t h, int32_t row, int32_t oc,
                                const float (&o)[D / 16], float m, float l)
{
    const int32_t oq = row / a.group, oh = h * a.group + (row - oq * a.group);
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    T *po = (T *)a.out + (sp.q0 + oq) * a.ldo + (int64_t)oh * D + oc * (D / 16);
#pragma unroll
    for (int j = 0; j < D / 16; j += 2) *(uint32_t *)(po + j) = pack2<T>(o[j] * inv, o[j + 1] * inv);
    if (a.lse && oc == 0)
        a.lse[(sp.q0 + oq) * (int64_t)(a.group * a.c.heads) + oh] =
            l == 0.f ? -__builtin_inff() : (m + __builtin_log2f(l)) * 0.6931471805599453f;
}

// How the keys [lo, hi) of a tile of rows are shared where each tile is cut by
// itself: nb blocks of keys from block b0, `per` to a workgroup, `ranges` workgroups
// (at most a.splits; one writes the output itself).
struct Ranges {
    int32_t b0, nb, per, ranges;
};
template <int BLOCK> __device__ inline Ranges ranges_of(const AttnArgs &a, int32_t lo, int32_t hi)
{
    Ranges s;
    s.b0 = lo / BLOCK;
    s.nb = max(0, (hi + BLOCK - 1) / BLOCK - s.b0);
    s.per = max(a.unit, (s.nb + a.splits - 1) / a.splits);
    s.ranges = max(1, (s.nb + s.per - 1) / s.per);
    return s;
}

__device__ inline float max_over_groups(float x)
{
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}
__device__ inline float sum_over_groups(float x)
{
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

// A sum of many blocks' sums, with what each addition rounds away carried to the next:
// a running fp32 sum drops weights below 2^-24 of it however many they are (20000 of
// 2^-24.4 beside a 1: 9e-5 of it, and 131072 equal weights were off by as much).
struct LongSum {
    float s = 0.f, over = 0.f;   // over: what s holds too much
    __device__ inline void add(float t)
    {
        const float y = t - over, n = s + y;
        over = (n - s) - y;
        s = n;
    }
    __device__ inline void scale(float f)   // by a power of two, or about one
    {
        s *= f;
        over *= f;
    }
};

// Sixteen rows (r0 ..) of a key head against blocks [first, last) of 32 keys.  Each
// of NW waves takes its share of the blocks (two half-blocks of 16 keys, each inside
// one page) and keeps its own maximum, sum and output; they meet in LDS.  part: where
// the rows' outputs (16 x D), maxima and sums (16 x 2) go unweighted, or null where
// these are all their keys and the output is written.  Lane l = 16 c + r:
//   scores    A: key r of a half-block, levels [c D/4, (c+1) D/4);  B: row r.
//             It ends with keys 4c .. 4c+3 of each half-block for row r;
//   values    those eight keys are its share of the contraction as they stand:
//             B: their weights; A: their levels of dims r D/16 .. (r+1) D/16 - 1,
//             one MFMA per dim.  It ends with dims (4c+i) D/16 + j of row r.
// Neither the weights nor the values change lanes, and nothing passes through LDS.
// Bound by the cache's bytes where keys are many: 8 heads of 128 of two sequences of
// 131072 keys (285 MB) in 58 us, 4.9 TB/s, what a copy reaches; by latency where they
// are few: one sequence of 777 keys 11.3 us, 12 sequences of 5 queries over windows
// of 1024 keys, 32 heads of 64, 15.0 us.
// The next block's keys are asked for as soon as this one's are multiplied, its
// values as soon as this one's are, into the same registers, and the numbers of
// its pages a block earlier.  (Two blocks' worth of registers cost more in waves
// per SIMD than the longer lead gave.)
template <int D, int NW> struct RowsLds {
    static constexpr int LDO = D + 4;
    float osum[NW * 16 * LDO];
    float stat[NW][16][4];
};

template <class T, int D, int NW>
__device__ __forceinline__ void rows_segment(const AttnArgs &a, RowsLds<D, NW> &lds, const Span &sp, int32_t b, int32_t h,
                                             int32_t r0, int32_t lo, int32_t hi, int32_t first, int32_t last, float *part)
{
    using MM = Mfma<T>;
    constexpr int KW = D / 32;     // words of a key a lane reads, = MFMAs per half-block
    constexpr int DPL = D / 16;    // dims of a value a lane reads, = MFMAs per block
    constexpr int VW = DPL / 8 ? DPL / 8 : 1;
    constexpr int LDO = RowsLds<D, NW>::LDO;
    auto &osum = lds.osum;
    auto &stat = lds.stat;
    const uint32_t lane = threadIdx.x & 63u;
    const int32_t wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int32_t r = (int32_t)(lane & 15u), c = (int32_t)(lane >> 4);
    const int32_t qi_first = r0 / a.group, qi_last = min(r0 + 15, sp.rows - 1) / a.group;

    uint32_t kw[2][KW], vw[8][VW];
    u32x4 kp[2], vp[2];
    const int32_t hi16 = max(hi - 1, 0) & ~15;
    const int64_t head_at = (int64_t)h * a.c.page, page_step = (int64_t)a.c.heads * a.c.page;
    int32_t pages[2];
    int64_t at[2];           // first vector of the half-blocks asked for
    bool there[2], there1[2];
    // (past the range the last half-block is read again)
    auto ask = [&](int32_t blk) {
#pragma unroll
        for (int s = 0; s < 2; ++s) pages[s] = page_number(a, b, min(32 * blk + 16 * s, hi16));
    };
    auto fetch_keys = [&](int32_t blk) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int32_t t = min(32 * blk + 16 * s, hi16), p = pages[s];
            there1[s] = (uint32_t)p < (uint32_t)a.c.pages;
            at[s] = (there1[s] ? p : 0) * page_step + head_at + (t - page_of(a, t) * a.c.page);
            const uint32_t *kk = (const uint32_t *)(a.c.k + at[s] * (D / 2)) + r * (D / 8) + c * KW;
#pragma unroll
            for (int j = 0; j < KW; ++j) kw[s][j] = kk[j];
            kp[s] = *(const u32x4 *)(a.c.kp + at[s] + 4 * c);
        }
    };
    auto fetch_vals = [&]() {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            vp[s] = *(const u32x4 *)(a.c.vp + at[s] + 4 * c);
            const uint8_t *v = a.c.v + at[s] * (D / 2) + 4 * c * (D / 2) + r * (DPL / 2);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (DPL == 4) vw[4 * s + i][0] = *(const uint16_t *)(v + i * (D / 2));
                else
#pragma unroll
                    for (int j = 0; j < VW; ++j) vw[4 * s + i][j] = ((const uint32_t *)(v + i * (D / 2)))[j];
            }
        }
    };
    const int32_t mine = first + wave;
    if (mine < last) {
        ask(mine);
        fetch_keys(mine);
        fetch_vals();
        ask(mine + NW);
    }

    const int32_t row = min(r0 + r, sp.rows - 1);
    const int32_t qi = row / a.group, hq = h * a.group + (row - qi * a.group);
    const int32_t my_lo = key_lo(a, sp, qi), my_hi = key_hi(a, sp, qi);
    const int32_t full_lo = key_lo(a, sp, qi_last), full_hi = key_hi(a, sp, qi_first);
    i32x4 qf[KW];
    float qsum = 0.f;
    {
        const T *q = (const T *)a.q + (sp.q0 + qi) * a.ldq + (int64_t)hq * D + c * (D / 4);
#pragma unroll
        for (int j = 0; j < KW; ++j) {
            const i32x4 w = *(const i32x4 *)(q + 8 * j);
#pragma unroll
            for (int i = 0; i < 4; ++i) qsum += lo_f32<T>((uint32_t)w[i]) + hi_f32<T>((uint32_t)w[i]);
            qf[j] = query_order(w);
        }
        qsum = sum_over_groups(qsum);
    }
    const float start = -MM::base * qsum, qsum2 = qsum * a.scale2;

    const float NEG = -__builtin_inff();
    float m_run = NEG, pm = 0.f;
    LongSum l_run;
    f32x4 acc[DPL], ones = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < DPL; ++j) acc[j] = f32x4{0, 0, 0, 0};
    const uint32_t mk = in_vgpr(MM::magic), mv = in_vgpr(MfmaV::magic);
    const i32x4 one = {0x3F803F80, 0x3F803F80, 0x3F803F80, 0x3F803F80};

    for (int32_t blk = mine; blk < last; blk += NW) {
        const int32_t t0 = blk * 32;
        there[0] = there1[0];
        there[1] = there1[1];
        // scores in units of log 2 above the running maximum
        float sc[2][4];
        const float top = m_run == NEG ? 0.f : m_run;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            f32x4 x = {start, start, start, start};
#pragma unroll
            for (int j = 0; j < KW; ++j) {
                const uint32_t w = kw[s][j];
                x = MM::mul(i32x4{(int)MM::pair(w, 0, mk), (int)MM::pair(w, 1, mk), (int)MM::pair(w, 2, mk),
                                  (int)MM::pair(w, 3, mk)},
                            qf[j], x);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sc[s][i] = __builtin_fmaf(lo_f32<T>(kp[s][i]), x[i] * a.scale2,
                                          __builtin_fmaf(hi_f32<T>(kp[s][i]), qsum2, -top));
        }
        fetch_keys(blk + NW);
        ask(blk + 2 * NW);
        const bool whole = t0 >= full_lo && t0 + 32 <= full_hi && there[0] && there[1];
        if (!whole) {
            asm volatile("" ::: "memory");  // keeps the comparisons in this branch
            const int32_t from = my_lo - t0 - 4 * c, to = my_hi - t0 - 4 * c;
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool ok = 16 * s + i >= from && 16 * s + i < to && there[s];
                    if (!ok) {  // whatever the place holds
                        sc[s][i] = NEG;
                        vp[s][i] = 0;
                    }
                }
        }
        // The running maximum is taken anew only when a score passes it by 2^8, and
        // first of all; only then do the lanes of a row compare.
        float mx = sc[0][0];
#pragma unroll
        for (int e = 1; e < 8; ++e) mx = fmaxf(mx, sc[e / 4][e % 4]);
        if (__any(mx > 8.f || m_run == NEG)) {
            const float m_new = fmaxf(m_run, max_over_groups(mx) + top);
            const float m_use = m_new == NEG ? 0.f : m_new;
            const float al = m_run == NEG ? 0.f : __builtin_amdgcn_exp2f(m_run - m_new);
#pragma unroll
            for (int e = 0; e < 8; ++e) sc[e / 4][e % 4] += top - m_use;
            m_run = m_new;
            l_run.scale(al);
            pm *= al;
            ones *= al;
#pragma unroll
            for (int j = 0; j < DPL; ++j) acc[j] *= al;
        }
        i32x4 whi, wlo;
        float sum = 0.f;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float p = __builtin_amdgcn_exp2f(sc[s][i]);
                sum += p;
                pm = __builtin_fmaf(p, hi_f32<T>(vp[s][i]), pm);
                w[i] = p * lo_f32<T>(vp[s][i]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t hi2 = pack2<__bf16>(w[2 * i], w[2 * i + 1]);
                whi[2 * s + i] = (int)hi2;
                wlo[2 * s + i] = (int)pack2<__bf16>(w[2 * i] - lo_f32<__bf16>(hi2), w[2 * i + 1] - hi_f32<__bf16>(hi2));
            }
        }
        l_run.add(sum);
        // values
        ones = MfmaV::mul(one, whi, ones);
        ones = MfmaV::mul(one, wlo, ones);
#pragma unroll
        for (int v = 0; v < VW; ++v)
#pragma unroll
            for (int half = 0; half < (DPL == 4 ? 1 : 2); ++half) {
                uint32_t x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t u0 = vw[2 * i][v], u1 = vw[2 * i + 1][v];
                    x[i] = half ? high_halves(u0, u1) : low_halves(u0, u1);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    i32x4 f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[i] = (int)MfmaV::pair(x[i], j, mv);
                    const int d = 8 * v + 4 * half + j;
                    acc[d] = MfmaV::mul(f, whi, acc[d]);
                    acc[d] = MfmaV::mul(f, wlo, acc[d]);
                }
            }
        fetch_vals();
    }

    // the waves' results
    const float l_wave = sum_over_groups(l_run.s);
    pm = sum_over_groups(pm);
    if (c == 0) {
        stat[wave][r][0] = m_run;
        stat[wave][r][1] = l_wave;
        stat[wave][r][2] = pm;
    }
    const float off = MfmaV::base * ones.x;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < DPL; ++j)
            osum[((int)wave * 16 + r) * LDO + (4 * c + i) * DPL + j] = acc[j][i] - off;
    __syncthreads();
    const int32_t orow = (int32_t)threadIdx.x / 16, oc = (int32_t)threadIdx.x % 16;
    if (orow >= 16 || r0 + orow >= sp.rows) return;
    float m = NEG;
#pragma unroll
    for (int w = 0; w < NW; ++w) m = fmaxf(m, stat[w][orow][0]);
    float o[DPL], l = 0.f, pmt = 0.f;
#pragma unroll
    for (int j = 0; j < DPL; ++j) o[j] = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        if (stat[w][orow][1] == 0.f) continue;  // nothing seen (a NaN score leaves a NaN sum)
        const float f = __builtin_amdgcn_exp2f(stat[w][orow][0] - m);
        l += f * stat[w][orow][1];
        pmt += f * stat[w][orow][2];
#pragma unroll
        for (int j = 0; j < DPL; ++j) o[j] += f * osum[(w * 16 + orow) * LDO + oc * DPL + j];
    }
    if (part) {
#pragma unroll
        for (int j = 0; j < DPL; ++j) part[orow * D + oc * DPL + j] = o[j] + pmt;
        if (oc == 0) *(f32x2 *)(part + 16 * D + 2 * orow) = f32x2{m, l};
        return;
    }
#pragma unroll
    for (int j = 0; j < DPL; ++j) o[j] += pmt;
    rows_out<T, D>(a, sp, h, r0 + orow, oc, o, m, l);
}

// Where a workgroup leaves a part of a tile: outputs, maxima and sums of 16 rows.
template <int D> struct Part {
    static constexpr int64_t FLOATS = 16 * (D + 2);
};

// Row `row` of a tile joined from n parts, part k at part_of(k), in their order.
template <class T, int D, class F>
__device__ inline void join_parts(const AttnArgs &a, const Span &sp, int32_t h, int32_t r0, int32_t n, F part_of)
{
    constexpr int DPL = D / 16;
    const int32_t orow = (int32_t)threadIdx.x / 16, oc = (int32_t)threadIdx.x % 16;
    if (r0 + orow >= sp.rows) return;
    float m = -__builtin_inff(), l = 0.f, o[DPL];
#pragma unroll
    for (int j = 0; j < DPL; ++j) o[j] = 0.f;
    for (int32_t k0 = 0; k0 < n; k0 += 8) {
        f32x2 ml[8];
        float v[8][DPL];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float *part = part_of(min(k0 + k, n - 1));
            ml[k] = *(const f32x2 *)(part + 16 * D + 2 * orow);
#pragma unroll
            for (int j = 0; j < DPL; ++j) v[k][j] = part[orow * D + oc * DPL + j];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k0 + k >= n || ml[k].y == 0.f) continue;   // nothing seen there
            const float m_new = fmaxf(m, ml[k].x);
            const float f0 = l == 0.f ? 0.f : __builtin_amdgcn_exp2f(m - m_new);
            const float f1 = __builtin_amdgcn_exp2f(ml[k].x - m_new);
            m = m_new;
            l = l * f0 + f1 * ml[k].y;
#pragma unroll
            for (int j = 0; j < DPL; ++j) o[j] = o[j] * f0 + f1 * v[k][j];
        }
    }
    rows_out<T, D>(a, sp, h, r0 + orow, oc, o, m, l);
}

// A tile of sixteen rows, or a range of its keys, to a workgroup.
template <class T, int D, int NW>
__global__ __launch_bounds__(64 * NW, NW == 4 ? (D == 256 ? 2 : 3) : NW / 4) void attn_rows_kernel(AttnArgs a)
{
    __shared__ RowsLds<D, NW> lds;
    const int32_t bh = (int32_t)(blockIdx.x / (uint32_t)a.tiles), tile = (int32_t)(blockIdx.x % (uint32_t)a.tiles);
    const int32_t b = bh / a.c.heads, h = bh - b * a.c.heads;
    const Span sp = span_of(a, b);
    const int32_t r0 = tile * 16;
    if (r0 >= sp.rows) return;
    int32_t lo, hi;
    tile_keys(a, sp, r0, 16, lo, hi);
    const Ranges rg = ranges_of<32>(a, lo, hi);
    if ((int32_t)blockIdx.y >= rg.ranges) return;
    const int32_t first = rg.b0 + (int32_t)blockIdx.y * rg.per, last = min(rg.b0 + rg.nb, first + rg.per);
    rows_segment<T, D, NW>(a, lds, sp, b, h, r0, lo, hi, first, last,
                           rg.ranges == 1 ? nullptr
                                          : a.part + ((int64_t)blockIdx.x * a.splits + blockIdx.y) * Part<D>::FLOATS);
}

template <class T, int D> __global__ __launch_bounds__(256) void attn_rows_join_kernel(AttnArgs a)
{
    const int32_t bh = (int32_t)(blockIdx.x / (uint32_t)a.tiles), tile = (int32_t)(blockIdx.x % (uint32_t)a.tiles);
    const int32_t b = bh / a.c.heads, h = bh - b * a.c.heads;
    const Span sp = span_of(a, b);
    const int32_t r0 = tile * 16;
    if (r0 >= sp.rows) return;
    int32_t lo, hi;
    tile_keys(a, sp, r0, 16, lo, hi);
    const Ranges rg = ranges_of<32>(a, lo, hi);
    if (rg.ranges == 1) return;
    join_parts<T, D>(a, sp, h, r0, rg.ranges,
                     [&](int32_t k) { return a.part + ((int64_t)blockIdx.x * a.splits + k) * Part<D>::FLOATS; });
}

// The tiles of all sequences laid end to end, FLAT_COST units for a tile's start
// (which takes about as long as that many blocks) and one for each of its blocks, and
// cut into equal shares, one to a workgroup: lengths may differ as they like, and
// every compute unit has the same work.  Tiles that are nearly equal anyway, and no
// more than there are workgroups, stay whole, one to each.  A share's cut tiles leave
// their parts, the one that continues from the share before in part 2 i, the one that
// goes on in the next in 2 i + 1; the workgroup that ends a cut tile notes where it
// started, for attn_flat_join_kernel.  (64 sequences of 1 to 8191 keys, 8 heads of 128,
// 286 MB: 67 us, 4.3 TB/s, and 5 us for the join.)
enum { FLAT_COST = 14, FLAT_LEAST = 24, FLAT_BATCH = ATTN_FLAT_BATCH };
template <class T, int D>
__global__ __launch_bounds__(256, D == 256 ? 2 : 3) void attn_flat_kernel(AttnArgs a)
{
    __shared__ RowsLds<D, 4> lds;
    __shared__ int64_t before[FLAT_BATCH + 1];         // units of the sequences before each
    __shared__ int32_t tiles_before[FLAT_BATCH + 1];   // and their tiles
    __shared__ int64_t wave_sum[4];
    __shared__ int32_t wave_tiles[4], wave_most[4];   // tiles, and units of the largest
    __shared__ int32_t start_b;
    const int32_t tid = (int32_t)threadIdx.x;
    const int32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    auto tile_blocks = [&](const Span &sp, int32_t r0) {
        int32_t lo, hi;
        tile_keys(a, sp, r0, 16, lo, hi);
        return max(0, (hi + 31) / 32 - lo / 32);
    };
    auto tiles_of = [&](const Span &sp) { return min((sp.rows + 15) / 16, a.tiles); };
    {
        int64_t mine[4], sum = 0;
        int32_t mine_tiles[4], count = 0, most = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int32_t b = 4 * tid + k;
            mine[k] = sum;
            mine_tiles[k] = count;
            if (b >= a.batch) continue;
            const Span sp = lane_span_of(a, b);
            const int32_t tiles = tiles_of(sp);
            int64_t u = 0;
            for (int32_t t = 0; t < tiles; ++t) {
                const int32_t len = FLAT_COST + tile_blocks(sp, 16 * t);
                u += len;
                most = max(most, len);
            }
            sum += u * a.c.heads;
            count += tiles * a.c.heads;
        }
        int64_t upto = sum;
        int32_t upto_tiles = count;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int64_t x = __shfl_up(upto, d);
            const int32_t y = __shfl_up(upto_tiles, d);
            if ((tid & 63) >= d) {
                upto += x;
                upto_tiles += y;
            }
            most = max(most, __shfl_xor(most, d));
        }
        if ((tid & 63) == 63) {
            wave_sum[wave] = upto;
            wave_tiles[wave] = upto_tiles;
            wave_most[wave] = most;
        }
        __syncthreads();
        int64_t base = upto - sum;
        int32_t base_tiles = upto_tiles - count;
        for (int w = 0; w < wave; ++w) {
            base += wave_sum[w];
            base_tiles += wave_tiles[w];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            before[4 * tid + k] = base + mine[k];
            tiles_before[4 * tid + k] = base_tiles + mine_tiles[k];
        }
        if (tid == 255) {
            before[FLAT_BATCH] = base + sum;
            tiles_before[FLAT_BATCH] = base_tiles + count;
        }
        __syncthreads();
    }
    const int64_t total = before[FLAT_BATCH];
    const int32_t tiles = tiles_before[FLAT_BATCH];
    const int64_t most = max(max(wave_most[0], wave_most[1]), max(wave_most[2], wave_most[3]));
    const bool whole = tiles <= (int32_t)gridDim.x && 8 * most * tiles <= 9 * total;
    const int64_t shares = whole ? tiles : min((int64_t)gridDim.x, max((total + FLAT_LEAST - 1) / FLAT_LEAST, (int64_t)1));
    const int64_t i = blockIdx.x;
    int32_t *note = (int32_t *)(a.part + (int64_t)gridDim.x * 2 * Part<D>::FLOATS) + 4 * i;
    if (tid == 0) note[3] = -1;
    if (i >= shares) return;
    const int64_t each = total / shares, more = total - each * shares;   // a share: `each` units, or one more
    int64_t u = each * i + min(i, more), end = u + each + (i < more);
    for (int32_t b = tid; b < a.batch; b += 256)
        if (whole ? tiles_before[b] <= i && i < tiles_before[b + 1] : before[b] <= u && u < before[b + 1]) start_b = b;
    __syncthreads();
    int32_t b = __builtin_amdgcn_readfirstlane(start_b);
    if (whole) {
        const Span sp = span_of(a, b);
        const int32_t per_head = tiles_of(sp), n = (int32_t)i - tiles_before[b];
        u = before[b] + n / per_head * ((before[b + 1] - before[b]) / a.c.heads);
        for (int32_t t = 0; t < n % per_head; ++t) u += FLAT_COST + tile_blocks(sp, 16 * t);
        end = u + 1;   // as far as the tile goes, below
    }
    while (u < end) {
        while (before[b + 1] <= u) ++b;
        b = __builtin_amdgcn_readfirstlane(b);
        const Span sp = span_of(a, b);
        const int64_t in_b = u - before[b], per_head = (before[b + 1] - before[b]) / a.c.heads;
        const int32_t h = __builtin_amdgcn_readfirstlane((int32_t)(in_b / per_head));
        int64_t from = in_b - h * per_head;
        int32_t t = 0, len = FLAT_COST + tile_blocks(sp, 0);
        while (from >= len) {
            from -= len;
            ++t;
            len = FLAT_COST + tile_blocks(sp, 16 * t);
        }
        t = __builtin_amdgcn_readfirstlane(t);
        len = __builtin_amdgcn_readfirstlane(len);
        const int32_t u0 = __builtin_amdgcn_readfirstlane((int32_t)from);
        const int32_t u1 = __builtin_amdgcn_readfirstlane(whole ? len : (int32_t)min((int64_t)len, from + (end - u)));
        int32_t lo, hi;
        tile_keys(a, sp, 16 * t, 16, lo, hi);
        const int32_t b0 = lo / 32;
        float *part = u0 == 0 && u1 == len ? nullptr : a.part + (2 * i + (u0 == 0)) * Part<D>::FLOATS;
        if (u0 > 0 && u1 == len && tid == 0) {
            const int64_t s = u - u0, wide = (each + 1) * more;   // the tile's first unit, and its share
            note[0] = b;
            note[1] = h;
            note[2] = 16 * t;
            note[3] = (int32_t)(s < wide ? s / (each + 1) : more + (s - wide) / each);
        }
        rows_segment<T, D, 4>(a, lds, sp, b, h, 16 * t, lo, hi, b0 + max(u0 - FLAT_COST, 0), b0 + max(u1 - FLAT_COST, 0), part);
        __syncthreads();
        u += u1 - u0;
    }
}

// The parts of the cut tiles, each joined where it ends, in the shares' order.
template <class T, int D>
__global__ __launch_bounds__(256) void attn_flat_join_kernel(AttnArgs a)
{
    const int32_t i = (int32_t)blockIdx.x;
    const int32_t *note = (const int32_t *)(a.part + (int64_t)gridDim.x * 2 * Part<D>::FLOATS) + 4 * (int64_t)i;
    const int32_t b = note[0], h = note[1], r0 = note[2], i0 = note[3];
    if (i0 < 0) return;
    const Span sp = span_of(a, b);
    join_parts<T, D>(a, sp, h, r0, i - i0 + 1,
                     [&](int32_t k) { return a.part + (2 * (int64_t)(i0 + k) + (k == 0)) * Part<D>::FLOATS; });
}

// ---- many rows -------------------------------------------------------------
// 32 rows per wave, 256 per workgroup (D = 256: 16 and 128, whose outputs are as
// many registers), against tiles of 64 keys that the eight
// waves turn from nibbles into matrix operands once, in LDS, for all of them
// (16 rows per wave, each turning its own, spends half its instructions there).
// The lanes' shares of a tile are attn_rows_kernel's: keys as the A operand with
// the levels exact, so that a score is (s acc + m sum q) with per-key s and m;
// a wave's weights are already the B operand of the values' product.
//
// A wave's matrix instructions of one tile run beside its vector instructions of
// another: the sums q . u of tile t + 1 beside the softmax of tile t, the values'
// product of tile t beside the turning of the values of t + 1 and the keys of
// t + 2, whose nibbles were asked for at the tile's start, and the numbers of
// their pages a tile before.  One barrier a tile.  A fragment read takes 16
// lanes' 16-byte pieces at a time, so piece p of row n (keys: D numbers of a key;
// values: 64 keys of a dim) lies at p ^ (n % 16 or n % 8) of its row: 4 cycles a
// read, counted, where rows padded by 16 bytes took 8 (and every write 8).
//
// 32 heads over 8 of 128, 700 to 2048 queries of three sequences of up to 8192 keys,
// bf16: 476 us, 757 TFLOP/s, 62% of what a large bf16 product reaches (calls back to
// back; the first ones after a pause, at a lower clock, take up to 540).  The matrix
// cores are busy for 166 us of it, the vector ALUs for about 300 (two fused
// multiply-adds, an exponential, a maximum and a sum for each score, besides the
// turning), reads of LDS for about 230; a wave waits 29% of its time.
//
// The values' product goes one of two ways:
//   whole   values are made whole, u s + m, in fp16 scaled by one power of two for
//           the workgroup, which brings the largest |m| + 16 s of its keys to about
//           2^10, and weights are fp16: both are off by 2^-12, an eighth of a bf16
//           output's own rounding.  The reference of a row's weights lies 9 octaves below
//           its largest score (at 13 the reference is taken anew more often, 495 us; at 7,
//           477), so that weights down to 2^-23 of the largest keep that precision.  A
//           lighter one is off by 2^-25 in these units, and n of them by n 2^-14 of a
//           value: where a row's outputs are not 2^10 times that (a heavy key whose own
//           value is nothing beside many light ones), the workgroup starts again with the
//           levels (1100 us where all of them do; scores of three and six times the
//           ordinary spread do not: 500 and 512).
//   levels  levels stay exact and the weights p s go in two bf16 parts, as in
//           attn_rows_kernel, with fp32's range; 656 us where the other way takes 477.
// fp16 outputs take the levels: the other way would be as coarse as they are.  For bf16
// a pass over the scales of the workgroup's keys decides (value_scale): some row may not
// see the largest value, so whole values have to hold the smallest beside it, and
// vectors that are not finite, or 2^20 apart, leave the workgroup to the levels from the start.
template <int D> struct ChunkRows {
    static constexpr int RX = D == 256 ? 1 : 2;   // 16-row fragments per wave
    static constexpr int ROWS = 8 * 16 * RX;
};
template <class T, int D, bool WHOLE> struct ChunkTile {
    static constexpr int ROWS = ChunkRows<D>::ROWS;
    static constexpr int KROW = 2 * D, VROW = 128;
    static constexpr int KBYTES = 64 * KROW, VBYTES = D * VROW;
    // per-key numbers of a tile: scale and minimum of keys (fp32), of values (fp16 or
    // fp32), and bit g in word g where half-block g's page exists
    static constexpr int FLAG_AT = (WHOLE ? 3 : 4) * 256, PBYTES = FLAG_AT + 16;
    static constexpr int V_AT = 2 * KBYTES, P_AT = V_AT + 2 * VBYTES, Q_AT = P_AT + 4 * PBYTES;
    // D = 128: the queries' fragments stay in LDS; in registers they would spill
    static constexpr bool Q_LDS = D == 128;
    static constexpr int BYTES = Q_AT + (Q_LDS ? ROWS * 2 * D : 0);
    // byte of piece 4 j + c of key n, and of piece 4 q + c of dim n
    static __device__ inline int key_at(int n, int j, int c)
    {
        return n * KROW + 16 * ((4 * j + c) ^ (n & (D == 64 ? 7 : 15)));
    }
    static __device__ inline int val_at(int n, int q, int c) { return n * VROW + 16 * ((4 * q + c) ^ (n & 7)); }
};

// The power of two by which a workgroup's values (keys first * 64 .. of them, below hi)
// fit fp16 side by side, or 0 where they do not: it brings a quarter of the largest |m| +
// 16 s to 2^8 .. 2^9, and with 2^20 between them the smallest to 2^-12, whose parts s and
// m are then off by 2^-25 at most, 2^-13 of it.  (Vectors of zeros fit beside any.)
template <class T>
__device__ inline float value_scale(const AttnArgs &a, int32_t b, int32_t h, int32_t first, int32_t last, int32_t hi,
                                    uint32_t (&red)[8][2])
{
    const uint32_t lane = threadIdx.x & 63u;
    const int32_t wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    uint32_t most = 0, least = 0xFFFFFFFFu;
    // (unsigned: the step past the last key may pass 2^31)
    const uint32_t end = (uint32_t)min(last * 64, hi);
    for (uint32_t t = (uint32_t)first * 64u + 4u * threadIdx.x; t < end; t += 2048u) {
        const int32_t pi = page_of(a, (int32_t)t), p = a.table[(int64_t)b * a.ldt + pi];
        if ((uint32_t)p >= (uint32_t)a.c.pages) continue;
        const u32x4 w = *(const u32x4 *)(a.c.vp + ((int64_t)p * a.c.heads + h) * a.c.page + ((int32_t)t - pi * a.c.page));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // a quarter of |m| + 16 s: cannot overflow for finite vectors, and orders as its
            // bits do (infinity and NaN above all)
            const uint32_t bits = __float_as_uint(0.25f * __builtin_fabsf(hi_f32<T>(w[i])) + 4.f * lo_f32<T>(w[i])) & 0x7FFFFFFFu;
            if (t + i >= (uint32_t)hi || bits == 0) continue;
            most = max(most, bits);
            least = min(least, bits);
        }
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        most = max(most, (uint32_t)__shfl_xor((int)most, d));
        least = min(least, (uint32_t)__shfl_xor((int)least, d));
    }
    if (lane == 0) {
        red[wave][0] = most;
        red[wave][1] = least;
    }
    __syncthreads();
    most = red[0][0];
    least = red[0][1];
#pragma unroll
    for (int w = 1; w < 8; ++w) {
        most = max(most, red[w][0]);
        least = min(least, red[w][1]);
    }
    most = (uint32_t)__builtin_amdgcn_readfirstlane((int)most);
    least = (uint32_t)__builtin_amdgcn_readfirstlane((int)least);
    if (most == 0) return 1.f;
    if (most >= 0x7F800000u || (most >> 23) - (least >> 23) > 20) return 0.f;
    // 2^125 at most, whose reciprocal is a normal number
    return __uint_as_float(min(254u + 8u - (most >> 23), 252u) << 23);
}

// What a workgroup of attn_chunk_kernel does: rows r0 .. of key head h against tiles
// [first, last) of 64 keys.  Not 0 (WHOLE only, nothing written): light weights count for
// more than fp16 keeps of them.
template <class T, int D, bool WHOLE>
__device__ __forceinline__ int32_t chunk_rows(const AttnArgs &a, char *smem, const Span &sp, int32_t b, int32_t h, int32_t r0,
                                           int32_t hi, const Ranges &rg, int32_t first, int32_t last, float vscale,
                                           uint32_t (&red)[8][2])
{
    using MM = Mfma<T>;
    using LT = ChunkTile<T, D, WHOLE>;
    constexpr int RX = ChunkRows<D>::RX;
    constexpr int KW = D / 32;      // MFMAs per 16 keys
    constexpr int KH = KW / 2;      // words of a key a lane turns
    constexpr int DPT = D / 64;     // dims of eight keys a lane turns
    constexpr int ND = D / 16;      // 16-dim fragments of the output
    const uint32_t lane = threadIdx.x & 63u;
    const int32_t wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int32_t r = (int32_t)(lane & 15u), c = (int32_t)(lane >> 4);
    // keys that every row of this wave sees, and the range of each of its lanes' rows
    const int32_t w0 = r0 + 16 * RX * wave;
    const bool busy = w0 < sp.rows;
    const int32_t wf = min(w0, sp.rows - 1) / a.group, wl = min(w0 + 16 * RX - 1, sp.rows - 1) / a.group;
    const int32_t full_lo = key_lo(a, sp, wl), full_hi = key_hi(a, sp, wf);
    int32_t my_lo[RX], my_hi[RX];
    i32x4 qf[RX][LT::Q_LDS ? 1 : KW];
    char *const qlds = smem + LT::Q_AT + wave * (RX * KW * 1024) + lane * 16;
    float qsum[RX];
#pragma unroll
    for (int x = 0; x < RX; ++x) {
        const int32_t row = min(w0 + 16 * x + r, sp.rows - 1);
        const int32_t qi = row / a.group, hq = h * a.group + (row - qi * a.group);
        my_lo[x] = key_lo(a, sp, qi);
        my_hi[x] = key_hi(a, sp, qi);
        const T *q = (const T *)a.q + (sp.q0 + qi) * a.ldq + (int64_t)hq * D + c * (D / 4);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < KW; ++j) {
            const i32x4 w = *(const i32x4 *)(q + 8 * j);
#pragma unroll
            for (int i = 0; i < 4; ++i) sum += lo_f32<T>((uint32_t)w[i]) + hi_f32<T>((uint32_t)w[i]);
            if constexpr (LT::Q_LDS) *(i32x4 *)(qlds + (x * KW + j) * 1024) = query_order(w);
            else qf[x][j] = query_order(w);
        }
        qsum[x] = sum_over_groups(sum);
    }

    // What a thread turns: words khalf KH .. of the levels [c D/4, (c+1) D/4) of key
    // 16 part + r; and of the values eight keys, 4 vc + i of the half-blocks 2 kb and
    // 2 kb + 1, dims vd .. vd + DPT - 1 (lanes 4 apart lie 4 dims apart, which spreads
    // their writes over the banks).
    const int32_t part = wave & 3, khalf = wave >> 2, kb = wave & 1, vc = (int32_t)(lane & 3u);
    int32_t vd;
    {
        const int32_t u = (int32_t)(lane >> 2);
        const int32_t v = DPT == 4   ? u
                          : DPT == 2 ? (u & 12) | ((u & 1) << 1) | ((u >> 1) & 1)
                                     : (u & 8) | ((u & 1) << 2) | ((u >> 1) & 3);
        vd = ((wave >> 1) * 16 + v) * DPT;
    }
    uint32_t kw[KH], vw[8], kpw, vpw;
    const uint32_t mk = in_vgpr(MM::magic), mv = in_vgpr(WHOLE ? Mfma<_Float16>::magic : MfmaV::magic);
    const int32_t hi16 = max(hi - 1, 0) & ~15;
    const int64_t head_at = (int64_t)h * a.c.page, page_step = (int64_t)a.c.heads * a.c.page;
    // Page numbers of the half-blocks to turn next, asked for a tile ahead: keys 16
    // part of one tile, values 32 kb and 32 kb + 16 of the one before it.
    int32_t pages_of_keys = 0, pages_of_vals[2] = {0, 0};
    bool there = false;
    auto ask_keys = [&](int32_t t) { pages_of_keys = page_number(a, b, min(64 * t + 16 * part, hi16)); };
    auto ask_vals = [&](int32_t t) {
        pages_of_vals[0] = page_number(a, b, min(64 * t + 32 * kb, hi16));
        pages_of_vals[1] = page_number(a, b, min(64 * t + 32 * kb + 16, hi16));
    };
    auto vector_of = [&](int32_t key, int32_t p) {
        key = min(key, hi16);
        return ((uint32_t)p < (uint32_t)a.c.pages ? p : 0) * page_step + head_at + (key - page_of(a, key) * a.c.page);
    };
    auto fetch_keys = [&](int32_t t) {
        there = (uint32_t)pages_of_keys < (uint32_t)a.c.pages;
        const int64_t at = vector_of(64 * t + 16 * part, pages_of_keys) + r;
        const uint32_t *k = (const uint32_t *)(a.c.k + at * (D / 2)) + c * KW + khalf * KH;
#pragma unroll
        for (int j = 0; j < KH; ++j) kw[j] = k[j];
        kpw = a.c.kp[at];
        vpw = a.c.vp[at];
    };
    auto fetch_vals = [&](int32_t t) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int64_t at = vector_of(64 * t + 32 * kb + 16 * s, pages_of_vals[s]) + 4 * vc;
            const uint8_t *v = a.c.v + at * (D / 2) + vd / 2;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (DPT == 4) vw[4 * s + i] = *(const uint16_t *)(v + i * (D / 2));
                else vw[4 * s + i] = v[i * (D / 2)];
            }
        }
    };
    // Turning, in units of one 16-byte write: word j of the keys, the per-key
    // numbers, dim j of the values.
    auto turn_key_word = [&](int j, char *kbuf) {
        *(i32x4 *)(kbuf + LT::key_at(16 * part + r, khalf * KH + j, c)) = i32x4{
            (int)MM::pair(kw[j], 0, mk), (int)MM::pair(kw[j], 1, mk), (int)MM::pair(kw[j], 2, mk), (int)MM::pair(kw[j], 3, mk)};
    };
    auto turn_numbers = [&](int32_t t, char *prm) {
        // (lanes and waves that share a key write the same numbers)
        float *f = (float *)prm + 16 * part + r;
        // the levels are base + u in the products
        f[0] = lo_f32<T>(kpw) * a.scale2;
        f[64] = (hi_f32<T>(kpw) - MM::base * lo_f32<T>(kpw)) * a.scale2;
        const float s0 = lo_f32<T>(vpw), m0 = hi_f32<T>(vpw);
        if constexpr (WHOLE) {
            // a key past the range or on a page that is not there counts as zeros
            const bool in = (64 * t + 16 * part + r < hi) & there;
            const float sv = s0 * vscale, mv = (m0 + 8.f * s0) * vscale;
            _Float16 *g = (_Float16 *)(prm + 512) + 16 * part + r;
            g[0] = (_Float16)(in ? sv : 0.f);
            g[64] = (_Float16)(in ? mv : 0.f);
        } else {
            f[128] = s0;
            f[192] = m0;
        }
        ((uint32_t *)(prm + LT::FLAG_AT))[part] = there ? 1u << part : 0u;
    };
    auto turn_val_dim = [&](int j, char *vbuf, const char *prm) {
        i32x4 f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t x = vw[2 * i] | (vw[2 * i + 1] << 16);
            if constexpr (DPT == 1) x >>= 4 * (vd & 1);
            if constexpr (WHOLE) {
                const char *g = prm + 512 + 2 * (32 * kb + 16 * (i / 2) + 4 * vc + 2 * (i % 2));
                const f16x2 u = __builtin_bit_cast(f16x2, Mfma<_Float16>::pair(x, j, mv)) - (_Float16)72.f;
                f[i] = __builtin_bit_cast(int, __builtin_elementwise_fma(u, *(const f16x2 *)g, *(const f16x2 *)(g + 128)));
            } else {
                f[i] = (int)MfmaV::pair(x, j, mv);
            }
        }
        *(i32x4 *)(vbuf + LT::val_at(vd + j, kb, vc)) = f;
    };
    constexpr int UNITS = DPT + KH + 1;
    auto turn_unit = [&](int u, int32_t t, char *kbuf, char *kprm, char *vbuf, const char *vprm) {
        if (u < DPT) turn_val_dim(u, vbuf, vprm);
        else if (u < DPT + KH) turn_key_word(u - DPT, kbuf);
        else turn_numbers(t, kprm);
    };
    auto turn_keys = [&](int32_t t, char *kbuf, char *prm) {
#pragma unroll
        for (int j = 0; j < KH; ++j) turn_key_word(j, kbuf);
        turn_numbers(t, prm);
    };
    auto turn_vals = [&](char *vbuf, const char *prm) {
#pragma unroll
        for (int j = 0; j < DPT; ++j) turn_val_dim(j, vbuf, prm);
    };

    const float NEG = -__builtin_inff();
    float m_run[RX], extra[RX];
    LongSum l_run[RX];
    f32x4 acc[RX][ND], ones[RX], z[RX][4];
#pragma unroll
    for (int x = 0; x < RX; ++x) {
        m_run[x] = NEG;
        extra[x] = 0.f;
        ones[x] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int d = 0; d < ND; ++d) acc[x][d] = f32x4{0, 0, 0, 0};
    }
    const i32x4 one = {0x3F803F80, 0x3F803F80, 0x3F803F80, 0x3F803F80};
    // Sums q . (base + u) of the 64 keys in kbuf, in 4 KW steps of one fragment read
    // and RX products; beside(step) adds the caller's vector instructions to a step.
    // A step is fenced, so that its read goes out PF steps before its products: left
    // to itself the compiler waits for each read where it stands.  The first PF reads
    // are start_products', some way ahead; the last PF steps make room for the
    // caller's next ones, after(0 .. PF - 1).  (Both right before their products: 480
    // against 477 us, fp16 665 against 656; D = 64 382 against 387.)
    constexpr int STEPS = 4 * KW, PF = 3;
    i32x4 kf[PF + 1], qr[2][RX];
    auto read_key = [&](const char *kbuf, int st) {
        kf[st % (PF + 1)] = *(const i32x4 *)(kbuf + LT::key_at(16 * (st % 4) + r, st / 4, c));
    };
    auto read_query = [&](int j) {
#pragma unroll
        for (int x = 0; x < RX; ++x) {
            if constexpr (LT::Q_LDS) qr[j & 1][x] = *(const i32x4 *)(qlds + (x * KW + j) * 1024);
            else qr[j & 1][x] = qf[x][j];
        }
    };
    auto start_products = [&](const char *kbuf) {
        read_query(0);
#pragma unroll
        for (int st = 0; st < PF; ++st) read_key(kbuf, st);
    };
    auto products = [&](const char *kbuf, auto beside, auto after) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int st = 0; st < STEPS; ++st) {
            const int j = st / 4, g = st % 4;
            if (st + PF < STEPS) read_key(kbuf, st + PF);
            else after(st + PF - STEPS);
            if (g == 0 && j + 1 < KW) read_query(j + 1);
#pragma unroll
            for (int x = 0; x < RX; ++x)
                z[x][g] = MM::mul(kf[st % (PF + 1)], qr[j & 1][x], j ? z[x][g] : f32x4{0, 0, 0, 0});
            beside(st);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    if (first < last) {
        ask_keys(first);
        fetch_keys(first);
        ask_keys(first + 1);
        turn_keys(first, smem, smem + LT::P_AT);
        ask_vals(first);
        fetch_keys(first + 1);
        turn_keys(first + 1, smem + LT::KBYTES, smem + LT::P_AT + LT::PBYTES);
        fetch_vals(first);
        ask_keys(first + 2);
        ask_vals(first + 1);
        __syncthreads();
        turn_vals(smem + LT::V_AT, smem + LT::P_AT);
        start_products(smem);
        products(smem, [](int) {}, [](int) {});
    }
    __syncthreads();
    // Tile t: its scores' sums are in z; the next tile's are made beside its softmax,
    // the next values and the keys after those are turned beside its values' product.
    for (int32_t t = first; t < last; ++t) {
        const int32_t n = t - first;
        char *const kcur = smem + (n & 1) * LT::KBYTES, *const knext = smem + (~n & 1) * LT::KBYTES;
        char *const vcur = smem + LT::V_AT + (n & 1) * LT::VBYTES, *const vnext = smem + LT::V_AT + (~n & 1) * LT::VBYTES;
        auto slot = [&](int k) { return smem + LT::P_AT + ((n + k) & 3) * LT::PBYTES; };
        fetch_keys(t + 2);
        fetch_vals(t + 1);
        ask_keys(t + 3);
        ask_vals(t + 2);
        if (!busy) {
            turn_vals(vnext, slot(1));
            turn_keys(t + 2, kcur, slot(2));
            __syncthreads();
            continue;
        }
        const int32_t t0 = 64 * t;
        const char *prm = slot(0);
        const u32x4 flags = *(const u32x4 *)(prm + LT::FLAG_AT);
        const uint32_t ok_pages = __builtin_amdgcn_readfirstlane(flags.x | flags.y | flags.z | flags.w);
        const bool whole = t0 >= full_lo && t0 + 64 <= full_hi && ok_pages == 15u;
        // scores in units of log 2 above the row's reference
        float top[RX];
#pragma unroll
        for (int x = 0; x < RX; ++x) top[x] = m_run[x] == NEG ? 0.f : m_run[x];
        f32x4 sc[RX][4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const f32x4 ks = *(const f32x4 *)(prm + 4 * (16 * g + 4 * c)), km = *(const f32x4 *)(prm + 256 + 4 * (16 * g + 4 * c));
#pragma unroll
            for (int x = 0; x < RX; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sc[x][g][i] = __builtin_fmaf(ks[i], z[x][g][i], __builtin_fmaf(km[i], qsum[x], -top[x]));
        }
        uint32_t seen[RX];
#pragma unroll
        for (int x = 0; x < RX; ++x) seen[x] = 0xFFFFu;
        if (!whole) {
            asm volatile("" ::: "memory");  // keeps the comparisons in this branch
#pragma unroll
            for (int x = 0; x < RX; ++x) {
                const int32_t from = my_lo[x] - t0 - 4 * c, to = my_hi[x] - t0 - 4 * c;
                seen[x] = 0;
#pragma unroll
                for (int g = 0; g < 4; ++g)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bool ok = 16 * g + i >= from && 16 * g + i < to && ((ok_pages >> g) & 1u);
                        seen[x] |= ok ? 1u << (4 * g + i) : 0u;
                        if (!ok) sc[x][g][i] = NEG;
                    }
            }
        }
        start_products(knext);
        // The weights' reference is taken anew only when a weight passes 2^8 (WHOLE: 2^15),
        // and first of all; only then do the lanes of a row compare.
        constexpr float MOST = WHOLE ? 15.f : 8.f, BELOW = WHOLE ? 9.f : 0.f;
        bool raise = false;
#pragma unroll
        for (int x = 0; x < RX; ++x) {
            float mx = sc[x][0][0];
#pragma unroll
            for (int e = 1; e < 16; ++e) mx = fmaxf(mx, sc[x][e / 4][e % 4]);
            raise |= mx > MOST || m_run[x] == NEG;
        }
        if (__any(raise)) {
#pragma unroll
            for (int x = 0; x < RX; ++x) {
                float mx = sc[x][0][0];
#pragma unroll
                for (int e = 1; e < 16; ++e) mx = fmaxf(mx, sc[x][e / 4][e % 4]);
                const float m_new = fmaxf(m_run[x], max_over_groups(mx) + (top[x] - BELOW));
                const float m_use = m_new == NEG ? 0.f : m_new;
                const float al = m_run[x] == NEG ? 0.f : __builtin_amdgcn_exp2f(m_run[x] - m_new);
#pragma unroll
                for (int e = 0; e < 16; ++e) sc[x][e / 4][e % 4] += top[x] - m_use;
                m_run[x] = m_new;
                l_run[x].scale(al);
                if constexpr (!WHOLE) {
                    extra[x] *= al;
                    ones[x] *= al;
                }
#pragma unroll
                for (int d = 0; d < ND; ++d) acc[x][d] *= al;
            }
        }
        // this tile's weights, beside the next tile's sums
        i32x4 whi[RX][2], wlo2[RX][2];
        constexpr int QUADS = 4 * RX;   // four weights each
        constexpr int VSTEPS = 2 * ND;
        i32x4 vf[PF + 1];
        float sum[RX];
#pragma unroll
        for (int x = 0; x < RX; ++x) sum[x] = 0.f;
        auto read_val = [&](int st) { vf[st % (PF + 1)] = *(const i32x4 *)(vcur + LT::val_at(16 * (st % ND) + r, st / ND, c)); };
        __builtin_amdgcn_s_setprio(1);   // (2% faster than none, or than over both products)
        products(knext, [&](int st) {
#pragma unroll
            for (int e = 4 * QUADS * st / STEPS; e < 4 * QUADS * (st + 1) / STEPS; ++e) {
                const int x = e / 16, g = e / 4 % 4, i = e % 4;
                sc[x][g][i] = __builtin_amdgcn_exp2f(sc[x][g][i]);
                sum[x] += sc[x][g][i];
                if (i != 3) continue;
                float w[4] = {sc[x][g][0], sc[x][g][1], sc[x][g][2], sc[x][g][3]};
                if constexpr (WHOLE) {
                    whi[x][g / 2][2 * (g % 2)] = (int)pack2<_Float16>(w[0], w[1]);
                    whi[x][g / 2][2 * (g % 2) + 1] = (int)pack2<_Float16>(w[2], w[3]);
                } else {
                    const f32x4 vs = *(const f32x4 *)(prm + 512 + 4 * (16 * g + 4 * c));
                    const f32x4 vm = *(const f32x4 *)(prm + 768 + 4 * (16 * g + 4 * c));
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const bool ok = (seen[x] >> (4 * g + k)) & 1u;
                        extra[x] = __builtin_fmaf(w[k], ok ? vm[k] : 0.f, extra[x]);
                        w[k] = ok ? w[k] * vs[k] : 0.f;
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t hi2 = pack2<__bf16>(w[2 * k], w[2 * k + 1]);
                        whi[x][g / 2][2 * (g % 2) + k] = (int)hi2;
                        wlo2[x][g / 2][2 * (g % 2) + k] = (int)pack2<__bf16>(w[2 * k] - lo_f32<__bf16>(hi2),
                                                                             w[2 * k + 1] - hi_f32<__bf16>(hi2));
                    }
                }
            }
        }, read_val);
        __builtin_amdgcn_s_setprio(0);
#pragma unroll
        for (int x = 0; x < RX; ++x) l_run[x].add(sum[x]);
        // the values' product, beside the turning of what comes next
#pragma unroll
        for (int st = 0; st < VSTEPS; ++st) {
            const int d = st % ND, q = st / ND;
            if (st + PF < VSTEPS) read_val(st + PF);
            if constexpr (!WHOLE)
                if (d == 0) {
#pragma unroll
                    for (int x = 0; x < RX; ++x) {
                        ones[x] = MfmaV::mul(one, whi[x][q], ones[x]);
                        ones[x] = MfmaV::mul(one, wlo2[x][q], ones[x]);
                    }
                }
#pragma unroll
            for (int x = 0; x < RX; ++x) {
                if constexpr (WHOLE) acc[x][d] = Mfma<_Float16>::mul(vf[st % (PF + 1)], whi[x][q], acc[x][d]);
                else acc[x][d] = MfmaV::mul(vf[st % (PF + 1)], whi[x][q], acc[x][d]);
            }
            if constexpr (!WHOLE)
#pragma unroll
                for (int x = 0; x < RX; ++x) acc[x][d] = MfmaV::mul(vf[st % (PF + 1)], wlo2[x][q], acc[x][d]);
#pragma unroll
            for (int u = UNITS * st / VSTEPS; u < UNITS * (st + 1) / VSTEPS; ++u)
                turn_unit(u, t + 2, kcur, slot(2), vnext, slot(1));
            __builtin_amdgcn_sched_barrier(0);
        }
        __syncthreads();
    }

    int32_t again = 0;
    if constexpr (WHOLE) {
        bool lost = false;   // outputs (2^11 stands for the largest value) below 2^10 n 2^-25 2^11
#pragma unroll
        for (int x = 0; x < RX; ++x) {
            float most = 0.f;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) most = fmaxf(most, __builtin_fabsf(acc[x][d][i]));
            const int32_t n = min(my_hi[x], 64 * last) - max(my_lo[x], 64 * first);
            lost |= max_over_groups(most) < 0.0625f * (float)n;
        }
        lost = __any(lost);
        if (lane == 0) red[wave][0] = lost && busy;
        __syncthreads();
        uint32_t any = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) any |= red[w][0];
        again = __builtin_amdgcn_readfirstlane((int)any);
    }

#pragma unroll
    for (int x = 0; x < RX; ++x) {
        const int32_t row = w0 + 16 * x + r;
        float l = sum_over_groups(l_run[x].s);
        const float add = WHOLE ? 0.f : sum_over_groups(extra[x]);
        if (again || row >= sp.rows) continue;
        const float mul = WHOLE ? 1.f / vscale : 1.f;
        const float off = WHOLE ? 0.f : MfmaV::base * ones[x].x - add;
        const int32_t oq = row / a.group, oh = h * a.group + (row - oq * a.group);
        const int64_t hq = (int64_t)a.group * a.c.heads, grow = (sp.q0 + oq) * hq + oh;
        if (rg.ranges > 1) {
            const int64_t nrows = a.total_q * hq;
            float *po = a.part + ((int64_t)blockIdx.y * nrows + grow) * D + 4 * c;
#pragma unroll
            for (int d = 0; d < ND; ++d) *(f32x4 *)(po + 16 * d) = acc[x][d] * mul - off;
            if (c == 0) {
                float *ps = a.part + (int64_t)a.splits * nrows * D + ((int64_t)blockIdx.y * nrows + grow) * 2;
                ps[0] = m_run[x];
                ps[1] = l;
            }
            continue;
        }
        const float inv = l == 0.f ? 0.f : 1.0f / l;
        T *po = (T *)a.out + (sp.q0 + oq) * a.ldo + (int64_t)oh * D + 4 * c;
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            const f32x4 o = acc[x][d] * mul - off;
            *(u32x2 *)(po + 16 * d) = u32x2{pack2<T>(o.x * inv, o.y * inv), pack2<T>(o.z * inv, o.w * inv)};
        }
        if (a.lse && c == 0) a.lse[grow] = l == 0.f ? NEG : (m_run[x] + __builtin_log2f(l)) * 0.6931471805599453f;
    }
    return again;
}

template <class T, int D>
__global__ __launch_bounds__(512, 2) void attn_chunk_kernel(AttnArgs a)
{
    constexpr int ROWS = ChunkRows<D>::ROWS, LEVELS = ChunkTile<T, D, false>::BYTES, WHOLE = ChunkTile<T, D, true>::BYTES;
    __shared__ __attribute__((aligned(16))) char smem[LEVELS > WHOLE ? LEVELS : WHOLE];
    // The tiles that see the most keys start first: the last of a sequence, and of
    // several sequences (up to 512 tiles) this workgroup's place in the order of
    // their keys, which each finds for itself.  (3 x 2048 queries over up to 8192
    // keys 477 us; the last tile of every sequence first, and so on, 574.)
    const int32_t place = (int32_t)(blockIdx.x / (uint32_t)a.c.heads), h = (int32_t)(blockIdx.x % (uint32_t)a.c.heads);
    const int32_t tasks = a.batch * a.tiles;
    int32_t b = place % a.batch, tile = a.tiles - 1 - place / a.batch;
    if (a.batch > 1 && tasks <= 512) {
        int32_t *cost = (int32_t *)smem, *found = cost + 512;
        const int32_t mine = (int32_t)threadIdx.x;
        if (mine < tasks) {
            const Span s = lane_span_of(a, mine / a.tiles);
            const int32_t from = mine % a.tiles * ROWS;
            int32_t from_key = 0, to_key = -1;   // no rows: after all others
            if (from < s.rows) tile_keys(a, s, from, ROWS, from_key, to_key);
            cost[mine] = to_key - from_key;
        }
        __syncthreads();
        if (mine < tasks) {
            const int32_t c0 = cost[mine];
            int32_t rank = 0;
            for (int32_t k = 0; k < tasks; ++k) rank += cost[k] > c0 || (cost[k] == c0 && k < mine);
            if (rank == place) *found = mine;
        }
        __syncthreads();
        const int32_t f = __builtin_amdgcn_readfirstlane(*found);
        b = f / a.tiles;
        tile = f - b * a.tiles;
        __syncthreads();
    }
    const Span sp = span_of(a, b);
    const int32_t r0 = tile * ROWS;
    if (r0 >= sp.rows) return;

    const int32_t lo = key_lo(a, sp, r0 / a.group), hi = key_hi(a, sp, min(r0 + ROWS - 1, sp.rows - 1) / a.group);
    const Ranges rg = ranges_of<64>(a, lo, hi);
    if ((int32_t)blockIdx.y >= rg.ranges) return;
    const int32_t first = rg.b0 + (int32_t)blockIdx.y * rg.per, last = min(rg.b0 + rg.nb, first + rg.per);
    __shared__ uint32_t red[8][2];
    if constexpr (__is_same(T, __bf16)) {
        const float vscale = value_scale<T>(a, b, h, first, last, hi, red);
        if (vscale != 0.f && !chunk_rows<T, D, true>(a, smem, sp, b, h, r0, hi, rg, first, last, vscale, red)) return;
    }
    chunk_rows<T, D, false>(a, smem, sp, b, h, r0, hi, rg, first, last, 1.f, red);
}

// The partial results of attn_chunk_kernel's key ranges joined, in the ranges'
// order: a wave per row, whose lanes read whole partial rows, eight ranges at a time.
template <class T, int D>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, int32_t row_tiles)
{
    constexpr int DPL = D / 64;
    const int32_t lane = (int32_t)(threadIdx.x & 63u);
    const int32_t bh = (int32_t)(blockIdx.x / (uint32_t)row_tiles), tile = (int32_t)(blockIdx.x % (uint32_t)row_tiles);
    const int32_t b = bh / a.c.heads, h = bh - b * a.c.heads;
    const Span sp = span_of(a, b);
    const int32_t row = tile * 4 + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    if (row >= sp.rows) return;
    constexpr int ROWS = ChunkRows<D>::ROWS;
    const int32_t r0 = row / ROWS * ROWS;
    const Ranges rg = ranges_of<64>(a, key_lo(a, sp, r0 / a.group),
                                       key_hi(a, sp, min(r0 + ROWS - 1, sp.rows - 1) / a.group));
    if (rg.ranges == 1) return;
    const int32_t oq = row / a.group, oh = h * a.group + (row - oq * a.group);
    const int64_t hq = (int64_t)a.group * a.c.heads, nrows = a.total_q * hq;
    const int64_t grow = (sp.q0 + oq) * hq + oh;
    const float NEG = -__builtin_inff();
    // lane s holds range s's maximum and sum (at most 64 ranges)
    f32x2 ml = {NEG, 0.f};
    if (lane < rg.ranges)
        ml = *(const f32x2 *)(a.part + (int64_t)a.splits * nrows * D + ((int64_t)lane * nrows + grow) * 2);
    float m = ml.x;
#pragma unroll
    for (int d = 32; d; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
    const float f = ml.y == 0.f ? 0.f : __builtin_amdgcn_exp2f(ml.x - m);
    float l = f * ml.y;
#pragma unroll
    for (int d = 32; d; d >>= 1) l += __shfl_xor(l, d);
    float o[DPL];
#pragma unroll
    for (int j = 0; j < DPL; ++j) o[j] = 0.f;
    const float *po = a.part + grow * D + lane * DPL;
    for (int32_t s0 = 0; s0 < rg.ranges; s0 += 8) {
        float w[8], v[8][DPL];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int32_t s = min(s0 + k, rg.ranges - 1);
            w[k] = s0 + k < rg.ranges ? __shfl(f, s) : 0.f;
#pragma unroll
            for (int j = 0; j < DPL; ++j) v[k][j] = po[(int64_t)s * nrows * D + j];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (w[k] != 0.f)   // a range that saw nothing holds zeros; a NaN weight counts
#pragma unroll
                for (int j = 0; j < DPL; ++j) o[j] = __builtin_fmaf(w[k], v[k][j], o[j]);
    }
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    T *out = (T *)a.out + (sp.q0 + oq) * a.ldo + (int64_t)oh * D + lane * DPL;
#pragma unroll
    for (int j = 0; j < DPL; ++j) out[j] = (T)(o[j] * inv);
    if (a.lse && lane == 0) a.lse[grow] = l == 0.f ? NEG : (m + __builtin_log2f(l)) * 0.6931471805599453f;
}

template <class T, int D> static hipError_t attn_t(const AttnArgs &all, hipStream_t s)
{
    const int64_t most = LAUNCH_THREADS / 512 / ((int64_t)all.c.heads * all.tiles);   // sequences of a launch
    if (all.kernel != ATTN_FLAT && all.batch > most) {
        // (so many tiles are not cut into ranges, and need no workspace)
        for (int64_t b = 0; b < all.batch; b += most) {
            AttnArgs a = all;
            a.batch = (int32_t)(all.batch - b < most ? all.batch - b : most);
            a.table += b * a.ldt;
            a.q_off += b;
            a.lens += b;
            const hipError_t e = attn_t<T, D>(a, s);
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    }
    const AttnArgs &a = all;
    if (a.kernel == ATTN_FLAT) {
        hipLaunchKernelGGL((attn_flat_kernel<T, D>), dim3((uint32_t)a.splits), dim3(256), 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL((attn_flat_join_kernel<T, D>), dim3((uint32_t)a.splits), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    const int64_t wgs = (int64_t)a.batch * a.c.heads * a.tiles;
    constexpr int WIDE = attn_wide_waves(D);
    const dim3 grid((uint32_t)wgs, (uint32_t)a.splits);
    if (a.kernel != ATTN_CHUNK) {
        if (a.kernel == ATTN_WIDE)
            hipLaunchKernelGGL((attn_rows_kernel<T, D, WIDE>), grid, dim3(64 * WIDE), 0, s, a);
        else
            hipLaunchKernelGGL((attn_rows_kernel<T, D, 4>), grid, dim3(256), 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || a.splits == 1) return e;
        hipLaunchKernelGGL((attn_rows_join_kernel<T, D>), dim3((uint32_t)wgs), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((attn_chunk_kernel<T, D>), grid, dim3(512), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    const int64_t row_tiles = ChunkRows<D>::ROWS / 4 * (int64_t)a.tiles;
    const int64_t joins = (int64_t)a.batch * a.c.heads * row_tiles;
    hipLaunchKernelGGL((attn_join_kernel<T, D>), dim3((uint32_t)joins), dim3(256), 0, s, a, (int32_t)row_tiles);
    return hipGetLastError();
}

hipError_t launch_attn(int ftype, int D, const AttnArgs &a, hipStream_t s)
{
#define CALL(TY, DD) attn_t<TY, DD>(a, s)
    LB_KV4_BY_TYPE(CALL)
#undef CALL
}

}  // namespace lb
