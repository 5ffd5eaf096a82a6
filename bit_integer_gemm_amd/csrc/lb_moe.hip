// lb_moe.hip -- a mixture of experts with 4-bit weights, for few tokens.
//
//   l = Wr x,  p = softmax(l),  e_1 .. e_k the k largest (ties: the lowest index first),
//   q_j = scale p_{e_j}  (renorm: over the k chosen),
//   out = sum_j q_j W2_{e_j} (silu(Wg_{e_j} x) * (Wu_{e_j} x))
//
// Four launches: the router's product; gate and up rows with the activation; the down
// product; the weighted sum.  Nothing has to be sorted, counted or waited for between them:
// a workgroup finds the tokens of its expert from the logits itself (an expert's rank in a
// token's order is the number of larger logits, a few ballots), and results lie at (token,
// rank), so that every sum has a fixed order.
#include "lb_internal.hpp"
#include "lb_w4.hpp"

namespace lb {

// Logits as whole numbers in the same order, any NaN above all: a total order whatever the
// values, so that every token has exactly k chosen experts.
__device__ inline uint32_t order_of(float v)
{
    const uint32_t b = __float_as_uint(v);
    if (v != v) return 0xFFFFFFFFu;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// ---- router ----------------------------------------------------------------
// 16 experts by 16 tokens to a workgroup, a share of H to each wave.
enum { ROUTER_WAVES = 8 };
template <class T>
__global__ __launch_bounds__(64 * ROUTER_WAVES) void moe_router_kernel(MoeArgs a)
{
    typedef W4Join<1, 1, ROUTER_WAVES> Join;
    __shared__ float sums[Join::FLOATS];
    const int32_t lane = (int32_t)(threadIdx.x & 63u), q = lane >> 4, r = lane & 15;
    const int32_t wave = (int32_t)(threadIdx.x >> 6);
    const int32_t e0 = (int32_t)blockIdx.x * 16, t0 = (int32_t)blockIdx.y * 16;
    const T *wrow = (const T *)a.wr + (int64_t)min(e0 + r, a.E - 1) * a.H;
    const T *xrow = (const T *)a.x + (int64_t)min(t0 + r, a.T - 1) * a.ldx;
    const int32_t steps = a.H / 32, last = (wave + 1) * steps / ROUTER_WAVES;
    f32x4 acc[1][1] = {{f32x4{0.f, 0.f, 0.f, 0.f}}};
    for (int32_t st = wave * steps / ROUTER_WAVES; st < last; st += 4) {
        u32x4 x[4], w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = w[i] = u32x4{0u, 0u, 0u, 0u};
            if (st + i < last) {
                x[i] = *(const u32x4 *)(xrow + 32 * (st + i) + 8 * q);
                w[i] = *(const u32x4 *)(wrow + 32 * (st + i) + 8 * q);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[0][0] = mfma16<T>(x[i], w[i], acc[0][0]);
    }
    Join::put(sums, wave, acc);
    __syncthreads();
    for (int32_t i = (int32_t)threadIdx.x; i < 256; i += 64 * ROUTER_WAVES) {
        const int32_t t = t0 + i / 16, e = e0 + i % 16;
        if (t < a.T && e < a.E) a.logits[t * a.E + e] = Join::sum(sums, i / 16, i % 16);
    }
}

// ---- who goes where --------------------------------------------------------
// The expert of a workgroup and its tokens.  Slots are experts where tokens are many, and
// (token, rank) pairs where those are fewer; of pairs that name the same expert the first
// one's workgroups work for all its tokens, the others end.
struct MoeList {
    int32_t rank[MOE_TOKENS];   // the expert's rank in each token's order, if below k, else -1
    int32_t row[MOE_TOKENS];    // token * k + rank of each of its tokens
    int32_t expert, count, first;
};

template <int NW>
__device__ inline bool moe_list(const MoeArgs &a, int32_t slot, bool by_pair, MoeList &l)
{
    const int32_t tid = (int32_t)threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (by_pair) {
        const int32_t t = slot / a.top_k, j = slot % a.top_k;
        const float *row = a.logits + t * a.E;
        for (int32_t e = tid; e < a.E; e += 64 * NW) {
            const uint32_t mine = order_of(row[e]);
            int32_t above = 0;
            for (int32_t f = 0; f < a.E; ++f) {
                const uint32_t o = order_of(row[f]);
                above += o > mine || (o == mine && f < e);
            }
            if (above == j) {
                l.expert = e;
                l.first = t;
            }
        }
    } else if (tid == 0) {
        l.expert = slot;
        l.first = 0;
    }
    __syncthreads();
    const int32_t e = l.expert;
    for (int32_t t = wave; t < a.T; t += NW) {
        const float *row = a.logits + t * a.E;
        const uint32_t mine = order_of(row[e]);
        int32_t above = 0;
        for (int32_t f0 = 0; f0 < a.E; f0 += 64) {
            const int32_t f = f0 + lane;
            const uint32_t o = f < a.E ? order_of(row[f]) : 0u;
            above += __popcll(__ballot(f < a.E && (o > mine || (o == mine && f < e))));
        }
        if (lane == 0) l.rank[t] = above < a.top_k ? above : -1;
    }
    __syncthreads();
    if (wave == 0) {
        const int32_t rank = lane < a.T ? l.rank[lane] : -1;
        const uint64_t in = __ballot(rank >= 0);
        if (rank >= 0) l.row[__popcll(in & ((1ull << lane) - 1))] = lane * a.top_k + rank;
        if (lane == 0) l.count = (by_pair && (in & ((1ull << l.first) - 1))) ? 0 : __popcll(in);
    }
    __syncthreads();
    return l.count > (int32_t)blockIdx.z * 16;
}

// ---- gate and up, activation -----------------------------------------------
enum { MOE_WAVES = 8 };
template <class T, int G>
__global__ __launch_bounds__(64 * MOE_WAVES) void moe_up_kernel(MoeArgs a, bool by_pair)
{
    typedef W4Join<1, 2, MOE_WAVES> Join;
    __shared__ float sums[Join::FLOATS];
    __shared__ MoeList list;
    if (!moe_list<MOE_WAVES>(a, (int32_t)blockIdx.y, by_pair, list)) return;
    const int32_t lane = (int32_t)(threadIdx.x & 63u);
    const int32_t wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int32_t i0 = (int32_t)blockIdx.x * 16, at = (int32_t)blockIdx.z * 16, rows = min(16, list.count - at);
    const int64_t n0 = (int64_t)__builtin_amdgcn_readfirstlane(list.expert) * 2 * a.I + i0;
    const T *xrow[1] = {(const T *)a.x + (int64_t)(list.row[at + min(lane & 15, rows - 1)] / a.top_k) * a.ldx};
    const int32_t lines = (a.H + 255) / 256;
    const int64_t left = a.I + 16;   // rows from the first gate row of the tile to the last up row
    f32x4 acc[1][2] = {{f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}}};
    w4_product<T, T, 1, 2, G>(a.w1 + n0 * (a.H / 2), (uint64_t)left * (uint32_t)(a.H / 2), (const uint32_t *)a.p1 + n0 * (a.H / G),
                              (uint64_t)left * (uint32_t)(a.H / G) * 4u, a.H, a.I, wave * lines / MOE_WAVES,
                              (wave + 1) * lines / MOE_WAVES, xrow, 0, acc);
    Join::put(sums, wave, acc);
    __syncthreads();
    __bf16 *const hi = (__bf16 *)a.h, *const lo = hi + (int64_t)a.T * a.top_k * a.I;
    for (int32_t i = (int32_t)threadIdx.x; i < 16 * rows; i += 64 * MOE_WAVES) {
        const int32_t m = i / 16, n = i % 16;
        const float g = Join::sum(sums, m, n), u = Join::sum(sums, m, 16 + n);
        const float h = g / (1.0f + __expf(-g)) * u;
        const int64_t o = (int64_t)list.row[at + m] * a.I + i0 + n;
        hi[o] = (__bf16)h;
        lo[o] = (__bf16)(h - (float)hi[o]);
    }
}

// ---- down ------------------------------------------------------------------
template <class T, int G>
__global__ __launch_bounds__(64 * MOE_WAVES) void moe_down_kernel(MoeArgs a, bool by_pair)
{
    typedef W4Join<1, 2, MOE_WAVES> Join;
    __shared__ float sums[Join::FLOATS];
    __shared__ MoeList list;
    if (!moe_list<MOE_WAVES>(a, (int32_t)blockIdx.y, by_pair, list)) return;
    const int32_t lane = (int32_t)(threadIdx.x & 63u);
    const int32_t wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int32_t c0 = (int32_t)blockIdx.x * 32, at = (int32_t)blockIdx.z * 16, rows = min(16, list.count - at);
    const int64_t n0 = (int64_t)__builtin_amdgcn_readfirstlane(list.expert) * a.H + c0;
    const __bf16 *xrow[1] = {(const __bf16 *)a.h + (int64_t)list.row[at + min(lane & 15, rows - 1)] * a.I};
    const int32_t lines = (a.I + 255) / 256;
    const int32_t left = min(32, a.H - c0);
    f32x4 acc[1][2] = {{f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}}};
    w4_product<__bf16, T, 1, 2, G, 2>(a.w2 + n0 * (a.I / 2), (uint64_t)left * (uint32_t)(a.I / 2),
                                      (const uint32_t *)a.p2 + n0 * (a.I / G), (uint64_t)left * (uint32_t)(a.I / G) * 4u, a.I,
                                      16, wave * lines / MOE_WAVES, (wave + 1) * lines / MOE_WAVES, xrow,
                                      (int64_t)a.T * a.top_k * a.I, acc);
    Join::put(sums, wave, acc);
    __syncthreads();
    for (int32_t i = (int32_t)threadIdx.x; i < 32 * rows; i += 64 * MOE_WAVES) {
        const int32_t m = i / 32, n = i % 32;
        if (c0 + n < a.H) a.y[(int64_t)list.row[at + m] * a.H + c0 + n] = Join::sum(sums, m, n);
    }
}

// ---- weighted sum ----------------------------------------------------------
enum { COMBINE_THREADS = 256, MOE_TOP_MAX = 64 };
template <class T>
__global__ __launch_bounds__(COMBINE_THREADS) void moe_combine_kernel(MoeArgs a)
{
    __shared__ float part[COMBINE_THREADS / 64], chosen[MOE_TOP_MAX];
    __shared__ float largest;
    const int32_t t = (int32_t)blockIdx.y, tid = (int32_t)threadIdx.x;
    const float *row = a.logits + t * a.E;
    for (int32_t e = tid; e < a.E; e += COMBINE_THREADS) {
        const uint32_t mine = order_of(row[e]);
        int32_t above = 0;
        for (int32_t f = 0; f < a.E; ++f) {
            const uint32_t o = order_of(row[f]);
            above += o > mine || (o == mine && f < e);
        }
        if (above < a.top_k) {
            chosen[above] = row[e];
            if (a.ids && blockIdx.x == 0) a.ids[t * a.top_k + above] = e;
        }
        if (above == 0) largest = row[e];
    }
    __syncthreads();
    float total = 0.f;
    if (a.renorm) {
        for (int32_t j = 0; j < a.top_k; ++j) total += expf(chosen[j] - largest);
    } else {
        for (int32_t e = tid; e < a.E; e += COMBINE_THREADS) total += expf(row[e] - largest);
#pragma unroll
        for (int d = 32; d; d >>= 1) total += __shfl_xor(total, d);
        if (tid % 64 == 0) part[tid / 64] = total;
        __syncthreads();
        total = 0.f;
#pragma unroll
        for (int w = 0; w < COMBINE_THREADS / 64; ++w) total += part[w];
    }
    if (a.weights && blockIdx.x == 0 && tid < a.top_k) a.weights[t * a.top_k + tid] = a.scale * (expf(chosen[tid] - largest) / total);
    const int32_t c = ((int32_t)blockIdx.x * COMBINE_THREADS + tid) * 4;
    if (c >= a.H) return;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    for (int32_t j = 0; j < a.top_k; ++j) {
        const float p = a.scale * (expf(chosen[j] - largest) / total);
        const f32x4 y = *(const f32x4 *)(a.y + (int64_t)(t * a.top_k + j) * a.H + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += p * y[i];
    }
    *(u32x2 *)((T *)a.out + (int64_t)t * a.H + c) = u32x2{pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3])};
}

template <class T, int G> static hipError_t moe_t(const MoeArgs &a, hipStream_t s)
{
    const bool by_pair = a.T * a.top_k < a.E;
    const uint32_t slots = (uint32_t)(by_pair ? a.T * a.top_k : a.E), passes = (uint32_t)(a.T + 15) / 16;
    hipLaunchKernelGGL((moe_router_kernel<T>), dim3((uint32_t)(a.E + 15) / 16, passes), dim3(64 * ROUTER_WAVES), 0, s, a);
    hipLaunchKernelGGL((moe_up_kernel<T, G>), dim3((uint32_t)a.I / 16, slots, passes), dim3(64 * MOE_WAVES), 0, s, a, by_pair);
    hipLaunchKernelGGL((moe_down_kernel<T, G>), dim3((uint32_t)(a.H + 31) / 32, slots, passes), dim3(64 * MOE_WAVES), 0, s, a, by_pair);
    hipLaunchKernelGGL((moe_combine_kernel<T>), dim3((uint32_t)(a.H + 4 * COMBINE_THREADS - 1) / (4 * COMBINE_THREADS), (uint32_t)a.T),
                       dim3(COMBINE_THREADS), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_moe_w4(int ftype, int group, const MoeArgs &a, hipStream_t s)
{
    if (ftype == LB_BF16)
        return group == 32 ? moe_t<__bf16, 32>(a, s) : group == 64 ? moe_t<__bf16, 64>(a, s) : moe_t<__bf16, 128>(a, s);
    if (ftype == LB_F16)
        return group == 32 ? moe_t<_Float16, 32>(a, s) : group == 64 ? moe_t<_Float16, 64>(a, s) : moe_t<_Float16, 128>(a, s);
    return hipErrorInvalidValue;
}

}  // namespace lb
