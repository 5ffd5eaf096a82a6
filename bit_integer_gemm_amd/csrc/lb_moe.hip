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
// rank), so that every sum has a fixed order.  One token needs no last launch, few experts no
// first one.
// Between the products h is fp32, in the down product's nibble order, and the down product's outputs
// are fp32.
//
// Bound by the chosen experts' weights, read once (2 of 8 of 4096 x 11008: 98.6 MB in 28 us and
// 48.8 in 16.6; about 118 of 128 of 2048 x 1024, met by 48 tokens: 262 MB in 56 us, 4.6 TB/s, and 133
// in 37), and by what each launch takes before its first weights: 9 us for the first product of 5
// tokens, 6 for the second.  5 tokens of 6 of 64 experts of 2048 x 1376, G = 32: 4.9 + 25.9 + 17.1
// + 5.0 us, where the bytes would take 26.
#include <algorithm>

#include "lb_layer.hpp"
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
// 16 experts by 16 tokens, a share of H to each of NW waves, whose loads (of up to 256 numbers
// of a row) are all under way at once.  sums: LDS for NW tiles; the logits of thread i < 256,
// token t0 + i / 16 and expert e0 + i % 16, are returned to it.
enum { ROUTER_WAVES = 16, ROUTER_STEPS = 8, ROUTER_TILE = 16 * W4_SLOT_LD };
template <class T, int NW> __device__ inline float router_tile(const MoeArgs &a, int32_t e0, int32_t t0, float *sums)
{
    const int32_t lane = (int32_t)(threadIdx.x & 63u), q = lane >> 4, r = lane & 15;
    const int32_t wave = (int32_t)(threadIdx.x >> 6);
    const T *wrow = (const T *)a.wr + (int64_t)min(e0 + r, a.E - 1) * a.H;
    const T *xrow = (const T *)a.x + (int64_t)min(t0 + 4 * (r & 3) + (r >> 2), a.T - 1) * a.ldx;   // (as w4_put has them)
    const int32_t steps = a.H / 32, last = (wave + 1) * steps / NW;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int32_t st = wave * steps / NW; st < last; st += ROUTER_STEPS) {
        u32x4 x[ROUTER_STEPS], w[ROUTER_STEPS];
#pragma unroll
        for (int i = 0; i < ROUTER_STEPS; ++i) {
            x[i] = w[i] = u32x4{0u, 0u, 0u, 0u};
            if (st + i < last) {
                x[i] = *(const u32x4 *)(xrow + 32 * (st + i) + 8 * q);
                w[i] = *(const u32x4 *)(wrow + 32 * (st + i) + 8 * q);
            }
        }
#pragma unroll
        for (int i = 0; i < ROUTER_STEPS; ++i) acc = mfma16<T>(x[i], w[i], acc);
    }
    w4_put(sums + wave * ROUTER_TILE, 16, acc, false);
    __syncthreads();
    float v = 0.f;
    if (threadIdx.x < 256)
#pragma unroll
        for (int w = 0; w < NW; ++w) v += sums[w * ROUTER_TILE + (int32_t)threadIdx.x / 16 * W4_SLOT_LD + (int32_t)threadIdx.x % 16];
    return v;
}
template <class T>
__global__ __launch_bounds__(64 * ROUTER_WAVES) void moe_router_kernel(MoeArgs a)
{
    __shared__ float sums[ROUTER_WAVES * ROUTER_TILE];
    const int32_t e0 = (int32_t)blockIdx.x * 16, t0 = (int32_t)blockIdx.y * 16;
    const float v = router_tile<T, ROUTER_WAVES>(a, e0, t0, sums);
    const int32_t t = t0 + (int32_t)threadIdx.x / 16, e = e0 + (int32_t)threadIdx.x % 16;
    if (threadIdx.x < 256 && t < a.T && e < a.E) a.logits[t * a.E + e] = v;
}

// ---- who goes where --------------------------------------------------------
// Workgroups are shared out evenly among the experts that have tokens: each workgroup finds
// these from the logits, or, where there are five pairs of a token and an expert for every four
// experts, shares them out among all.  Both products of 13 tokens of 6 of 64 experts take 98 us with the
// search and 110 without, 18 of 8 of 128 92 and 95, 60 of 1 of 60 100 and 118; 20 of 8 of 128 102 and 96,
// 47 of them 127 and 113, 16 of 6 of 64 111 and 109, 12 of 2 of 16 47 and 45 (whole calls).
enum { EXPERTS_MAX = LB_MOE_EXPERTS_MAX, MOE_TOP_MAX = LB_MOE_TOP_MAX };
static_assert(EXPERTS_MAX <= 16 * 64 && EXPERTS_MAX % 32 == 0, "the logits of a token in 16 registers of a wave, a bit each");
static_assert(MOE_TOP_MAX <= 64 && MOE_TOKENS <= 64, "a lane to each of a token's experts, to each token");
enum { MOE_LIST = 2 + MOE_TOKENS };   // in the workspace: count, expert, rows (one token: count, expert, row, logit)
struct MoeList {
    int32_t rank[MOE_TOKENS];   // the expert's rank in each token's order, if below k, else -1
    int32_t row[MOE_TOKENS];    // token * k + rank of each of its tokens
    uint32_t any[EXPERTS_MAX / 32];   // experts that have tokens, a bit each
    float logits[256];          // where a workgroup forms them itself: 16 experts, 16 tokens
};

// Number j (from 0) in a token's order of its logits, by every wave for itself: lane l holds
// o[i], the order of logit 64 i + l; the value bit by bit from the top, by counting those not
// below a candidate.  above: how many are larger.
//   Returns [value, upper) that holds it, and no others but equal ones.  WHOLE: all of the first
//   j + 1 are in it or above, and no others.
template <int NC, bool WHOLE> __device__ inline uint32_t nth_value(const uint32_t (&o)[NC], int32_t j, int32_t &above, uint32_t &upper)
{
    uint32_t value = 0;
    int32_t from = INT32_MAX;   // how many are not below value
    above = 0;
    upper = 0xFFFFFFFFu;        // (with above 0: all ones, which a NaN has, belongs to it)
#pragma unroll 1
    for (uint32_t bit = 0x80000000u; bit; bit >>= 1) {
        int32_t n = 0;
#pragma unroll
        for (int i = 0; i < NC; ++i) n += __popcll(__ballot(o[i] >= (value | bit)));
        if (n > j) {
            value |= bit;
            from = n;
        } else {
            above = n;
            upper = value | bit;
        }
        if (WHOLE ? from == j + 1 : from - above == 1) break;
    }
    return value;
}
template <int NC> __device__ inline void orders_of(const float *row, int32_t E, uint32_t (&o)[NC])
{
    const int32_t lane = (int32_t)threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const float v = row[min(64 * i + lane, E - 1)];
        o[i] = 64 * i + lane < E ? order_of(v) : 0u;   // (every logit's is above 0)
    }
}
// Expert number j: of equal logits the lowest index first.
template <int NC> __device__ inline int32_t nth_expert(const float *row, int32_t E, int32_t j)
{
    uint32_t o[NC];
    orders_of<NC>(row, E, o);
    int32_t above, e = 0;
    uint32_t upper;
    const uint32_t value = nth_value<NC, false>(o, j, above, upper);
    int32_t left = j - above;   // how many equal ones come before
    bool found = false;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        uint64_t same = __ballot(o[i] >= value && (o[i] < upper || above == 0));
        const int32_t n = __popcll(same);
        if (!found && left < n) {
            for (; left > 0; --left) same &= same - 1;
            e = 64 * i + __builtin_ctzll(same);
            found = true;
        }
        left -= n;
    }
    return __builtin_amdgcn_readfirstlane(e);
}
// The first k experts' bits.
template <int NC> __device__ inline void mark_experts(const uint32_t (&o)[NC], int32_t k, uint32_t *any)
{
    int32_t above;
    uint32_t upper;
    const uint32_t value = nth_value<NC, true>(o, k - 1, above, upper);
    int32_t left = k - above;   // of those in [value, upper), all or equal ones
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        uint64_t in = __ballot(o[i] >= upper && above > 0), same = __ballot(o[i] >= value) & ~in;
        for (; left > 0 && same; --left) {
            in |= same & -same;
            same &= same - 1;
        }
        if (((int32_t)threadIdx.x & 63) == 0 && in) {
            atomicOr(any + 2 * i, (uint32_t)in);
            atomicOr(any + 2 * i + 1, (uint32_t)(in >> 32));
        }
    }
}

// What a workgroup does: a part of an expert's tiles.
struct MoeGrid {
    bool active;     // experts that have tokens share the workgroups, else all experts
    bool one;        // all of K in a chunk
    int32_t rows;    // tokens at a time, at most 16
    int32_t tiles, chunk;
    uint32_t x_bytes;
};
struct MoePlace {
    int32_t slot, part, first, have;   // the expert's number; its tiles
};
// `experts` of them.  False: nothing to do.
__device__ inline bool moe_place(const MoeGrid &g, int32_t experts, MoePlace &p)
{
    const int32_t wgs = max((int32_t)gridDim.x / experts, 1), per = (g.tiles + wgs - 1) / wgs;
    p.slot = (int32_t)blockIdx.x / wgs;
    p.part = (int32_t)blockIdx.x - p.slot * wgs;
    p.first = p.part * per;
    p.have = p.slot < experts ? min(per, g.tiles - p.first) : 0;
    return p.have > 0;
}

// Ranks of an expert in the orders of the tokens of this wave (every eighth).  ask() loads the first
// 128 logits of each, ahead of the search for the expert.
constexpr int MOE_EACH = MOE_TOKENS / W4_WAVES;
struct MoeRanks {
    enum : int { AHEAD = 2 };
    float v[AHEAD][MOE_EACH];
    int32_t above[MOE_EACH];
    __device__ inline void load(const MoeArgs &a, const float *logits, int32_t f0)
    {
        const int32_t lane = (int32_t)threadIdx.x & 63, wave = (int32_t)threadIdx.x >> 6;
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
#pragma unroll
            for (int i = 0; i < MOE_EACH; ++i)
                v[u][i] = logits[min(wave + W4_WAVES * i, a.T - 1) * a.E + min(f0 + 64 * u + lane, a.E - 1)];
    }
    __device__ inline void ask(const MoeArgs &a, const float *logits) { load(a, logits, 0); }
    __device__ inline void count(const MoeArgs &a, const float *logits, int32_t e)
    {
        const int32_t lane = (int32_t)threadIdx.x & 63, wave = (int32_t)threadIdx.x >> 6;
        float own[MOE_EACH];
#pragma unroll
        for (int i = 0; i < MOE_EACH; ++i) {
            own[i] = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(e < 64 ? v[0][i] : v[1][i]), e & 63));
            above[i] = 0;
        }
        if (e >= 64 * AHEAD)
#pragma unroll
            for (int i = 0; i < MOE_EACH; ++i) own[i] = logits[min(wave + W4_WAVES * i, a.T - 1) * a.E + e];
        for (int32_t f0 = 0;;) {
#pragma unroll
            for (int i = 0; i < MOE_EACH; ++i) {
                if (__builtin_amdgcn_readfirstlane(wave) + W4_WAVES * i >= a.T) break;
                const uint32_t mine = order_of(own[i]);
#pragma unroll
                for (int u = 0; u < AHEAD; ++u) {
                    if (f0 + 64 * u >= a.E) break;
                    const int32_t f = f0 + 64 * u + lane;
                    const uint32_t o = order_of(v[u][i]);
                    above[i] += __popcll(__ballot(f < a.E && (o > mine || (o == mine && f < e))));
                }
            }
            f0 += 64 * AHEAD;
            if (f0 >= a.E) break;
            load(a, logits, f0);
        }
    }
    // The list of the expert's tokens.  Returns how many.  (Every wave writes the same list and reads
    // what it wrote.)
    __device__ inline int32_t list(const MoeArgs &a, MoeList &l) const
    {
        const int32_t lane = (int32_t)threadIdx.x & 63, wave = (int32_t)threadIdx.x >> 6;
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < MOE_EACH; ++i) l.rank[wave + W4_WAVES * i] = wave + W4_WAVES * i < a.T && above[i] < a.top_k ? above[i] : -1;
        __syncthreads();
        const int32_t rank = l.rank[lane];
        const uint64_t in = __ballot(rank >= 0);
        if (rank >= 0) l.row[__popcll(in & ((1ull << lane) - 1))] = lane * a.top_k + rank;
        return __popcll(in);
    }
};

// Place, expert, list of tokens and their number; 0: nothing to do.  start(): called between, when
// place and expert are known.
template <class Start>
__device__ inline int32_t moe_route(const MoeArgs &a, const MoeGrid &g, const float *logits, MoePlace &p, int32_t &expert,
                                    MoeList &l, Start &&start)
{
    const int32_t tid = (int32_t)threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    if (a.T == 1) {   // slot j is expert number j
        if (!moe_place(g, a.top_k, p)) return 0;
        expert = a.E <= 64 ? nth_expert<1>(logits, a.E, p.slot) : a.E <= 128 ? nth_expert<2>(logits, a.E, p.slot)
               : a.E <= 256 ? nth_expert<4>(logits, a.E, p.slot) : nth_expert<16>(logits, a.E, p.slot);
        start();
        if (tid == 0) l.row[0] = p.slot;
        __syncthreads();
        return 1;
    }
    MoeRanks ranks;
    ranks.ask(a, logits);
    int32_t experts = a.E;
    if (g.active) {
        if (tid < EXPERTS_MAX / 32) l.any[tid] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MOE_EACH; ++i) {
            const int32_t t = wave + W4_WAVES * i;
            if (t >= a.T) break;
            if (a.E <= 64) {
                uint32_t o[1] = {(tid & 63) < a.E ? order_of(ranks.v[0][i]) : 0u};
                mark_experts<1>(o, a.top_k, l.any);
            } else if (a.E <= 64 * MoeRanks::AHEAD) {
                uint32_t o[MoeRanks::AHEAD];
#pragma unroll
                for (int u = 0; u < MoeRanks::AHEAD; ++u) o[u] = 64 * u + (tid & 63) < a.E ? order_of(ranks.v[u][i]) : 0u;
                mark_experts<MoeRanks::AHEAD>(o, a.top_k, l.any);
            } else {
                uint32_t o[EXPERTS_MAX / 64];
                orders_of<EXPERTS_MAX / 64>(logits + t * a.E, a.E, o);
                mark_experts<EXPERTS_MAX / 64>(o, a.top_k, l.any);
            }
        }
        __syncthreads();
        const uint32_t bits = l.any[tid % (EXPERTS_MAX / 32)];
        const int32_t words = (a.E + 31) / 32;
        experts = 0;
        for (int32_t w = 0; w < words; ++w) experts += __builtin_popcount((uint32_t)__builtin_amdgcn_readlane((int)bits, w));
        if (blockIdx.x == 0 && tid == 0) *a.found = experts;
        if (!moe_place(g, experts, p)) return 0;
        int32_t left = p.slot;
        for (int32_t w = 0; w < words; ++w) {
            uint32_t here = (uint32_t)__builtin_amdgcn_readlane((int)bits, w);
            const int32_t n = __builtin_popcount(here);
            if (left < n) {
                for (; left > 0; --left) here &= here - 1;
                expert = 32 * w + __builtin_ctz(here);
                break;
            }
            left -= n;
        }
    } else {
        if (!moe_place(g, experts, p)) return 0;
        expert = p.slot;
    }
    ranks.count(a, logits, expert);
    start();
    return ranks.list(a, l);
}

// ---- gate and up, activation -----------------------------------------------
// A workgroup: an expert, some blocks of 16 columns (a tile of gate rows and one of up rows
// each), g.rows of its tokens at a time.
// ONE: all of a row of x is in LDS at once.  x is asked for when the tokens are known: all tokens'
// rows ahead of that take 1.5 us more of 26 (5 tokens of 6 of 64: more rows to put in order and to
// scale).
// ROUTE (one router tile, at most 16 tokens and experts, of at most 128 KB): every workgroup forms
// the logits for itself, which takes a us where a launch for them takes five (one token of 2 of 8:
// 46 us in all, 50 with the launch).  Beyond that each workgroup would read more than its share
// of weights.
template <class T, int G, bool ONE, bool ROUTE>
__global__ __launch_bounds__(64 * W4_WAVES) void moe_up_kernel(MoeArgs a, MoeGrid g)
{
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    __shared__ MoeList list;
    const int32_t wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    MoePlace p = {};
    auto put = [&](int32_t m, int32_t c, float gate, float up) {
        // in the order in which the down product's nibbles come
        a.h[(int64_t)list.row[m] * a.I + p.first * 16 + (c & ~7) + 2 * (c & 3) + (c >> 2 & 1)] = gate / (1.0f + expf(-gate)) * up;
    };
    int32_t expert = 0;
    auto tile_at = [&](int32_t t) { return W4Tile{((int64_t)expert * 2 + t % 2) * a.I + (p.first + t / 2) * 16, 16}; };
    W4Flow<T, T, G, 1, decltype(tile_at)> flow(smem, g.x_bytes, a.w1, (const uint32_t *)a.p1, a.H, g.chunk, tile_at);
    const i32x4 rx = make_rsrc(a.x, 0xFFFFFFF0u);
    const float *logits = a.logits;
    if constexpr (ROUTE) {
        const float v = router_tile<T, W4_WAVES>(a, 0, 0, (float *)(smem + g.x_bytes));   // (where the rings will be)
        const int32_t t = (int32_t)threadIdx.x / 16, e = (int32_t)threadIdx.x % 16;
        if (threadIdx.x < 256 && t < a.T && e < a.E) {
            list.logits[t * a.E + e] = v;
            if (blockIdx.x + blockIdx.y == 0) a.logits[t * a.E + e] = v;
        }
        __syncthreads();
        logits = list.logits;
    }
    // the first weights are on their way while the tokens are gathered
    const int32_t count = __builtin_amdgcn_readfirstlane(moe_route(a, g, logits, p, expert, list, [&] {
        expert = __builtin_amdgcn_readfirstlane(expert);
        flow.start(2 * p.have);
    }));
    if (p.part == 0 && p.have > 0) {   // for the down product
        int32_t *const l = a.lists + p.slot * MOE_LIST;
        if (a.T == 1 && threadIdx.x == 66) l[3] = (int32_t)__float_as_uint(logits[expert]);
        if (threadIdx.x < (uint32_t)count) l[2 + threadIdx.x] = list.row[threadIdx.x];
        if (threadIdx.x == 64) l[0] = count;
        if (threadIdx.x == 65) l[1] = expert;
    }
    if (count == 0) flow.finish();
    for (int32_t at = 0; at < count; at += g.rows) {
        const int32_t rows = min(g.rows, count - at);
        const W4Sums<ONE> sums(smem + g.x_bytes + W4Lds<G>::RINGS, p.have, 2, rows);
        f32x4 gate = {0.f, 0.f, 0.f, 0.f};
        auto x_at = [&](int32_t i) { return (uint32_t)(list.row[at + i] / a.top_k) * (uint32_t)a.ldx * 2u; };
        auto done = [&](int32_t t, const f32x4 &acc, bool more) {
            if (!sums.whole(wave, t / 2)) w4_put(sums.at(wave, t / 2, t % 2), rows, acc, more);
            else if (t % 2 == 0) gate = acc;
            else w4_rows(rows, [&](int32_t i, int32_t m, int32_t c) { put(at + m, t / 2 * 16 + c, gate[i], acc[i]); });
        };
        if (at == 0) {
            flow.template run<true>(2 * p.have, rows, rx, x_at, done);
        } else {
            __syncthreads();
            flow.template run<false>(2 * p.have, rows, rx, x_at, done);
        }
        __syncthreads();
        sums.each([&](int32_t u, int32_t m, int32_t c) { put(at + m, u * 16 + c, sums.sum(u, 0, m, c), sums.sum(u, 1, m, c)); });
    }
}

// ---- down ------------------------------------------------------------------
template <class T, int G, bool ONE>
__global__ __launch_bounds__(64 * W4_WAVES) void moe_down_kernel(MoeArgs a, MoeGrid g)
{
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    __shared__ MoeList list;
    const int32_t lane = (int32_t)(threadIdx.x & 63u), wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    MoePlace p = {};
    if (!moe_place(g, a.T == 1 ? a.top_k : g.active ? *a.found : a.E, p)) return;
    const int32_t *const l = a.lists + p.slot * MOE_LIST;
    const int32_t count = l[0], expert = l[1];
    if (count == 0) return;
    auto tile_at = [&](int32_t t) { return W4Tile{(int64_t)expert * a.H + (p.first + t) * 16, 16}; };
    W4Flow<_Float16, T, G, 2, decltype(tile_at)> flow(smem, g.x_bytes, a.w2, (const uint32_t *)a.p2, a.I, g.chunk, tile_at);
    const i32x4 rx = make_rsrc(a.h, 0xFFFFFFF0u);
    const int32_t mine_row = l[2 + min(lane, count - 1)];
    list.row[lane] = mine_row;   // (every wave writes the same, and reads what it wrote)
    flow.start(p.have);
    for (int32_t at = 0; at < count; at += g.rows) {
        const int32_t rows = min(g.rows, count - at);
        const W4Sums<ONE> sums(smem + g.x_bytes + W4Lds<G>::RINGS, p.have, 1, rows);
        auto put = [&](int32_t t, int32_t m, int32_t c, float v) { a.y[(int64_t)list.row[at + m] * a.H + (p.first + t) * 16 + c] = v; };
        auto x_at = [&](int32_t i) { return (uint32_t)list.row[at + i] * (uint32_t)a.I * 4u; };
        auto done = [&](int32_t t, const f32x4 &acc, bool more) {
            if (!sums.whole(wave, t)) return w4_put(sums.at(wave, t, 0), rows, acc, more);
            w4_rows(rows, [&](int32_t i, int32_t m, int32_t c) { put(t, m, c, acc[i]); });
        };
        if (at == 0) {
            flow.template run<true>(p.have, rows, rx, x_at, done);
        } else {
            __syncthreads();
            flow.template run<false>(p.have, rows, rx, x_at, done);
        }
        __syncthreads();
        sums.each([&](int32_t t, int32_t m, int32_t c) { put(t, m, c, sums.sum(t, 0, m, c)); });
    }
}

// One token: a workgroup's columns get all of its experts' sums, weighted here (tile k c + j: column
// tile c of expert j), and no launch follows.  16.6 us for 2 experts of 4096 x 11008 (15 before what
// passes between the products kept fp32's digits, where a product and the weighted sum took 15.4 + 4.6).
template <class T, int G>
__global__ __launch_bounds__(64 * W4_WAVES) void moe_down_token_kernel(MoeArgs a, int32_t per, uint32_t x_bytes)
{
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    const int32_t lane = (int32_t)(threadIdx.x & 63u), k = a.top_k;
    const int32_t wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int32_t t0 = (int32_t)blockIdx.x * per, have = min(per, a.H / 16 - t0);
    const W4Sums<false> sums(smem + x_bytes + W4Lds<G>::RINGS, k * have, 1, 1);
    int32_t expert = 0, row = 0;   // of slot `lane`
    auto tile_at = [&](int32_t t) {
        const int32_t j = t % k;
        return W4Tile{(int64_t)__builtin_amdgcn_readlane(expert, j) * a.H + (t0 + t / k) * 16, 16};
    };
    W4Flow<_Float16, T, G, 2, decltype(tile_at)> flow(smem, x_bytes, a.w2, (const uint32_t *)a.p2, a.I, (a.I + 255) / 256, tile_at);
    const i32x4 rx = make_rsrc(a.h, 0xFFFFFFF0u);
    auto x_at = [&](int32_t i) { return (uint32_t)i * (uint32_t)a.I * 4u; };
    const int32_t *const l = a.lists + min(lane, k - 1) * MOE_LIST;
    expert = l[1];
    row = l[2];
    const float logit = __uint_as_float((uint32_t)l[3]);
    // the sum of all experts' exponentials, or of the chosen ones'; any NaN or infinity spoils it
    const float other = !a.renorm ? a.logits[min(lane, a.E - 1)] : 0.f;
    flow.start(k * have);
    float largest = logit;
#pragma unroll
    for (int d = 32; d; d >>= 1) largest = fmaxf(largest, __shfl_xor(largest, d));
    const float own = expf(logit - largest);
    float total = lane < k ? own : 0.f;
    if (!a.renorm) {
        total = lane < a.E ? expf(other - largest) : 0.f;
        for (int32_t e = lane + 64; e < a.E; e += 64) total += expf(a.logits[e] - largest);
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) total += __shfl_xor(total, d);
    const float weight = a.scale * (own / total);
    if (blockIdx.x == 0 && wave == 0 && lane < k) {
        if (a.ids) a.ids[row] = expert;
        if (a.weights) a.weights[row] = weight;
    }
    flow.template run_n<1, true, true>(
        k * have, k, rx, x_at,
        [&](int32_t t, const f32x4 &acc, bool) {
            const float q = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(weight), t % k));
            w4_put(sums.at(wave, t, 0), 1, acc * q, false);
        },
        [&](int32_t t) { return __builtin_amdgcn_readlane(row, t % k); });
    __syncthreads();
    for (int32_t c = (int32_t)threadIdx.x; c < have * 16; c += 64 * W4_WAVES) {
        float v = 0.f;
        for (int32_t j = 0; j < k; ++j) v += sums.sum(c / 16 * k + j, 0, 0, c % 16);
        ((T *)a.out)[t0 * 16 + c] = (T)v;
    }
}

// ---- weighted sum ----------------------------------------------------------
// How many of a token's logits come before number e, whose order is `mine`.
__device__ inline int32_t rank_of(const uint32_t *order, int32_t E, int32_t e, uint32_t mine)
{
    int32_t above = 0;
    for (int32_t f = 0; f < E; f += 4) {   // (order[E ..] up to a multiple of 4 is 0)
        const u32x4 o = *(const u32x4 *)(order + f);
#pragma unroll
        for (int i = 0; i < 4; ++i) above += o[i] > mine || (o[i] == mine && f + i < e);
    }
    return above;
}

enum { COMBINE_THREADS = 256 };
static_assert(MOE_TOP_MAX <= COMBINE_THREADS, "a thread to each of a token's weights");
template <class T>
__global__ __launch_bounds__(COMBINE_THREADS) void moe_combine_kernel(MoeArgs a)
{
    __shared__ uint32_t order[EXPERTS_MAX];
    __shared__ float part[COMBINE_THREADS / 64], chosen[MOE_TOP_MAX];
    const int32_t t = (int32_t)blockIdx.y, tid = (int32_t)threadIdx.x;
    const float *row = a.logits + t * a.E;
    // the first results are on their way while the weights are found
    constexpr int AHEAD = 8;
    const int32_t c = ((int32_t)blockIdx.x * COMBINE_THREADS + tid) * 4, cc = min(c, a.H - 4);
    const float *y0 = a.y + (int64_t)t * a.top_k * a.H + cc;
    f32x4 y[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) y[j] = *(const f32x4 *)(y0 + (int64_t)min(j, a.top_k - 1) * a.H);
    for (int32_t e = tid; e < (a.E + 3) / 4 * 4; e += COMBINE_THREADS) order[e] = e < a.E ? order_of(row[e]) : 0u;
    __syncthreads();
    for (int32_t e = tid; e < a.E; e += COMBINE_THREADS) {
        const int32_t above = rank_of(order, a.E, e, order[e]);
        if (above < a.top_k) {
            chosen[above] = row[e];
            if (a.ids && blockIdx.x == 0) a.ids[t * a.top_k + above] = e;
        }
    }
    __syncthreads();
    const float largest = chosen[0];
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
    if (c >= a.H) return;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
        if (j < a.top_k) {
            const float p = a.scale * (expf(chosen[j] - largest) / total);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += p * y[j][i];
        }
    for (int32_t j = AHEAD; j < a.top_k; ++j) {
        const float p = a.scale * (expf(chosen[j] - largest) / total);
        const f32x4 z = *(const f32x4 *)(y0 + (int64_t)j * a.H);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += p * z[i];
    }
    *(u32x2 *)((T *)a.out + (int64_t)t * a.H + c) = u32x2{pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3])};
}

// One of the two products' launches: `tiles` of an expert, sums of `per_tile` tiles of 16 columns
// each in LDS.
enum { MOE_LDS = 156 * 1024 };
struct MoeShape {
    MoeGrid g;
    uint32_t wgs, lds;
};
template <int G> static MoeShape moe_shape(const MoeArgs &a, int32_t tiles, int32_t K, int planes, int per_tile, int cu)
{
    MoeShape m;
    const int32_t lines = (K + 255) / 256, pairs = a.T * a.top_k;
    m.g.active = 4 * pairs < 5 * a.E;   // (never without where there are fewer pairs than experts: lists are for as many)
    m.g.rows = a.T < 16 ? a.T : 16;
    m.g.tiles = tiles;
    // 66 KiB of x: 16 rows of it, the longest rings and a first product's sums fill MOE_LDS.  Longer rows come
    // in chunks: 16 tokens of 2 of 8 of 2048 x 4096 take 45 us, of 2304 x 4096 67 (which the router's launch
    // adds 5 to)
    m.g.chunk = w4_chunk(lines, planes * m.g.rows, 66 * 1024);
    m.g.one = m.g.chunk >= lines;
    m.g.x_bytes = W4Lds<G>::x_bytes(planes, m.g.rows, m.g.chunk);
    // a workgroup to a compute unit, or more where their sums would not find room
    const int32_t most = m.g.active ? std::min(pairs, a.E) : a.E;
    for (int32_t wgs = std::max(cu, most);; wgs += most) {
        const int32_t per = (tiles + wgs / most - 1) / (wgs / most);
        m.wgs = (uint32_t)wgs;
        m.lds = (uint32_t)std::min<int64_t>(m.g.x_bytes + W4Lds<G>::RINGS + w4_sums_bytes(m.g.one, per, per_tile, m.g.rows), INT32_MAX);
        if (m.lds <= MOE_LDS || per == 1) return m;
    }
}

template <class T, int G> static hipError_t moe_t(const MoeArgs &a, int cu, hipStream_t s)
{
    const dim3 block(64 * W4_WAVES);
    MoeShape up = moe_shape<G>(a, a.I / 16, a.H, 1, 2, cu), dn = moe_shape<G>(a, a.H / 16, a.I, 2, 1, cu);
    if (up.lds > MOE_LDS || dn.lds > MOE_LDS) return hipErrorInvalidValue;
    const bool route = up.g.one && a.E <= 16 && a.T <= 16 && a.E * a.H <= 65536;
    if (!route) hipLaunchKernelGGL((moe_router_kernel<T>), dim3((uint32_t)(a.E + 15) / 16, (uint32_t)(a.T + 15) / 16), dim3(64 * ROUTER_WAVES), 0, s, a);
    if (route) hipLaunchKernelGGL((moe_up_kernel<T, G, true, true>), dim3(up.wgs), block, up.lds, s, a, up.g);
    else if (up.g.one) hipLaunchKernelGGL((moe_up_kernel<T, G, true, false>), dim3(up.wgs), block, up.lds, s, a, up.g);
    else hipLaunchKernelGGL((moe_up_kernel<T, G, false, false>), dim3(up.wgs), block, up.lds, s, a, up.g);
    if (a.T == 1) {   // all of its experts' activations in LDS, if they find room there
        const int32_t tiles = a.H / 16, per = (tiles + cu - 1) / cu;
        const uint32_t x_bytes = W4Lds<G>::x_bytes(2, a.top_k, (a.I + 255) / 256);
        const int64_t lds = x_bytes + W4Lds<G>::RINGS + w4_sums_bytes(false, (int64_t)a.top_k * per, 1, 1);
        if (lds <= MOE_LDS) {
            hipLaunchKernelGGL((moe_down_token_kernel<T, G>), dim3((uint32_t)((tiles + per - 1) / per)), block, (uint32_t)lds, s, a, per,
                               x_bytes);
            return hipGetLastError();
        }
    }
    if (dn.g.one) hipLaunchKernelGGL((moe_down_kernel<T, G, true>), dim3(dn.wgs), block, dn.lds, s, a, dn.g);
    else hipLaunchKernelGGL((moe_down_kernel<T, G, false>), dim3(dn.wgs), block, dn.lds, s, a, dn.g);
    hipLaunchKernelGGL((moe_combine_kernel<T>), dim3((uint32_t)(a.H + 4 * COMBINE_THREADS - 1) / (4 * COMBINE_THREADS), (uint32_t)a.T),
                       dim3(COMBINE_THREADS), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_moe_w4(int ftype, int group, const MoeArgs &a, int cu, hipStream_t s)
{
    if (ftype == LB_BF16)
        return group == 32 ? moe_t<__bf16, 32>(a, cu, s) : group == 64 ? moe_t<__bf16, 64>(a, cu, s) : moe_t<__bf16, 128>(a, cu, s);
    if (ftype == LB_F16)
        return group == 32 ? moe_t<_Float16, 32>(a, cu, s) : group == 64 ? moe_t<_Float16, 64>(a, cu, s) : moe_t<_Float16, 128>(a, cu, s);
    return hipErrorInvalidValue;
}

}  // namespace lb
