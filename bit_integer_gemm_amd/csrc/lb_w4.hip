// lb_w4.hip -- linear layer with 4-bit weights and group scales on 16-bit activations.
//
//   out[m,n] = round(sum_k x[m,k] (u[n,k] s[n,g] + b[n,g]) + bias[n]),  g = k / G
#include "lb_layer.hpp"
#include "lb_w4.hpp"

namespace lb {

// Up to 16 rows: a workgroup takes all of x against some tiles of 16 columns.  1 x 4096 x 4096
// (G = 128) in 5.9 us (a launch and three latencies; the bytes alone would take 1.8), 8 x 11008 x
// 4096 (G = 64) in 10.7 us, 2.5 TB/s.  x is asked for first: with the weights first, the latter took
// 1.2 us more.  As calls in a graph 16 x 4096 x 4096 and 16 x 11008 x 4096 (G = 128) take 10.8 and 13.4 us,
// where the tiles for more rows take 14.8 and 22.4 (their three launches); 16 x 4096 x 11008 (G = 64)
// 21.4 and 22.0.  17 rows of them take 14.8, 22.3 and 21.8 there, and would read all weights twice here.
// ONE: all of x is in LDS at once.
struct FewArgs {
    const uint8_t *w;
    const uint32_t *p;
    int64_t ldx;
    int32_t M, N, K;
    int32_t per, chunk;   // tiles of a workgroup, lines whose x is in LDS together
};
template <class T, int G, bool ONE>
__global__ __launch_bounds__(64 * W4_WAVES) void w4_few_kernel(const T *__restrict__ X, const T *__restrict__ bias,
                                                                  T *__restrict__ out, FewArgs a)
{
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    const int32_t wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), rows = a.M;
    const int32_t t0 = (int32_t)blockIdx.x * a.per, tiles = min(a.per, (a.N + 15) / 16 - t0);
    const uint32_t x_bytes = W4Lds<G>::x_bytes(1, rows, a.chunk);
    const W4Sums<ONE> sums(smem + x_bytes + W4Lds<G>::RINGS, tiles, 1, rows);
    auto put = [&](int32_t t, int32_t m, int32_t c, float v) {
        const int32_t n = (t0 + t) * 16 + c;
        if (n < a.N) out[(int64_t)m * a.N + n] = (T)(bias ? v + (float)bias[n] : v);
    };
    auto tile_at = [&](int32_t t) { return W4Tile{(int64_t)(t0 + t) * 16, min(16, a.N - (t0 + t) * 16)}; };
    W4Flow<T, T, G, 1, decltype(tile_at)> flow(smem, x_bytes, a.w, a.p, a.K, a.chunk, tile_at);
    flow.template run<false>(
        tiles, rows, make_rsrc(X, 0xFFFFFFF0u), [&](int32_t row) { return (uint32_t)row * (uint32_t)a.ldx * 2u; },
        [&](int32_t t, const f32x4 &acc, bool more) {
            if (!sums.whole(wave, t)) return w4_put(sums.at(wave, t, 0), rows, acc, more);
            w4_rows(rows, [&](int32_t i, int32_t m, int32_t c) { put(t, m, c, acc[i]); });
        });
    __syncthreads();
    sums.each([&](int32_t t, int32_t m, int32_t c) { put(t, m, c, sums.sum(t, 0, m, c)); });
}

enum { FEW_LDS = 160 * 1024 };
static_assert((int64_t)LB_W4_N_MAX / 16 * 64 * W4_WAVES <= LAUNCH_THREADS, "all columns in a launch");
template <class T, int G> static hipError_t w4_g(const W4Args &a, int cu, hipStream_t s)
{
    const int64_t tiles = (a.N + 15) / 16, lines = (a.K + 255) / 256;
    // a workgroup to a compute unit, if its sums find room
    int64_t per = (tiles + cu - 1) / cu;
    int32_t chunk = w4_chunk(lines, a.M, FEW_LDS - 1024 - W4Lds<G>::RINGS - w4_sums_bytes(true, per, 1, a.M));
    const bool one = chunk >= lines;
    while (!one && per > 1 && w4_sums_bytes(false, per, 1, a.M) > 40 * 1024) per = (per + 1) / 2;
    const int64_t sums = w4_sums_bytes(one, per, 1, a.M), wgs = (tiles + per - 1) / per;
    if (!one) chunk = w4_chunk(lines, a.M, FEW_LDS - 1024 - W4Lds<G>::RINGS - sums);
    const FewArgs f{a.w, (const uint32_t *)a.p, a.ldx, (int32_t)a.M, (int32_t)a.N, (int32_t)a.K, (int32_t)per, chunk};
    const uint32_t lds = W4Lds<G>::x_bytes(1, f.M, f.chunk) + W4Lds<G>::RINGS + (uint32_t)sums;
    if (a.M > W4_FEW_ROWS || wgs * 64 * W4_WAVES > LAUNCH_THREADS || lds > FEW_LDS) return hipErrorInvalidValue;
    const dim3 grid((uint32_t)wgs), block(64 * W4_WAVES);
    const T *x = (const T *)a.x, *bias = (const T *)a.bias;
    T *out = (T *)a.out;
    if (one) hipLaunchKernelGGL((w4_few_kernel<T, G, true>), grid, block, lds, s, x, bias, out, f);
    else hipLaunchKernelGGL((w4_few_kernel<T, G, false>), grid, block, lds, s, x, bias, out, f);
    return hipGetLastError();
}

template <class T> static hipError_t w4_t(const W4Args &a, int group, int cu, hipStream_t s)
{
    return group == 32 ? w4_g<T, 32>(a, cu, s) : group == 64 ? w4_g<T, 64>(a, cu, s) : w4_g<T, 128>(a, cu, s);
}

hipError_t launch_linear_w4(int ftype, int group, const W4Args &a, int cu, hipStream_t s)
{
    switch (ftype) {
    case LB_BF16: return w4_t<__bf16>(a, group, cu, s);
    case LB_F16: return w4_t<_Float16>(a, group, cu, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace lb
