// lb_layer.hpp -- host-side interface between the C ABI and the kernels of the operators that
// complete a decoder layer.  (Apart from lb_internal.hpp, whose code the counter profiles of the
// GEMM kernels are stamped with.)
#pragma once

#include "lb_internal.hpp"

namespace lb {

// The norms between two blocks (formula in lb_gemm.h): y, r, post_w, gate, r_out and x may
// be null.
struct NormArgs {
    const void *y, *r, *post_w, *gate, *w;
    void *r_out, *x;
    int64_t ldy, ldr, ldg, ldro, ldx;
    int32_t H;
    float alpha, eps;
};
hipError_t launch_residual_norm(int ftype, int rtype, const NormArgs &a, int64_t M, hipStream_t s);

// Rotary positions of Hq heads of q and Hk of k (k may be null, Hk 0).  tokens, heads: those of
// a workgroup, items: vectors of 8 of a head (launch_rope sets them).
struct RopeArgs {
    const void *q, *k;
    void *qo, *ko;
    const int64_t *pos;
    const double *freqs;
    int64_t ldq, ldk, ldqo, ldko, T;
    int32_t Hq, Hk, D, R;
    float mult;
    int32_t tokens, heads, items;
};
hipError_t launch_rope(int ftype, const RopeArgs &a, bool pairs, bool in_place, int cu, hipStream_t s);

// The linear layer with 4-bit weights.
struct W4Args {
    const void *x;
    int64_t ldx;
    const uint8_t *w;
    const void *p, *bias;
    void *out;
    int64_t M, N, K;
};
hipError_t launch_linear_w4(int ftype, int group, const W4Args &a, int cu, hipStream_t s);

// The same for many rows, with a workspace of linear_w4_rows_workspace bytes.
hipError_t launch_linear_w4_rows(int ftype, int group, const W4Args &a, int cu, void *workspace, hipStream_t s);
int64_t linear_w4_rows_workspace(int64_t M, int64_t N, int64_t K, int64_t group, int cu);
enum { W4_FEW_ROWS = 16 };   // rows that the first of these takes

// The mixture of experts, for at most MOE_TOKENS tokens a launch.
enum { MOE_TOKENS = 64 };
struct MoeArgs {
    const void *x;
    int64_t ldx;
    const void *wr;
    const uint8_t *w1, *w2;
    const void *p1, *p2;
    void *out;
    int32_t *ids;      // T x top_k, or null
    float *weights;    // likewise
    int32_t T, E, top_k, H, I;
    int32_t renorm;
    float scale;
    float *logits;     // workspace: T x E
    int32_t *found;    // how many experts have tokens
    int32_t *lists;    // and 2 + MOE_TOKENS for each expert or (token, rank) pair
    float *h;          // T top_k x I
    float *y;          // T top_k x H
};
hipError_t launch_moe_w4(int ftype, int group, const MoeArgs &a, int cu, hipStream_t s);

}  // namespace lb
