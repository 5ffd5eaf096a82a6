// lb_internal.hpp -- host-side interface between the C ABI and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lb_gemm.h"

namespace lb {

// KIND_B1 runs the 1-bit GEMM on the int8 instruction (eight weighted bit
// planes per 64-byte block), KIND_B1F4 on the FP4 instruction (four bit planes
// per block, fp32 accumulation exact below 2^24).
// KIND_SCALED is the int8 product with both scales, a bias and a 16- or 32-bit
// floating output (launch_scaled).
enum { KIND_S8 = 0, KIND_S4 = 1, KIND_LINEAR = 2, KIND_B1 = 3, KIND_B1F4 = 4, KIND_SCALED = 5 };

// Internal tile codes beside the nine public variants (never accepted from a
// caller): the four-wave kernel on 256x192 tiles (int8, int4 and 1-bit FP4-
// route GEMMs, linear layer) and on 192x256 tiles (int8 GEMM, linear layer).
enum { W4_256x192 = 16, W4_192x256 = 17 };
// Internal tile code of the convolutions: a 64x64 tile with two 64-byte
// stages (16 KiB of LDS, up to eight workgroups per CU).
enum { CONV_64x64_K64 = 18 };
// Internal tile codes of the scaled product: tiles with four 128-byte stages, one
// workgroup per CU, where all of them run at once.
enum { SCALED_128x64 = 19, SCALED_64x128 = 20, SCALED_128x128 = 21 };

// int8 MFMA family (int8 GEMM, packed-int4 GEMM, int8 linear layer, and the
// 1-bit GEMM on weighted bit planes).  Kb is the row length of A and B in
// bytes (K for int8, K/2 for int4, K/8 for 1-bit); ldo is the distance in
// elements between rows of the output (N for a whole product, more when the
// launch covers a band of its columns).  ksplit < Kb (integer GEMMs only, a
// multiple of the variant's stage depth) runs ceil(Kb / ksplit) bands of K in
// one grid, each adding its partial sums into C, which must hold zeros.
hipError_t launch_mfma(int kind, int variant, const void *A, const void *B, void *out,
                       const float *sx, const float *sw, int64_t M, int64_t N, int64_t Kb,
                       int64_t ldo, int64_t ksplit, hipStream_t s);
// Output of a scaled product: its float type (lb_ftype) and the bias of each
// column in that type (null: none).
struct ScaledOut {
    const void *bias;
    int32_t ftype;
};
// out = ((float)(A x B) * sx[m]) * sw[n] + bias[n], rounded to so.ftype; tiles as
// launch_mfma's linear layer.
hipError_t launch_scaled(int variant, const int8_t *A, const int8_t *B, void *out, const float *sx,
                         const float *sw, int64_t M, int64_t N, int64_t K, int64_t ldo,
                         const ScaledOut &so, hipStream_t s);
// The same with the launches of an automatic choice; an lb_status.
int scaled_auto(const int8_t *X, const int8_t *W, const float *sx, const float *sw, void *out, int64_t M,
                int64_t N, int64_t K, int64_t ldo, const ScaledOut &so, hipStream_t s);
// Threads of one launch: the runtime takes fewer than 2^32, and calls that need more
// make several launches.
enum : int64_t { LAUNCH_THREADS = (int64_t)1 << 31 };
// Whether LB_AUTO_VARIANT fixes the variant of automatic calls.
bool variant_is_forced();
// Rows of X (K elements, ldx apart, 16-byte aligned) quantised to int8 with a
// scale each.
hipError_t launch_quant_rows(int ftype, const void *X, int64_t ldx, int8_t *Q, float *sx, int64_t M,
                             int64_t K, hipStream_t s);
// The scaled product where few tiles cover it (linear_is_few).
bool linear_is_few(int64_t M, int64_t N, int cu);
bool linear_few_tile(int64_t M, int64_t N, int cu, int *tm, int *tn);   // and the tile it takes there
hipError_t launch_linear_few(int ftype, const int8_t *Xq, const int8_t *W, const float *sx, const float *sw,
                             const void *bias, void *out, int64_t M, int64_t N, int64_t K, int cu,
                             hipStream_t s);
// The same from floating activations, quantised on the way (where linear_fuses).
bool linear_fuses(int64_t M, int64_t N, int64_t K, int cu);
hipError_t launch_linear_fused(int ftype, const void *X, int64_t ldx, const int8_t *W, const float *sw,
                               const void *bias, void *out, int64_t M, int64_t N, int64_t K, int cu,
                               hipStream_t s);
// Zero n int32 values on the stream (a kernel, not a memset).
hipError_t launch_zero_i32(int32_t *p, int64_t n, hipStream_t s);
// Workgroup tile and stage of a variant; bk_bytes is the K depth of a stage in bytes.
int mfma_variant_info(int kind, int variant, int *bm, int *bn, int *bk_bytes, int *stages);

// Geometry of a convolution run as a GEMM whose A rows are gathered from an
// NHWC image: output pixel r = (n*Ho + ho)*Wo + wo is row r, the filter taps
// (kh, kw, channel byte) are the K axis.  Cb is bytes per pixel (C or C/2) and
// a multiple of 16; x_bytes = N*H*W*Cb < 2^31.
struct ConvGeom {
    int32_t H, W, Cb, Kh, Kw, sh, sw, ph, pw, Ho, Wo;
    uint32_t x_bytes;
};
// kind KIND_S8 or KIND_S4; M = N*Ho*Wo, N = Co, Kb = Kh*Kw*Cb.
hipError_t launch_conv(int kind, int variant, const void *X, const void *F, int32_t *Y,
                       int64_t M, int64_t N, int64_t Kb, const ConvGeom &g, hipStream_t s);

// The 4-bit paged cache (layout in lb_gemm.h).
struct Kv4Cache {
    uint8_t *k, *v;
    uint32_t *kp, *vp;   // one word per vector: scale in the low half, minimum in the high half
    int64_t pages;
    int32_t page, heads;
    uint32_t page_mul, page_shift;   // slot / page = mulhi(slot, page_mul) >> page_shift, slots below 2^31
};
// New keys and values (T tokens, ld elements apart, heads x D each) into slots;
// and vectors of slots out again.
hipError_t launch_kv4_write(int ftype, const void *K, const void *V, int64_t ldk, int64_t ldv,
                            const int64_t *slots, const Kv4Cache &c, int64_t T, int D, hipStream_t s);
hipError_t launch_kv4_read(int ftype, const Kv4Cache &c, const int64_t *slots, void *K, void *V, int64_t T,
                           int D, hipStream_t s);

// The attention kernels: a tile of 16 rows to a workgroup of four waves, or of as
// many as a compute unit holds; the work of all such tiles in equal shares; tiles of
// 256 rows (D = 256: 128).
enum { ATTN_ROWS = 0, ATTN_WIDE = 1, ATTN_FLAT = 2, ATTN_CHUNK = 3 };
enum { ATTN_FLAT_BATCH = 1024 };   // sequences, at most
struct AttnArgs {
    const void *q;
    void *out;
    float *lse;
    const int32_t *table, *q_off, *lens;
    float *part;          // workspace: partial results of key ranges or shares
    Kv4Cache c;
    int64_t ldq, ldo, ldt, width;
    int64_t total_q;
    int32_t group, batch, window, causal;
    int32_t splits;       // key ranges of a tile at most; ATTN_FLAT: shares at most
    int32_t unit;         // fewest blocks of keys (ATTN_CHUNK: of 64, else of 32) worth a workgroup of their own
    int32_t kernel, tiles; // ATTN_*, and how many tiles of its rows a key head has
    float scale2;         // softmax scale * log2(e)
};
// Waves of an ATTN_WIDE workgroup.
constexpr int attn_wide_waves(int D) { return D == 64 ? 16 : D == 128 ? 12 : 8; }
hipError_t launch_attn(int ftype, int D, const AttnArgs &a, hipStream_t s);

// Measured selection table lookup (host only).
int select_from_table(int dtype, int64_t M, int64_t N, int64_t K, int cu_count, int *best,
                      int *second);
// Compute units of the current device (cached per device).
int device_cu_count(int *cu);

}  // namespace lb
