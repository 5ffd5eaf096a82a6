// lb_float.hpp -- 16-bit and 32-bit floating types of the serving operators:
// loads, exact widening and one rounding (to nearest, ties to even) back.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lb_device.hpp"

namespace lb {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// Two 16-bit floats packed in a word.
template <class T> __device__ inline float lo_f32(uint32_t w);
template <class T> __device__ inline float hi_f32(uint32_t w);
template <> __device__ inline float lo_f32<__bf16>(uint32_t w) { return __uint_as_float(w << 16); }
template <> __device__ inline float hi_f32<__bf16>(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
template <> __device__ inline float lo_f32<_Float16>(uint32_t w)
{
    return (float)__builtin_bit_cast(f16x2, w).x;
}
template <> __device__ inline float hi_f32<_Float16>(uint32_t w)
{
    return (float)__builtin_bit_cast(f16x2, w).y;
}

// Round two floats to T and pack them (the first in the low half).
template <class T> __device__ inline uint32_t pack2(float a, float b)
{
    typedef T t2 __attribute__((ext_vector_type(2)));
    const t2 v = {(T)a, (T)b};
    return __builtin_bit_cast(uint32_t, v);
}

// Store of the scaled product: four consecutive columns of a row
// as ((float)acc * sx[m]) * sw[n] + bias[n] in fp32, rounded once to the output
// type.  o: element offset of the first; left: columns from it to N; vec: all
// four exist and the row stride keeps them aligned.  (The type is a template
// parameter of the kernel: chosen at run time inside the unrolled epilogue, its
// three copies of every store cost 90 us of 350 at 8192 x 11008 x 4096.)
template <class T>
__device__ inline void store_scaled(const T *bias, T *out, int64_t o, int64_t n, int64_t left, bool vec, f32x4 v)
{
    typedef T t4 __attribute__((ext_vector_type(4)));
    if (vec) {
        if (bias) {
            const t4 b = *(const t4 *)(bias + n);
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] += (float)b[r];
        }
        *(t4 *)(out + o) = t4{(T)v.x, (T)v.y, (T)v.z, (T)v.w};
    } else {
        for (int r = 0; r < 4 && r < left; ++r) out[o + r] = (T)(bias ? v[r] + (float)bias[n + r] : v[r]);
    }
}

}  // namespace lb
