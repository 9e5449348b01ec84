// Operands of the tensor cores made from rows that do not fit them as they are:
// padded copies, and fp32 rows as three bf16 parts.
#pragma once

#include "mt_block.cuh"

namespace mt {

// x as three bf16 numbers whose sum is x: each takes the next eight bits, rounded to nearest, so what it leaves is at most 2^-8
// of it, and three times eight bits are all that x has (what is below the least subnormal of bf16 is lost).  The products of
// parts that the six leave out are then at most 2 x 2^-25 + 2^-34 of the whole.  A value that rounds to an infinity is cut off
// instead; an infinity or NaN is the first part alone, and becomes NaN in a product with parts that are zero.
__device__ __forceinline__ void split3(float x, __nv_bfloat16& a, __nv_bfloat16& b, __nv_bfloat16& c) {
  a = __float2bfloat16_rn(x);
  if (__hisinf(a) && !isinf(x)) a = __float2bfloat16_rz(x);
  const float r = x - __bfloat162float(a);  // exact
  const bool finite = fabsf(x) <= 3.4028235e38f;
  b = finite ? __float2bfloat16_rn(r) : __float2bfloat16_rn(0.0f);
  c = finite ? __float2bfloat16_rn(r - __bfloat162float(b)) : __float2bfloat16_rn(0.0f);
}
__device__ __forceinline__ uint32_t bf16_bits(__nv_bfloat16 a, __nv_bfloat16 b) {
  return (uint32_t)__bfloat16_as_ushort(a) | (uint32_t)__bfloat16_as_ushort(b) << 16;
}

// The same of two values into pairs, where none is near the largest number (one that is, or an infinity, becomes NaN).
__device__ __forceinline__ void split3_pair(float x, float y, uint32_t (&w)[3]) {
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    w[q] = bf16x2_of(x, y);
    x -= __uint_as_float(w[q] << 16);
    y -= __uint_as_float(w[q] & 0xFFFF0000u);
  }
}

// Columns of a part of a padded copy: a multiple of 8 (the copies' strides), of 64 where several parts lie side by side (a
// step of the contraction must not reach into the next part).
inline int64_t part_columns(int64_t d, int parts) { return parts == 1 ? (d + 7) / 8 * 8 : (d + 63) / 64 * 64; }

// planes x rows x d values of dtype, rows ld apart, into planes x padded_rows x (parts x part_columns(d)) bf16; what is added
// is zero.  parts: 1 (bf16) or 3 (fp32).
cudaError_t launch_parts(const void* in, int64_t ld, int64_t planes, int64_t rows, int64_t padded_rows, int64_t d, int dtype,
                         __nv_bfloat16* out, cudaStream_t s);
// The reverse for bf16: planes x rows x d values, rows ldo apart, out of planes x padded_rows x ldi.
cudaError_t launch_unpad(const __nv_bfloat16* in, int64_t ldi, int64_t planes, int64_t rows, int64_t padded_rows, int64_t d,
                         __nv_bfloat16* out, int64_t ldo, cudaStream_t s);

}  // namespace mt
