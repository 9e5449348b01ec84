// Padded copies and fp32 rows in three bf16 parts (mt_parts.cuh).  Bound by HBM; a
// thread makes eight columns of every part.
#include "mt_parts.cuh"

namespace mt {
namespace {

template <typename T, bool AL>
__global__ void __launch_bounds__(256) k_parts(const T* in, int64_t ld, long long planes, long long rows, long long padded, int d,
                                               int dp, __nv_bfloat16* out) {
  constexpr int kParts = sizeof(T) == 4 ? 3 : 1;
  const int vecs = dp / 8;
  const long long total = planes * padded * vecs;
  for (long long t = (long long)blockIdx.x * blockDim.x + threadIdx.x; t < total; t += (long long)gridDim.x * blockDim.x) {
    const long long row = t / vecs, plane = row / padded, i = row - plane * padded;
    const int vec = (int)(t - row * vecs);
    Raw8<T> v;
    if (i < rows) {
      v = load8<T, AL>(Rows{const_cast<T*>(in) + (plane * rows + i) * ld, 0, nullptr, nullptr}, 0, vec, d);
    } else {
      v.a = make_uint4(0u, 0u, 0u, 0u);
      if constexpr (sizeof(T) == 4) v.b = v.a;
    }
    __nv_bfloat16* to = out + (size_t)row * (kParts * dp) + vec * 8;
    if constexpr (kParts == 1) {
      *reinterpret_cast<uint4*>(to) = v.a;
    } else {
      float f[8];
      widen8<T>(v, false, f);
      uint32_t w[3][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        __nv_bfloat16 a[3], b[3];
        split3(f[2 * j], a[0], a[1], a[2]);
        split3(f[2 * j + 1], b[0], b[1], b[2]);
#pragma unroll
        for (int q = 0; q < 3; ++q) w[q][j] = bf16_bits(a[q], b[q]);
      }
#pragma unroll
      for (int q = 0; q < 3; ++q) *reinterpret_cast<uint4*>(to + (size_t)q * dp) = make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
    }
  }
}

__global__ void __launch_bounds__(256) k_unpad(const __nv_bfloat16* in, int64_t ldi, long long planes, long long rows, long long padded,
                                               int d, __nv_bfloat16* out, int64_t ldo) {
  const long long total = planes * rows * d;
  for (long long t = (long long)blockIdx.x * blockDim.x + threadIdx.x; t < total; t += (long long)gridDim.x * blockDim.x) {
    const long long row = t / d, plane = row / rows;
    const int j = (int)(t - row * d);
    out[(size_t)row * ldo + j] = in[(size_t)(plane * padded + row - plane * rows) * ldi + j];
  }
}

}  // namespace

cudaError_t launch_parts(const void* in, int64_t ld, int64_t planes, int64_t rows, int64_t padded, int64_t d, int dtype,
                         __nv_bfloat16* out, cudaStream_t s) {
  const int parts = dtype == MT_F32 ? 3 : 1;
  const int dp = (int)part_columns(d, parts);
  const bool al = d % 8 == 0 && is_aligned(in, 16) && ld * elem_bytes(dtype) % 16 == 0;
  const long long work = planes * padded * (dp / 8);
  if (work == 0) return cudaSuccess;
  const int grid = grid_for(work, 256, 8);
  MT_LAUNCH("k_parts", s);
  if (dtype == MT_F32) {
    if (al) k_parts<float, true><<<grid, 256, 0, s>>>(static_cast<const float*>(in), ld, planes, rows, padded, (int)d, dp, out);
    else k_parts<float, false><<<grid, 256, 0, s>>>(static_cast<const float*>(in), ld, planes, rows, padded, (int)d, dp, out);
  } else {
    if (al) k_parts<__nv_bfloat16, true><<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(in), ld, planes, rows, padded, (int)d, dp, out);
    else k_parts<__nv_bfloat16, false><<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(in), ld, planes, rows, padded, (int)d, dp, out);
  }
  return cudaGetLastError();
}

cudaError_t launch_unpad(const __nv_bfloat16* in, int64_t ldi, int64_t planes, int64_t rows, int64_t padded, int64_t d,
                         __nv_bfloat16* out, int64_t ldo, cudaStream_t s) {
  const long long work = planes * rows * d;
  if (work == 0) return cudaSuccess;
  MT_LAUNCH("k_unpad", s);
  k_unpad<<<grid_for(work, 256, 8), 256, 0, s>>>(in, ldi, planes, rows, padded, (int)d, out, ldo);
  return cudaGetLastError();
}

}  // namespace mt
