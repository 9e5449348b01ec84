// Activation checkpoints in 8 bits: written from and read back to fp32 or bf16 rows.
//
// A block of 32 columns shares one power-of-two scale (mt_block.cuh): 33 bytes
// per 32 values against bf16's 64.  Both kernels only stream (a row is read
// once and written once), so HBM bandwidth bounds them.  A lane holds eight
// columns (one 16-byte bf16 load, one 8-byte code store), four neighbouring
// lanes a block, whose largest magnitude meets in two shuffles.
#include "mt_block.cuh"

namespace mt {
namespace {

struct PackParams {
  Rows r;          // plain rows (data, ld)
  Rows q;          // codes, exps
  long long n;
  int d, vecs;     // vecs: vectors of eight columns per row, rounded up to whole blocks of four
};

template <typename T, bool AL>
__global__ void __launch_bounds__(256) k_pack8(const PackParams p) {
  const long long total = p.n * p.vecs;  // a multiple of four: a block's four lanes stay together
  const long long step = (long long)gridDim.x * blockDim.x;
  const long long rounds = (total + step - 1) / step;
  long long it = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  for (long long k = 0; k < rounds; ++k, it += step) {
    const bool live = it < total;
    const long long row = live ? it / p.vecs : 0;
    const int vec = live ? (int)(it - row * p.vecs) : 0;
    Raw8<T> v{};
    if (live) v = load8<T, AL>(p.r, row, vec, p.d);
    put_packed8<T, AL>(p.q, row, vec, p.d, v, live);
  }
}

template <typename T, bool AL>
__global__ void __launch_bounds__(256) k_unpack8(const PackParams p) {
  const long long total = p.n * p.vecs;
  for (long long it = (long long)blockIdx.x * blockDim.x + threadIdx.x; it < total;
       it += (long long)gridDim.x * blockDim.x) {
    const long long row = it / p.vecs;
    const int vec = (int)(it - row * p.vecs);
    f32x2 f[4];
    widen8<T>(load8<T, AL>(p.q, row, vec, p.d), true, f);
    put8<T, AL>(p.r, row, vec, p.d, narrow8<T>(f));
  }
}

int pack_check(const PackParams& p, int dtype) {
  if (dtype != MT_F32 && dtype != MT_BF16) return MT_EINVAL;
  if (p.n < 0 || p.n > 0x7FFFFFFF || p.d < 1 || p.d > MT_MAX_BLOCK_DIM) return MT_EINVAL;
  if (p.n > 0 && (!rows_ok(p.r.data, p.r.ld, p.d, dtype) || p.q.codes == nullptr || p.q.exps == nullptr)) return MT_EINVAL;
  return MT_OK;
}

bool pack_wide(const PackParams& p, int dtype) { return rows_wide(p.r, p.d, dtype) && rows_wide(p.q, p.d, dtype); }

}  // namespace
}  // namespace mt

extern "C" {

int mt_pack8(const void* x, int64_t ldx, int64_t n, int32_t d, int dtype, int8_t* codes, uint8_t* exps,
             mt_stream stream) {
  using namespace mt;
  PackParams p{};
  p.r = Rows{const_cast<void*>(x), ldx, nullptr, nullptr};
  p.q = Rows{nullptr, 0, codes, exps};
  p.n = n;
  p.d = d;
  const int rc = pack_check(p, dtype);
  if (rc != MT_OK || n == 0) return rc;
  p.vecs = (d + kPackBlock - 1) / kPackBlock * 4;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int grid = grid_for(n * p.vecs, 256, 8);
  const bool wide = pack_wide(p, dtype);
  {
    MT_LAUNCH("k_pack8", s);
    if (dtype == MT_F32) {
      if (wide) k_pack8<float, true><<<grid, 256, 0, s>>>(p);
      else k_pack8<float, false><<<grid, 256, 0, s>>>(p);
    } else {
      if (wide) k_pack8<__nv_bfloat16, true><<<grid, 256, 0, s>>>(p);
      else k_pack8<__nv_bfloat16, false><<<grid, 256, 0, s>>>(p);
    }
  }
  return cudaGetLastError() == cudaSuccess ? MT_OK : MT_ECUDA;
}

int mt_unpack8(const int8_t* codes, const uint8_t* exps, int64_t n, int32_t d, int dtype, void* out, int64_t ldo,
               mt_stream stream) {
  using namespace mt;
  PackParams p{};
  p.r = Rows{out, ldo, nullptr, nullptr};
  p.q = Rows{nullptr, 0, const_cast<int8_t*>(codes), const_cast<uint8_t*>(exps)};
  p.n = n;
  p.d = d;
  const int rc = pack_check(p, dtype);
  if (rc != MT_OK || n == 0) return rc;
  p.vecs = (d + 7) / 8;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int grid = grid_for(n * p.vecs, 256, 8);
  const bool wide = pack_wide(p, dtype);
  {
    MT_LAUNCH("k_unpack8", s);
    if (dtype == MT_F32) {
      if (wide) k_unpack8<float, true><<<grid, 256, 0, s>>>(p);
      else k_unpack8<float, false><<<grid, 256, 0, s>>>(p);
    } else {
      if (wide) k_unpack8<__nv_bfloat16, true><<<grid, 256, 0, s>>>(p);
      else k_unpack8<__nv_bfloat16, false><<<grid, 256, 0, s>>>(p);
    }
  }
  return cudaGetLastError() == cudaSuccess ? MT_OK : MT_ECUDA;
}

}  // extern "C"
