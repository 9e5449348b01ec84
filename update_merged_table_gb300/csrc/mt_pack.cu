// Activation checkpoints in 8 bits: written from and read back to fp32 or bf16 rows.
//
// A block of 32 columns shares one power-of-two scale (mt_block.cuh): 33 bytes
// per 32 values against bf16's 64.  Both kernels only stream (a row is read
// once and written once), so HBM bandwidth bounds them.  A lane holds eight
// columns (one 16-byte bf16 load, one 8-byte code store), four neighbouring
// lanes a block, whose largest magnitude meets in two shuffles.  Measured, of the
// copy bandwidth: bf16 490,011 x 512 packed in 139 us (81%), unpacked in 131 (86%);
// fp32 245,003 x 512 100 (93%) and 139 (67%); bf16 200,003 x 777, an element at a time,
// 180 (39%) and 387 (18%).
#include "mt_block.cuh"

namespace mt {
namespace {

struct PackParams {
  Rows r;          // plain rows (data, ld)
  Rows q;          // codes, exps
  long long n, total;  // total: vectors of all rows
  int d, vecs;     // vecs: vectors of eight columns per row (packing: rounded up to whole blocks of four)
};

// Vectors a lane has in flight.  Reading bf16 and writing codes gains from four (1.97M x 64: 72 us, one 78), reading codes
// and writing bf16 is bound by its writes and loses by them (78 us, one 67).
constexpr int kPackVecs = 4, kUnpackVecs = 1;

// Vectors of a launch: lane `lane` of a warp takes the vectors it0 + 32 u + lane.  Where the rows follow one another without gaps and are whole blocks (FLAT), finding a vector
// takes no division: everything is cut into rows of 2^20 vectors.
struct Item {
  long long row;
  int vec;
};
template <bool FLAT>
__device__ __forceinline__ Item item_of(const PackParams& p, long long it) {
  if (FLAT) return Item{it >> 20, (int)(it & ((1 << 20) - 1))};
  const long long row = p.total >> 32 ? it / p.vecs : (long long)((uint32_t)it / (uint32_t)p.vecs);
  return Item{row, (int)(it - row * p.vecs)};
}

template <typename T, bool AL, bool FLAT>
__global__ void __launch_bounds__(256) k_pack8(const PackParams p) {
  const long long total = p.total;  // a multiple of four: a block's four lanes stay together
  const int lane = threadIdx.x & 31;
  const long long warp = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5, warps = ((long long)gridDim.x * blockDim.x) >> 5;
  for (long long it0 = warp * 32 * kPackVecs; it0 < total; it0 += warps * 32 * kPackVecs) {
    Raw8<T> v[kPackVecs];
    Item x[kPackVecs];
#pragma unroll
    for (int u = 0; u < kPackVecs; ++u) {
      const long long it = it0 + u * 32 + lane;
      x[u] = item_of<FLAT>(p, it < total ? it : 0);
      v[u] = it < total ? load8<T, AL>(p.r, x[u].row, x[u].vec, p.d) : Raw8<T>{};
    }
#pragma unroll
    for (int u = 0; u < kPackVecs; ++u)
      put_packed8<T, AL>(p.q, x[u].row, x[u].vec, p.d, v[u], it0 + u * 32 + lane < total);
  }
}

template <typename T, bool AL, bool FLAT>
__global__ void __launch_bounds__(256) k_unpack8(const PackParams p) {
  const long long total = p.total;
  const int lane = threadIdx.x & 31;
  const long long warp = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5, warps = ((long long)gridDim.x * blockDim.x) >> 5;
  for (long long it0 = warp * 32 * kUnpackVecs; it0 < total; it0 += warps * 32 * kUnpackVecs) {
    Raw8<T> v[kUnpackVecs];
    Item x[kUnpackVecs];
#pragma unroll
    for (int u = 0; u < kUnpackVecs; ++u) {
      const long long it = it0 + u * 32 + lane;
      x[u] = item_of<FLAT>(p, it < total ? it : 0);
      v[u] = it < total ? load8<T, AL>(p.q, x[u].row, x[u].vec, p.d) : Raw8<T>{};
    }
#pragma unroll
    for (int u = 0; u < kUnpackVecs; ++u) {
      f32x2 f[4];
      widen8<T>(v[u], true, f);
      if (it0 + u * 32 + lane < total) put8<T, AL>(p.r, x[u].row, x[u].vec, p.d, narrow8<T>(f));
    }
  }
}

int pack_check(const PackParams& p, int dtype) {
  if (dtype != MT_F32 && dtype != MT_BF16) return MT_EINVAL;
  if (p.n < 0 || p.n > 0x7FFFFFFF || p.d < 1 || p.d > MT_MAX_BLOCK_DIM) return MT_EINVAL;
  if (p.n > 0 && (!rows_ok(p.r.data, p.r.ld, p.d, dtype) || p.q.codes == nullptr || p.q.exps == nullptr)) return MT_EINVAL;
  Regions all;  // the rows and the two parts of the checkpoint: all apart, whichever is written
  all.out(p.r, p.n, p.d, dtype);
  all.out_packed(p.q, p.n, p.d);
  return all.clash() ? MT_EINVAL : MT_OK;
}

bool pack_wide(const PackParams& p, int dtype) { return rows_wide(p.r, p.d, dtype) && rows_wide(p.q, p.d, dtype); }

// Sets the vectors of a launch and, where the rows allow it, cuts them anew (FLAT).
bool pack_flat(PackParams& p, bool wide, int vecs) {
  p.vecs = vecs;
  p.total = p.n * vecs;
  if (!wide || p.r.ld != p.d || p.d % kPackBlock != 0) return false;
  p.d = 8 << 20;
  p.r.ld = p.d;
  return true;
}

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
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool wide = pack_wide(p, dtype), flat = pack_flat(p, wide, (d + kPackBlock - 1) / kPackBlock * 4);
  const int grid = grid_for((p.total + kPackVecs - 1) / kPackVecs, 256, 8);
  {
    MT_LAUNCH("k_pack8", s);
    if (dtype == MT_F32) {
      if (flat) k_pack8<float, true, true><<<grid, 256, 0, s>>>(p);
      else if (wide) k_pack8<float, true, false><<<grid, 256, 0, s>>>(p);
      else k_pack8<float, false, false><<<grid, 256, 0, s>>>(p);
    } else {
      if (flat) k_pack8<__nv_bfloat16, true, true><<<grid, 256, 0, s>>>(p);
      else if (wide) k_pack8<__nv_bfloat16, true, false><<<grid, 256, 0, s>>>(p);
      else k_pack8<__nv_bfloat16, false, false><<<grid, 256, 0, s>>>(p);
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
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool wide = pack_wide(p, dtype), flat = pack_flat(p, wide, (d + 7) / 8);
  const int grid = grid_for((p.total + kUnpackVecs - 1) / kUnpackVecs, 256, 8);
  {
    MT_LAUNCH("k_unpack8", s);
    if (dtype == MT_F32) {
      if (flat) k_unpack8<float, true, true><<<grid, 256, 0, s>>>(p);
      else if (wide) k_unpack8<float, true, false><<<grid, 256, 0, s>>>(p);
      else k_unpack8<float, false, false><<<grid, 256, 0, s>>>(p);
    } else {
      if (flat) k_unpack8<__nv_bfloat16, true, true><<<grid, 256, 0, s>>>(p);
      else if (wide) k_unpack8<__nv_bfloat16, true, false><<<grid, 256, 0, s>>>(p);
      else k_unpack8<__nv_bfloat16, false, false><<<grid, 256, 0, s>>>(p);
    }
  }
  return cudaGetLastError() == cudaSuccess ? MT_OK : MT_ECUDA;
}

}  // extern "C"
