// Grouped matrix products in bf16 on the tensor cores (tcgen05): forward, dx and dW.
//
// One persistent block per SM walks the output tiles of all groups; inside it
// one thread keeps a ring of shared-memory stages filled by TMA, one thread
// issues the products into tensor memory, and four warps read finished tiles
// out while the next tile's products run (two accumulators).
//
//  k_linear_rows_tc     forward and dx: 128 rows of one group x BN columns.  The
//                       copies may read past a group's last row (the next
//                       group's rows, or zeros past n): those rows of the
//                       product are not stored.
//  k_linear_weights_tc  dW: 128 columns of x by BN columns of dy over one chunk
//                       of a group's rows, both operands with the rows as the
//                       contraction (their 64-row slabs land in shared memory as
//                       they lie in global memory).  Rows past the chunk's end
//                       are zeroed in shared memory before the product reads
//                       them.  x in 8 bits lands as codes and is widened in
//                       place by the eight read-out warps; x is the operand of
//                       128 columns and not of BN so that this work is the
//                       smaller.
//
// The tensor core cuts its fp32 accumulator off towards zero at every step:
// measured, a sum over r rows of unit normal products comes out 1.1e-9 * r short
// (4.4e-6 at 4096 rows, where an fp32 chain is 2.5e-7 off).  dW is fp32 and sums
// over many rows, so its accumulator starts anew every kPromote stages and the
// read-out warps add it to registers, rounding to nearest.
#include <algorithm>
#include <mutex>

#include "mt_linear.cuh"
#include "mt_tc.cuh"

namespace mt {

namespace tc {

namespace {
using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                            const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
Encode encoder() {
  static const Encode encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<Encode>(fn);
  }();
  return encode;
}
const cuuint32_t kUnit[3] = {1, 1, 1};
}  // namespace

bool encode_bf16(CUtensorMap* map, int rank, const void* base, uint64_t d0, uint64_t d1, uint64_t ld1, uint64_t d2,
                 uint64_t ld2, uint32_t box0, uint32_t box1) {
  const Encode encode = encoder();
  if (encode == nullptr) return false;
  const cuuint64_t dims[3] = {d0, d1, d2};
  const cuuint64_t strides[2] = {ld1 * 2, ld2 * 2};
  const cuuint32_t box[3] = {box0, box1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, kUnit,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_u8(CUtensorMap* map, const void* base, uint64_t d0, uint64_t d1, uint64_t ld1, uint32_t box0, uint32_t box1) {
  const Encode encode = encoder();
  if (encode == nullptr) return false;
  const cuuint64_t dims[2] = {d0, d1};
  const cuuint64_t strides[1] = {ld1};
  const cuuint32_t box[2] = {box0, box1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, kUnit,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tc

namespace {

constexpr int kBM = 128;         // tile rows: the lanes of tensor memory
constexpr int kBK = 64;          // contraction per stage: one 128-byte swizzled row of bf16
constexpr int kWarpsTC = 6;      // copies, products, four to read out
constexpr int kStageOut = 4096;  // bytes per read-out warp: 32 rows x 128 bytes

template <int BN>
struct Ring {
  static constexpr int kStageA = kBM * kBK * 2, kStageB = BN * kBK * 2;
  static constexpr int kStage = kStageA + kStageB;
  static constexpr int kStages = 196608 / kStage;       // 4 (BN 256), 6 (128), 8 (64)
  static constexpr int kBytes = kStages * kStage + 4 * kStageOut;
};

struct Barriers {
  uint64_t full[8], empty[8];    // a stage's copies have landed; its products are done
  uint64_t wide[8];              // a stage's 8-bit operand has been widened
  uint64_t acc_full[2], acc_empty[2];  // an accumulator is finished; it has been read out
  uint64_t done;                 // every product issued is done
  uint32_t tmem;
};

__device__ __forceinline__ void latch_status(int32_t* status, int code) {
  if (status != nullptr) atomicCAS(status, 0, code);
}

// Set-up that both kernels share: barriers, tensor memory.  Every thread calls it; ends with the block synchronised.
template <int BN>
__device__ __forceinline__ uint32_t tc_begin(Barriers& b, int read_warps) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < Ring<BN>::kStages; ++i) {
      tc::mbar_init(&b.full[i], 1);
      tc::mbar_init(&b.empty[i], 1);
      tc::mbar_init(&b.wide[i], read_warps);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&b.acc_full[i], 1);
      tc::mbar_init(&b.acc_empty[i], read_warps);
    }
    tc::mbar_init(&b.done, 1);
    tc::mbar_init_fence();
  }
  if (threadIdx.x >> 5 == 1) tc::tmem_alloc(&b.tmem, 2 * BN);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  return b.tmem;
}

template <int BN>
__device__ __forceinline__ void tc_end(uint32_t tmem) {
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (threadIdx.x >> 5 == 1) tc::tmem_free(tmem, 2 * BN);
}

// The ring's position: stage and the parity of its current use.
struct Slot {
  int stage = 0;
  uint32_t phase = 0;
  template <int STAGES>
  __device__ __forceinline__ void next() {
    if (++stage == STAGES) {
      stage = 0;
      phase ^= 1;
    }
  }
};

// After a wait ran out: the copies already issued are waited for (again with a limit) so that none lands in a block
// that has ended.
template <int STAGES>
__device__ __forceinline__ void drain(Barriers& b, Slot s, long long issued) {
  const long long k = issued < STAGES ? issued : STAGES;
  for (long long i = 0; i < k; ++i) {
    if (s.stage == 0) {
      s.stage = STAGES;
      s.phase ^= 1;
    }
    --s.stage;
    if (!tc::mbar_wait(&b.full[s.stage], s.phase)) return;
  }
}

// ---- forward and dx ------------------------------------------------------------------------

// B_MN: W_g(i, j) has its columns j contiguous (dx); otherwise its contraction i (forward).
template <int BN, bool B_MN>
__global__ void __launch_bounds__(kWarpsTC * 32, 1)
k_linear_rows_tc(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w, const LinearRows p) {
  using R = Ring<BN>;
  extern __shared__ uint8_t s_raw[];
  __shared__ Barriers bar;
  uint8_t* ring = reinterpret_cast<uint8_t*>(((uintptr_t)s_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* s_out = ring + R::kStages * R::kStage;
  long long* s_off = reinterpret_cast<long long*>(ring + R::kBytes);
  int* s_cum = reinterpret_cast<int*>(s_off + p.groups + 1);
  load_offsets(p.offsets, p.groups, p.n, s_off, p.status);
  count_tiles(s_off, p.groups, kBM, s_cum);
  const uint32_t tmem = tc_begin<BN>(bar, 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int steps = (p.I + kBK - 1) / kBK;
  const long long total = (long long)s_cum[p.groups] * p.jtiles;

  if (warp == 0) {
    if (lane == 0) {
      Slot s;
      long long issued = 0;
      bool ok = true;
      for (long long t = blockIdx.x; t < total && ok; t += gridDim.x) {
        const int rt = (int)(t / p.jtiles), j0 = (int)(t - (long long)rt * p.jtiles) * BN;
        const int g = tile_group(s_cum, p.groups, rt);
        const int r0 = (int)(s_off[g] + (long long)(rt - s_cum[g]) * kBM);
        for (int k = 0; k < steps; ++k) {
          ok = tc::mbar_wait(&bar.empty[s.stage], s.phase ^ 1);
          if (!ok) break;
          uint8_t* st = ring + s.stage * R::kStage;
          tc::mbar_expect(&bar.full[s.stage], R::kStage);
          tc::tma_load_2d(st, &map_a, &bar.full[s.stage], k * kBK, r0);
          if constexpr (B_MN) {
#pragma unroll
            for (int c = 0; c < BN / 64; ++c)
              tc::tma_load_3d(st + R::kStageA + c * 8192, &map_w, &bar.full[s.stage], j0 + c * 64, k * kBK, g);
          } else {
            tc::tma_load_3d(st + R::kStageA, &map_w, &bar.full[s.stage], k * kBK, j0, g);
          }
          ++issued;
          s.next<R::kStages>();
        }
      }
      if (!ok) {
        latch_status(p.status, MT_ECUDA);
        drain<R::kStages>(bar, s, issued);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t instr = tc::instr_bf16(kBM, BN, false, B_MN);
      Slot s;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (long long t = blockIdx.x; t < total && ok; t += gridDim.x) {
        ok = tc::mbar_wait(&bar.acc_empty[acc], acc_phase ^ 1);
        if (!ok) break;
        tc::fence_after();
        for (int k = 0; k < steps; ++k) {
          ok = tc::mbar_wait(&bar.full[s.stage], s.phase);
          if (!ok) break;
          tc::fence_after();
          const uint32_t a = tc::smem_addr(ring + s.stage * R::kStage), b = a + R::kStageA;
#pragma unroll
          for (int i = 0; i < kBK / 16; ++i) {
            const uint64_t da = tc::smem_desc(a + i * 32, 16);
            const uint64_t db = B_MN ? tc::smem_desc(b + i * 2048, 8192) : tc::smem_desc(b + i * 32, 16);
            tc::mma_bf16(tmem + acc * BN, da, db, instr, k > 0 || i > 0);
          }
          tc::mma_commit(&bar.empty[s.stage]);
          s.next<R::kStages>();
        }
        if (!ok) break;
        tc::mma_commit(&bar.acc_full[acc]);
        acc ^= 1;
        acc_phase ^= acc == 0;
      }
      tc::mma_commit(&bar.done);  // tensor memory is freed only when no product writes it, also after a wait ran out
      ok = tc::mbar_wait(&bar.done, 0) && ok;
      if (!ok) latch_status(p.status, MT_ECUDA);
    }
  } else {
    const int quad = warp & 3;  // the lanes of tensor memory this warp may read
    uint8_t* stage = s_out + quad * kStageOut;
    __nv_bfloat16* C = static_cast<__nv_bfloat16*>(p.c);
    zero_outside<__nv_bfloat16>(s_off, p.groups, p.n, C, p.ldc, p.J, (kWarpsTC - 2) * 32, threadIdx.x - 64);
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (long long t = blockIdx.x; t < total; t += gridDim.x) {
      const int rt = (int)(t / p.jtiles), j0 = (int)(t - (long long)rt * p.jtiles) * BN;
      const int g = tile_group(s_cum, p.groups, rt);
      const long long r0 = s_off[g] + (long long)(rt - s_cum[g]) * kBM + quad * 32;
      const int rows = (int)min((long long)32, s_off[g + 1] - r0);  // <= 0: none of this warp's rows is in the group
      ok = __all_sync(kFull, tc::mbar_wait(&bar.acc_full[acc], acc_phase));
      if (!ok) break;
      tc::fence_after();
      const uint32_t from = tmem + acc * BN + ((uint32_t)(quad * 32) << 16);
#pragma unroll
      for (int c0 = 0; c0 < BN; c0 += 64) {
        uint32_t v[2][32];
        tc::tmem_load32(from + c0, v[0]);
        tc::tmem_load32(from + c0 + 32, v[1]);
        tc::tmem_load_wait();
        if (c0 + 64 == BN) {  // read out: the accumulator may be written again
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&bar.acc_empty[acc]);
        }
        // 64 columns of the lane's row as eight 16-byte pieces, piece c at c ^ (lane & 7): writes and reads of eight
        // neighbouring lanes then meet all banks
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint32_t* w = &v[c >> 2][(c & 3) * 8];
          uint4 o;
          o.x = bf16x2_of(__uint_as_float(w[0]), __uint_as_float(w[1]));
          o.y = bf16x2_of(__uint_as_float(w[2]), __uint_as_float(w[3]));
          o.z = bf16x2_of(__uint_as_float(w[4]), __uint_as_float(w[5]));
          o.w = bf16x2_of(__uint_as_float(w[6]), __uint_as_float(w[7]));
          *reinterpret_cast<uint4*>(stage + lane * 128 + ((c ^ (lane & 7)) << 4)) = o;
        }
        __syncwarp();
        const int col = j0 + c0 + (lane & 7) * 8;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int r = q * 4 + (lane >> 3);
          if (r < rows && col < p.J)
            *reinterpret_cast<uint4*>(C + (r0 + r) * p.ldc + col) =
                *reinterpret_cast<const uint4*>(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
        }
        __syncwarp();
      }
      acc ^= 1;
      acc_phase ^= acc == 0;
    }
    if (!ok) latch_status(p.status, MT_ECUDA);
  }
  tc_end<BN>(tmem);
}

// ---- dW -----------------------------------------------------------------------------------------

constexpr int kPromote = 8;   // stages (of kBK rows) an accumulator sums before it is added to registers
constexpr int kReadWarps = 8;
constexpr int kWarpsW = 4 + kReadWarps;  // a warpgroup for copies and products (two of its warps idle), two to read out
// A read-out thread of the widest tile holds 128 sums beside its loads: the block's registers (384 threads x 168 at
// launch = 64512) are split anew, 56 for a control thread and 224 for a read-out thread (128 x 56 + 256 x 224 = 64512).
constexpr int kRegsLaunch = 168, kRegsControl = 56, kRegsRead = 224;
static_assert(128 * kRegsControl + 32 * kReadWarps * kRegsRead <= kWarpsW * 32 * kRegsLaunch, "the split fits the launch");

template <int BN, bool X8>
__global__ void __launch_bounds__(kWarpsW * 32, 1)
k_linear_weights_tc(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_dy, const LinearWeights p) {
  using R = Ring<BN>;
  extern __shared__ uint8_t s_raw[];
  __shared__ Barriers bar;
  uint8_t* ring = reinterpret_cast<uint8_t*>(((uintptr_t)s_raw + 1023) & ~(uintptr_t)1023);
  long long* s_off = reinterpret_cast<long long*>(ring + R::kStages * R::kStage);
  int* s_cum = reinterpret_cast<int*>(s_off + p.groups + 1);
  int* s_slot = s_cum + p.groups + 1;
  load_offsets(p.offsets, p.groups, p.n, s_off, p.status);
  count_tiles(s_off, p.groups, p.chunk, s_cum);
  count_slots(s_cum, p.groups, s_slot);
  const uint32_t tmem = tc_begin<BN>(bar, kReadWarps);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mt = (p.M + BN - 1) / BN, tiles = (p.K + kBM - 1) / kBM * mt;
  const long long total = (long long)s_cum[p.groups] * tiles;

  // tile t: chunk c of group g, the chunk's rows [first, last), dW's corner (m0, k0)
  struct Tile {
    int g, c, m0, k0, stages;
    long long first, last;
  };
  auto tile_of = [&](long long t) {
    Tile x;
    x.c = (int)(t / tiles);
    const int q = (int)(t - (long long)x.c * tiles);
    x.k0 = q / mt * kBM;
    x.m0 = (q - q / mt * mt) * BN;
    x.g = tile_group(s_cum, p.groups, x.c);
    x.first = s_off[x.g] + (long long)(x.c - s_cum[x.g]) * p.chunk;
    x.last = min(x.first + p.chunk, s_off[x.g + 1]);
    x.stages = (int)((x.last - x.first + kBK - 1) / kBK);
    return x;
  };

  if (warp < 4) {
    if constexpr (BN == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    if (warp == 0) {
      if (lane == 0) {
        constexpr uint32_t bytes = (X8 ? kBM * kBK : R::kStageA) + R::kStageB;
        Slot s;
        long long issued = 0;
        bool ok = true;
        for (long long t = blockIdx.x; t < total && ok; t += gridDim.x) {
          const Tile x = tile_of(t);
          for (long long r = x.first; r < x.last; r += kBK) {
            ok = tc::mbar_wait(&bar.empty[s.stage], s.phase ^ 1);
            if (!ok) break;
            uint8_t* st = ring + s.stage * R::kStage;
            tc::mbar_expect(&bar.full[s.stage], bytes);
            if constexpr (X8) {
              tc::tma_load_2d(st, &map_x, &bar.full[s.stage], x.k0, (int)r);
            } else {
  #pragma unroll
              for (int c = 0; c < kBM / 64; ++c)
                tc::tma_load_2d(st + c * 8192, &map_x, &bar.full[s.stage], x.k0 + c * 64, (int)r);
            }
  #pragma unroll
            for (int c = 0; c < BN / 64; ++c)
              tc::tma_load_2d(st + R::kStageA + c * 8192, &map_dy, &bar.full[s.stage], x.m0 + c * 64, (int)r);
            ++issued;
            s.next<R::kStages>();
          }
        }
        if (!ok) {
          latch_status(p.status, MT_ECUDA);
          drain<R::kStages>(bar, s, issued);
        }
      }
    }
    if (warp == 1) {
      constexpr uint32_t instr = tc::instr_bf16(kBM, BN, true, true);
      Slot s;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (long long t = blockIdx.x; t < total && ok; t += gridDim.x) {
        const Tile x = tile_of(t);
        for (int k = 0; k < x.stages; ++k) {
          if (k % kPromote == 0) {
            ok = __all_sync(kFull, tc::mbar_wait(&bar.acc_empty[acc], acc_phase ^ 1));
            if (!ok) break;
          }
          ok = __all_sync(kFull, tc::mbar_wait(X8 ? &bar.wide[s.stage] : &bar.full[s.stage], s.phase));
          if (!ok) break;
          uint8_t* st = ring + s.stage * R::kStage;
          const long long r = x.first + (long long)k * kBK;
          const int left = (int)min((long long)kBK, x.last - r);
          if (left < kBK) {
            // Rows past the chunk's end belong to others: both operands become zero there, so that nothing of them
            // (an infinity or NaN too) reaches the sum.  Row i of a 64-column slab is the 128 bytes at i * 128,
            // whatever the swizzle does inside them.
            for (int slab = 0; slab < kBM / 64 + BN / 64; ++slab)
              for (int i = left * 8 + lane; i < kBK * 8; i += 32)
                *reinterpret_cast<uint4*>(st + slab * 8192 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
            tc::fence_async_proxy();
            __syncwarp();
          }
          tc::fence_after();
          const bool closes = k % kPromote == kPromote - 1 || k + 1 == x.stages;
          if (lane == 0) {
            const uint32_t a = tc::smem_addr(st), b = a + R::kStageA;
  #pragma unroll
            for (int i = 0; i < kBK / 16; ++i)
              tc::mma_bf16(tmem + acc * BN, tc::smem_desc(a + i * 2048, 8192), tc::smem_desc(b + i * 2048, 8192), instr,
                           k % kPromote > 0 || i > 0);
            tc::mma_commit(&bar.empty[s.stage]);
            if (closes) tc::mma_commit(&bar.acc_full[acc]);
          }
          __syncwarp();
          if (closes) {
            acc ^= 1;
            acc_phase ^= acc == 0;
          }
          s.next<R::kStages>();
        }
      }
      if (lane == 0) {
        tc::mma_commit(&bar.done);  // tensor memory is freed only when no product writes it, also after a wait ran out
        ok = tc::mbar_wait(&bar.done, 0) && ok;
        if (!ok) latch_status(p.status, MT_ECUDA);
      }
    }
  } else {
    if constexpr (BN == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsRead));
    // a warp reads the 32 lanes (columns of x) that its number allows and half of the columns (of dy)
    constexpr int kCols = BN / 2;
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const uint32_t from = tmem + half * kCols + ((uint32_t)(quad * 32) << 16);
    const int tid = threadIdx.x - 128, crow = tid >> 2, cq = tid & 3;  // 8-bit x: this thread's row and 32 columns
    const int nb = (p.K + kPackBlock - 1) / kPackBlock;
    Slot s;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    float sum[kCols];

    auto read_out = [&]() {
      ok = __all_sync(kFull, tc::mbar_wait(&bar.acc_full[acc], acc_phase));
      if (!ok) return;
      tc::fence_after();
#pragma unroll
      for (int c0 = 0; c0 < kCols; c0 += 32) {
        uint32_t v[32];
        tc::tmem_load32(from + acc * BN + c0, v);
        tc::tmem_load_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) sum[c0 + j] += __uint_as_float(v[j]);
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bar.acc_empty[acc]);
      acc ^= 1;
      acc_phase ^= acc == 0;
    };

    for (long long t = blockIdx.x; t < total && ok; t += gridDim.x) {
      const Tile x = tile_of(t);
      const int parts = (x.stages + kPromote - 1) / kPromote;
#pragma unroll
      for (int j = 0; j < kCols; ++j) sum[j] = 0.0f;
      if constexpr (X8) {
        // The exponents of the next kAhead stages are on their way while one is widened.  The stages are unrolled so
        // that a register waits for its own load only (handing it on to another would wait at once).
        constexpr int kAhead = 4;
        static_assert(kPromote % kAhead == 0, "a part is whole rounds");
        const bool has = x.k0 + cq * 32 < p.K;
        const uint8_t* ex = p.x.exps + (x.first + crow) * nb + x.k0 / kPackBlock + cq;
        const int rows = (int)(x.last - x.first) - crow;  // rows of the chunk from this thread's first on
        const uint32_t ex_step = (uint32_t)(kBK * nb);
        uint32_t e[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) e[i] = has && i * kBK < rows ? (uint32_t)__ldg(ex + (size_t)i * ex_step) : 127u;
        for (int part = 0; part <= parts; ++part) {
          const int last_k = min((part + 1) * kPromote, x.stages);  // no stages are left for part = parts
#pragma unroll 1
          for (int k0 = part * kPromote; k0 < last_k; k0 += kAhead) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
              const int k = k0 + i;
              if (k >= last_k) break;
              const uint32_t byte = e[i];
              e[i] = has && (k + kAhead) * kBK < rows ? (uint32_t)__ldg(ex + (size_t)(k + kAhead) * ex_step) : 127u;
              // every warp goes through the barriers below, also after a wait ran out
              ok = __all_sync(kFull, tc::mbar_wait(&bar.full[s.stage], s.phase)) && ok;
              uint8_t* st = ring + s.stage * R::kStage;
              uint4 q[2];
#pragma unroll
              for (int j = 0; j < 2; ++j)
                q[j] = *reinterpret_cast<const uint4*>(st + crow * 128 + cq * 32 + ((j ^ (cq >> 1)) << 4));
              asm volatile("bar.sync 1, 256;" ::: "memory");  // the codes are in registers: their place may be written
              // 2^e as bf16, twice; bf16 holds every exponent a checkpoint has
              const uint32_t scale = byte == kPackNan ? 0x7FC07FC0u : (byte << 7) * 0x00010001u;
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const uint32_t w[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint4 o = make_uint4(tc::codes_bf16x2(w[2 * h], 0, scale), tc::codes_bf16x2(w[2 * h], 1, scale),
                                             tc::codes_bf16x2(w[2 * h + 1], 0, scale), tc::codes_bf16x2(w[2 * h + 1], 1, scale));
                  const int c = (cq & 1) * 4 + (j ^ (cq >> 1)) * 2 + h;  // piece of the row's 128 bytes
                  *reinterpret_cast<uint4*>(st + (cq >> 1) * 8192 + crow * 128 + ((c ^ (crow & 7)) << 4)) = o;
                }
              }
              tc::fence_async_proxy();
              __syncwarp();
              if (lane == 0) tc::mbar_arrive(&bar.wide[s.stage]);
              s.next<R::kStages>();
            }
          }
          // the part before this one: its products are done or nearly so, and this part's go on meanwhile
          if (part > 0 && ok) read_out();
        }
      } else {
        for (int part = 0; part < parts && ok; ++part) read_out();
      }
      if (!ok) break;
      // sum[j]: dW at column k0 + 32 quad + lane and row m0 + half kCols + j: 32 lanes write 128 bytes of a row
      const int k = x.k0 + quad * 32 + lane, m0 = x.m0 + half * kCols;
      float* out = weights_out(p, s_cum, s_slot, x.g, x.c) + (size_t)m0 * p.K + k;
      size_t ld = p.K;
      asm volatile("" : "+l"(ld));  // keeps the compiler from holding a register per row's offset across the tiles
      if (k < p.K) {
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
          if (m0 + j < p.M) *out = sum[j];
          out += ld;
        }
      }
      __syncwarp();
    }
    if (!ok) latch_status(p.status, MT_ECUDA);
  }
  tc_end<BN>(tmem);
}

// ---- host --------------------------------------------------------------------------------------------

// Tile width of a product with J columns and `rows` row tiles: the widest that leaves no half of a tile idle and
// still gives every SM a tile.
int tile_width(int J, long long row_tiles) {
  int bn = J <= 64 ? 64 : (J <= 128 || (J % 256 != 0 && J % 256 <= 128 && J < 512) ? 128 : 256);
  while (bn > 64 && row_tiles * ((J + bn - 1) / bn) < sm_count()) bn >>= 1;
  return bn;
}

template <typename Kernel>
cudaError_t allow_smem(Kernel k, size_t bytes) {
  return cudaFuncSetAttribute(reinterpret_cast<const void*>(k), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <int BN, bool B_MN>
cudaError_t rows_tc(const CUtensorMap& a, const CUtensorMap& w, LinearRows p, cudaStream_t s) {
  const size_t smem = 1024 + Ring<BN>::kBytes + (size_t)(p.groups + 1) * 12;
  cudaError_t e = allow_smem(k_linear_rows_tc<BN, B_MN>, smem);
  if (e != cudaSuccess) return e;
  p.jtiles = (p.J + BN - 1) / BN;
  const long long tiles = ((p.n + kBM - 1) / kBM + p.groups) * p.jtiles;
  const int grid = (int)std::min<long long>(tiles, sm_count());
  MT_LAUNCH("k_linear_rows_tc", s);
  k_linear_rows_tc<BN, B_MN><<<grid, kWarpsTC * 32, smem, s>>>(a, w, p);
  return cudaGetLastError();
}

template <int BN, bool X8>
cudaError_t weights_tc(const CUtensorMap& x, const CUtensorMap& dy, const LinearWeights& p, cudaStream_t s) {
  const size_t smem = 1024 + Ring<BN>::kStages * Ring<BN>::kStage + weights_smem(p.groups);
  cudaError_t e = allow_smem(k_linear_weights_tc<BN, X8>, smem);
  if (e != cudaSuccess) return e;
  if (BN == 256) {  // the split of the registers needs the launch to bring them
    cudaFuncAttributes a;
    e = cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(k_linear_weights_tc<BN, X8>));
    if (e != cudaSuccess) return e;
    if (a.numRegs < kRegsLaunch) return cudaErrorInvalidValue;
  }
  const long long tiles = (p.n / p.chunk + p.groups) * ((p.K + kBM - 1) / kBM) * ((p.M + BN - 1) / BN);
  const int grid = (int)std::min<long long>(tiles, sm_count());
  MT_LAUNCH("k_linear_weights_tc", s);
  k_linear_weights_tc<BN, X8><<<grid, kWarpsW * 32, smem, s>>>(x, dy, p);
  return cudaGetLastError();
}

}  // namespace

bool linear_rows_fits_tc(const LinearRows& p) {
  return p.I % 8 == 0 && p.J % 8 == 0 && p.lda % 8 == 0 && p.ldc % 8 == 0 && is_aligned(p.a, 16) && is_aligned(p.c, 16) &&
         is_aligned(p.w, 16);
}

cudaError_t launch_linear_rows_tc(const LinearRows& p, cudaStream_t s) {
  const bool b_mn = p.wj == 1 && p.wi != 1;
  const int bn = tile_width(p.J, (p.n + kBM - 1) / kBM + p.groups - 1);
  CUtensorMap a, w;
  if (!tc::encode_bf16(&a, 2, p.a, p.I, p.n, p.lda, 1, 0, kBK, kBM)) return cudaErrorInvalidValue;
  if (b_mn ? !tc::encode_bf16(&w, 3, p.w, p.J, p.I, p.J, p.groups, (uint64_t)p.I * p.J, 64, kBK)
           : !tc::encode_bf16(&w, 3, p.w, p.I, p.J, p.I, p.groups, (uint64_t)p.I * p.J, kBK, bn))
    return cudaErrorInvalidValue;
  if (b_mn) return bn == 256 ? rows_tc<256, true>(a, w, p, s) : bn == 128 ? rows_tc<128, true>(a, w, p, s) : rows_tc<64, true>(a, w, p, s);
  return bn == 256 ? rows_tc<256, false>(a, w, p, s) : bn == 128 ? rows_tc<128, false>(a, w, p, s) : rows_tc<64, false>(a, w, p, s);
}

// 8-bit x lands by byte copies whose rows lie K bytes apart: K has to be a multiple of 16 there.
bool linear_weights_fits_tc(const LinearWeights& p) {
  if (p.K % 8 != 0 || p.M % 8 != 0 || p.lddy % 8 != 0 || !is_aligned(p.dy, 16)) return false;
  if (p.x.data == nullptr) return p.K % 16 == 0 && is_aligned(p.x.codes, 16);
  return p.x.ld % 8 == 0 && is_aligned(p.x.data, 16);
}

cudaError_t launch_linear_weights_tc(const LinearWeights& p, cudaStream_t s) {
  const int bn = tile_width(p.M, (p.n / p.chunk + p.groups) * ((p.K + kBM - 1) / kBM));
  CUtensorMap dy, x;
  if (!tc::encode_bf16(&dy, 2, p.dy, p.M, p.n, p.lddy, 1, 0, 64, kBK)) return cudaErrorInvalidValue;
  if (p.x.data == nullptr) {
    if (!tc::encode_u8(&x, p.x.codes, p.K, p.n, p.K, kBM, kBK)) return cudaErrorInvalidValue;
    return bn == 256 ? weights_tc<256, true>(x, dy, p, s) : bn == 128 ? weights_tc<128, true>(x, dy, p, s)
                                                                      : weights_tc<64, true>(x, dy, p, s);
  }
  if (!tc::encode_bf16(&x, 2, p.x.data, p.K, p.n, p.x.ld, 1, 0, 64, kBK)) return cudaErrorInvalidValue;
  return bn == 256 ? weights_tc<256, false>(x, dy, p, s) : bn == 128 ? weights_tc<128, false>(x, dy, p, s)
                                                                     : weights_tc<64, false>(x, dy, p, s);
}

}  // namespace mt
