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
// measured, a sum over r rows of unit normal products has a relative error of
// 1.1e-9 * r (4.4e-6 at 4096 rows, where fp32 sums on the pipes have 2.5e-7).  dW
// is fp32 and sums over many rows, so its accumulator starts anew every kPromote
// stages and the read-out warps add it to registers, rounding to nearest: 4.9e-7
// at 700,000 rows, for 5% of the time of parts four times as long (65,536 x 1024
// x 1024, one group: 115 against 110 us).
//
// Bound: the arithmetic where the contraction is long, HBM where it is short.
// Measured, forward: 77,824 rows to 1024 columns 1.63 PFLOP/s from 1024 columns
// and 1.91 from 4096 (the library's product 1.79 and 1.93); 1,970,003 x 64 to 256
// 196 us, 95% of the copy bandwidth.  dx of 490,011 x 256 from 512 columns 121 us
// (91% of it).  dW of 65,536 x 1024 x 1024 in 8 groups: 123 us and 8 us of sums
// (1.12 PFLOP/s), from 8 bits 178 us, where the widening and one block's shared
// memory bound it.
#include <algorithm>

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

// Shared memory of a block: stages of both operands (of a pair's block: its half of the columns), and where the rows
// kernel turns its tiles.
template <int BN, int CG>
struct Ring {
  static constexpr int kStageA = kBM * kBK * 2, kStageB = BN / CG * kBK * 2;
  static constexpr int kStage = kStageA + kStageB;
  static constexpr int kStages = 196608 / kStage;       // 4 (BN 256), 6 (128, and 256 of a pair), 8 (64)
  static constexpr int kBytes = kStages * kStage + 4 * kStageOut;
};

struct Barriers {
  uint64_t full[8], empty[8];    // a stage's copies have landed; its products are done
  uint64_t ready[8];             // a stage's 8-bit operand has been widened
  // The second block of a pair, in a chunk's last, short stage: its copies have landed; their rows past the end are
  // zeroed.  One per stage, as the others: the short stages of several small chunks can be on their way at once.
  uint64_t tail_full[8], tail_ready[8];
  uint64_t acc_full[2], acc_empty[2];  // an accumulator is finished; it has been read out
  uint64_t done;                 // every product issued is done
  volatile uint32_t copied;      // pairs: stages whose copies this block has started
  uint32_t tmem;
};

__device__ __forceinline__ void latch_status(int32_t* status, int code) {
  if (status != nullptr) atomicCAS(status, 0, code);
}

// Set-up that both kernels share: barriers, tensor memory.  Every thread calls it; ends with the block (the pair)
// synchronised.
template <int BN, int CG>
__device__ __forceinline__ uint32_t tc_begin(Barriers& b, int ready_count, int read_warps) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < Ring<BN, CG>::kStages; ++i) {
      tc::mbar_init(&b.full[i], 1);
      tc::mbar_init(&b.empty[i], 1);
      tc::mbar_init(&b.ready[i], ready_count);
      tc::mbar_init(&b.tail_full[i], 1);
      tc::mbar_init(&b.tail_ready[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&b.acc_full[i], 1);
      tc::mbar_init(&b.acc_empty[i], read_warps * CG);
    }
    tc::mbar_init(&b.done, 1);
    b.copied = 0;
    tc::mbar_init_fence();
  }
  __syncwarp();
  if (threadIdx.x >> 5 == 1) tc::tmem_alloc<CG>(&b.tmem, 2 * BN);
  tc::fence_before();
  if constexpr (CG == 2) tc::cluster_sync();
  else __syncthreads();
  tc::fence_after();
  return b.tmem;
}

template <int BN, int CG>
__device__ __forceinline__ void tc_end(uint32_t tmem) {
  __syncwarp();
  tc::fence_before();
  if constexpr (CG == 2) tc::cluster_sync();
  else __syncthreads();
  tc::fence_after();
  if (threadIdx.x >> 5 == 1) tc::tmem_free<CG>(tmem, 2 * BN);
}

// Arrives at a barrier of the block that issues the products.
template <int CG>
__device__ __forceinline__ void arrive(uint64_t* bar) {
  if constexpr (CG == 2) tc::mbar_arrive_at(tc::of_leader(bar));
  else tc::mbar_arrive(bar);
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

// The last stages' products are done, and what a pair's first block signals of them has arrived here.
template <int STAGES>
__device__ __forceinline__ bool all_released(Barriers& b, Slot s, long long issued) {
  const long long k = issued < STAGES ? issued : STAGES;
  for (long long i = 0; i < k; ++i) {
    if (s.stage == 0) {
      s.stage = STAGES;
      s.phase ^= 1;
    }
    --s.stage;
    if (!tc::mbar_wait(&b.empty[s.stage], s.phase)) return false;
  }
  return true;
}

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
// CG = 2: a pair of blocks takes 256 rows, each its 128 and half of the tile's columns of W: a block then writes and
// reads 64 KB of shared memory per stage instead of 96, which at 128 bytes a clock is what the tensor core's 512 clocks
// allow (one block alone is bound by its shared memory: 768 clocks).
template <int BN, bool B_MN, int CG>
__global__ void __launch_bounds__(kWarpsTC * 32, 1)
k_linear_rows_tc(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w, const LinearRows p) {
  using R = Ring<BN, CG>;
  constexpr int kRows = kBM * CG, kCols = BN / CG;  // rows of a tile; columns of W that a block copies
  extern __shared__ uint8_t s_raw[];
  __shared__ Barriers bar;
  uint8_t* ring = reinterpret_cast<uint8_t*>(((uintptr_t)s_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* s_out = ring + R::kStages * R::kStage;
  long long* s_off = reinterpret_cast<long long*>(ring + R::kBytes);
  int* s_cum = reinterpret_cast<int*>(s_off + p.groups + 1);
  load_offsets(p.offsets, p.groups, p.n, s_off, p.status);
  count_tiles(s_off, p.groups, kRows, s_cum);
  const uint32_t tmem = tc_begin<BN, CG>(bar, 1, 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % CG;  // in the pair
  const int steps = (p.I + kBK - 1) / kBK;
  const long long total = (long long)s_cum[p.groups] * p.jtiles;
  const long long t0 = blockIdx.x / CG, tstep = gridDim.x / CG;

  if (warp == 0) {
    if (lane == 0) {
      Slot s;
      long long issued = 0;
      bool ok = true;
      for (long long t = t0; t < total && ok; t += tstep) {
        const int rt = (int)(t / p.jtiles), j0 = (int)(t - (long long)rt * p.jtiles) * BN + rank * kCols;
        const int g = tile_group(s_cum, p.groups, rt);
        const int r0 = (int)(s_off[g] + (long long)(rt - s_cum[g]) * kRows) + rank * kBM;
        for (int k = 0; k < steps; ++k) {
          ok = tc::mbar_wait(&bar.empty[s.stage], s.phase ^ 1);
          if (!ok) break;
          uint8_t* st = ring + s.stage * R::kStage;
          if constexpr (CG == 2) {  // both blocks' copies count on the first block's barrier
            const uint32_t full = tc::of_leader(&bar.full[s.stage]);
            if (rank == 0) tc::mbar_expect(&bar.full[s.stage], 2 * R::kStage);
            tc::tma_load_2d_pair(st, &map_a, full, k * kBK, r0);
            if constexpr (B_MN) {
#pragma unroll
              for (int c = 0; c < kCols / 64; ++c)
                tc::tma_load_3d_pair(st + R::kStageA + c * 8192, &map_w, full, j0 + c * 64, k * kBK, g);
            } else {
              tc::tma_load_3d_pair(st + R::kStageA, &map_w, full, k * kBK, j0, g);
            }
          } else {
            tc::mbar_expect(&bar.full[s.stage], R::kStage);
            tc::tma_load_2d(st, &map_a, &bar.full[s.stage], k * kBK, r0);
            if constexpr (B_MN) {
#pragma unroll
              for (int c = 0; c < kCols / 64; ++c)
                tc::tma_load_3d(st + R::kStageA + c * 8192, &map_w, &bar.full[s.stage], j0 + c * 64, k * kBK, g);
            } else {
              tc::tma_load_3d(st + R::kStageA, &map_w, &bar.full[s.stage], k * kBK, j0, g);
            }
          }
          ++issued;
          s.next<R::kStages>();
        }
      }
      ok = ok && all_released<R::kStages>(bar, s, issued);
      // what the first block signals of its last products has to have arrived here before this block ends
      if (rank != 0) ok = tc::mbar_wait(&bar.done, 0) && ok;
      if (!ok) {
        latch_status(p.status, MT_ECUDA);
        if (rank == 0) drain<R::kStages>(bar, s, issued);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      constexpr uint32_t instr = tc::instr_bf16(kRows, BN, false, B_MN);
      Slot s;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (long long t = t0; t < total && ok; t += tstep) {
        ok = tc::mbar_wait(&bar.acc_empty[acc], acc_phase ^ 1);
        if (!ok) break;
        tc::fence_after();
        for (int k = 0; k < steps; ++k) {
          ok = tc::mbar_wait<CG == 2>(&bar.full[s.stage], s.phase);  // a pair's copies into both blocks
          if (!ok) break;
          tc::fence_after();
          const uint32_t a = tc::smem_addr(ring + s.stage * R::kStage), b = a + R::kStageA;
#pragma unroll
          for (int i = 0; i < kBK / 16; ++i) {
            const uint64_t da = tc::smem_desc(a + i * 32, 16);
            const uint64_t db = B_MN ? tc::smem_desc(b + i * 2048, 8192) : tc::smem_desc(b + i * 32, 16);
            tc::mma_bf16<CG>(tmem + acc * BN, da, db, instr, k > 0 || i > 0);
          }
          tc::mma_commit<CG>(&bar.empty[s.stage]);
          s.next<R::kStages>();
        }
        if (!ok) break;
        tc::mma_commit<CG>(&bar.acc_full[acc]);
        acc ^= 1;
        acc_phase ^= acc == 0;
      }
      tc::mma_commit<CG>(&bar.done);  // tensor memory is freed only when no product writes it, also after a wait ran out
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
    for (long long t = t0; t < total; t += tstep) {
      const int rt = (int)(t / p.jtiles), j0 = (int)(t - (long long)rt * p.jtiles) * BN;
      const int g = tile_group(s_cum, p.groups, rt);
      const long long r0 = s_off[g] + (long long)(rt - s_cum[g]) * kRows + rank * kBM + quad * 32;
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
          if (lane == 0) arrive<CG>(&bar.acc_empty[acc]);
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
  tc_end<BN, CG>(tmem);
}

// ---- dW -----------------------------------------------------------------------------------------

constexpr int kPromote = 8;   // stages (of kBK rows) an accumulator sums before it is added to registers
constexpr int kReadWarps = 8;
constexpr int kWarpsW = 4 + kReadWarps;  // a warpgroup for copies and products (two of its warps idle), two to read out
// A read-out thread of the widest tile holds 128 sums beside its loads: the block's registers (384 threads x 168 at
// launch = 64512) are split anew, 72 for a control thread and 216 for a read-out thread (128 x 72 + 256 x 216 = 64512).
constexpr int kRegsLaunch = 168, kRegsControl = 72, kRegsRead = 216;
static_assert(128 * kRegsControl + 32 * kReadWarps * kRegsRead <= kWarpsW * 32 * kRegsLaunch, "the split fits the launch");

// Rows [left, kBK) of `slabs` slabs become zero, by a warp.  Row i of a 64-column slab is the 128 bytes at i * 128,
// whatever the swizzle does inside them.
__device__ __forceinline__ void zero_rows(uint8_t* st, int slabs, int left, int lane) {
  for (int slab = 0; slab < slabs; ++slab)
    for (int i = left * 8 + lane; i < kBK * 8; i += 32)
      *reinterpret_cast<uint4*>(st + slab * 8192 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
  tc::fence_async_proxy();
  __syncwarp();
}

// CG = 2: a pair takes 256 columns of x, each block its 128 and half of the tile's columns of dy (the split of
// k_linear_rows_tc, for the same reason).  Plain x only: the second block's widened rows would be ordinary writes that the
// first block's products read, so each stage would have to be handed over across the pair, 1.4 us at a time.  490,011 x 256 x
// 512 from 8 bits, whole calls: the hand-overs dealt over three warps 179 us, one warp's 289, by the widening warps 260;
// single blocks 171.
template <int BN, bool X8, int CG>
__global__ void __launch_bounds__(kWarpsW * 32, 1)
k_linear_weights_tc(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_dy, const LinearWeights p) {
  using R = Ring<BN, CG>;
  constexpr int kRowsD = kBM * CG, kColsB = BN / CG;  // columns of x in a tile; columns of dy that a block copies
  extern __shared__ uint8_t s_raw[];
  __shared__ Barriers bar;
  uint8_t* ring = reinterpret_cast<uint8_t*>(((uintptr_t)s_raw + 1023) & ~(uintptr_t)1023);
  long long* s_off = reinterpret_cast<long long*>(ring + R::kStages * R::kStage);
  __shared__ ChunkChoice s_choice;
  load_offsets(p.offsets, p.groups, p.n, s_off, p.status);
  const Plan plan = plan_in(s_off, p.groups);
  plan_chunks(p, plan, s_choice);
  const uint32_t tmem = tc_begin<BN, CG>(bar, kReadWarps / 2, kReadWarps);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % CG;
  const int mt = (p.M + BN - 1) / BN, tiles = (p.K + kRowsD - 1) / kRowsD * mt;
  const long long total = (long long)plan.ocum[p.groups] * tiles;
  const int unit = blockIdx.x / CG, units = gridDim.x / CG;

  // a tile: its chunk and dW's corner (m0, k0 of this block)
  struct Tile : Chunk {
    int m0, k0, stages;
  };
  auto tile_of = [&](long long t) {
    const int c = (int)(t / tiles), q = (int)(t - (long long)c * tiles);
    Tile x;
    static_cast<Chunk&>(x) = chunk_of(plan, p.groups, c);
    x.k0 = q / mt * kRowsD + rank * kBM;
    x.m0 = (q - q / mt * mt) * BN;
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
        for (long long r0 = 0; r0 * units < total && ok; ++r0) {
          const long long t = dealt(r0, unit, units);
          if (t >= total) continue;
          const Tile x = tile_of(t);
          for (long long r = x.first; r < x.last; r += kBK) {
            ok = tc::mbar_wait(&bar.empty[s.stage], s.phase ^ 1);
            if (!ok) break;
            uint8_t* st = ring + s.stage * R::kStage;
            const int dy0 = x.m0 + rank * kColsB;
            if (CG == 2 && x.last - r >= kBK) {  // both blocks' copies count on the first block's barrier
              const uint32_t full = tc::of_leader(&bar.full[s.stage]);
              if (rank == 0) tc::mbar_expect(&bar.full[s.stage], 2 * bytes);
#pragma unroll
              for (int c = 0; c < kBM / 64; ++c) tc::tma_load_2d_pair(st + c * 8192, &map_x, full, x.k0 + c * 64, (int)r);
#pragma unroll
              for (int c = 0; c < kColsB / 64; ++c)
                tc::tma_load_2d_pair(st + R::kStageA + c * 8192, &map_dy, full, dy0 + c * 64, (int)r);
            } else {
              uint64_t* full = rank != 0 ? &bar.tail_full[s.stage] : &bar.full[s.stage];
              tc::mbar_expect(full, bytes);
              if constexpr (X8) {
                tc::tma_load_2d(st, &map_x, full, x.k0, (int)r);
              } else {
#pragma unroll
                for (int c = 0; c < kBM / 64; ++c) tc::tma_load_2d(st + c * 8192, &map_x, full, x.k0 + c * 64, (int)r);
              }
#pragma unroll
              for (int c = 0; c < kColsB / 64; ++c)
                tc::tma_load_2d(st + R::kStageA + c * 8192, &map_dy, full, dy0 + c * 64, (int)r);
            }
            ++issued;
            if (CG == 2) bar.copied = (uint32_t)issued;
            s.next<R::kStages>();
          }
        }
        ok = ok && all_released<R::kStages>(bar, s, issued);
        if (rank != 0) ok = tc::mbar_wait(&bar.done, 0) && ok;  // as in k_linear_rows_tc
        if (!ok) {
          latch_status(p.status, MT_ECUDA);
          if (rank == 0) drain<R::kStages>(bar, s, issued);
        }
      }
    }
    // Plain x: the rows past the chunk's end in its last stage belong to others; warp 1 zeroes them in both operands, so
    // that nothing of them (an infinity or NaN too) reaches the sum.  The second block of a pair does so for its own
    // copies, which count on a barrier of its own in that stage, and hands them over to the first.  8-bit x: the widening
    // warps do it.
    if (warp == 1) {
      constexpr uint32_t instr = tc::instr_bf16(kRowsD, BN, true, true);
      Slot s;
      int acc = 0;
      uint32_t acc_phase = 0, tail_phase = 0;  // tail_phase: a bit per stage
      bool ok = true;
      if (rank != 0) {
        uint32_t seq = 0;  // stages before this tile
        for (long long r0 = 0; r0 * units < total && ok; ++r0) {
          const long long t = dealt(r0, unit, units);
          if (t >= total) continue;
          const Tile x = tile_of(t);
          const int left = (int)(x.last - x.first) & (kBK - 1);
          seq += x.stages;
          if (left == 0) continue;
          const uint32_t stage = (seq - 1) % R::kStages;
          // a whole chunk may lie between two short stages
          ok = __all_sync(kFull, tc::mbar_wait_while(&bar.tail_full[stage], tail_phase >> stage & 1, &bar.copied));
          if (!ok) break;
          tail_phase ^= 1u << stage;
          zero_rows(ring + stage * R::kStage, (kBM + kColsB) / 64, left, lane);
          if (lane == 0) tc::mbar_hand_over_at(tc::of_leader(&bar.tail_ready[stage]));
        }
      }
      for (long long r0 = 0; rank == 0 && r0 * units < total && ok; ++r0) {
        const long long t = dealt(r0, unit, units);
        if (t >= total) continue;
        const Tile x = tile_of(t);
        for (int k = 0; k < x.stages; ++k) {
          if (k % kPromote == 0) {
            ok = __all_sync(kFull, tc::mbar_wait(&bar.acc_empty[acc], acc_phase ^ 1));
            if (!ok) break;
          }
          uint8_t* st = ring + s.stage * R::kStage;
          ok = __all_sync(kFull, tc::mbar_wait<CG == 2>(X8 ? &bar.ready[s.stage] : &bar.full[s.stage], s.phase));
          if (!ok) break;
          const int left = (int)min((long long)kBK, x.last - x.first - (long long)k * kBK);
          if (!X8 && left < kBK) {
            zero_rows(st, (kBM + kColsB) / 64, left, lane);
            if constexpr (CG == 2) {
              ok = __all_sync(kFull, tc::mbar_wait<true>(&bar.tail_ready[s.stage], tail_phase >> s.stage & 1));
              if (!ok) break;
              tail_phase ^= 1u << s.stage;
            }
          }
          tc::fence_after();
          const bool closes = k % kPromote == kPromote - 1 || k + 1 == x.stages;
          if (lane == 0) {
            const uint32_t a = tc::smem_addr(st), b = a + R::kStageA;
#pragma unroll
            for (int i = 0; i < kBK / 16; ++i)
              tc::mma_bf16<CG>(tmem + acc * BN, tc::smem_desc(a + i * 2048, 8192), tc::smem_desc(b + i * 2048, 8192), instr,
                               k % kPromote > 0 || i > 0);
            tc::mma_commit<CG>(&bar.empty[s.stage]);
            if (closes) tc::mma_commit<CG>(&bar.acc_full[acc]);
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
        // tensor memory is freed only when no product writes it, also after a wait ran out
        if (rank == 0) {
          tc::mma_commit<CG>(&bar.done);
          ok = tc::mbar_wait(&bar.done, 0) && ok;
        }
        if (!ok) latch_status(p.status, MT_ECUDA);
      }
    }
  } else {
    if constexpr (BN == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsRead));
    // a warp reads the 32 lanes (columns of x) that its number allows and half of the columns (of dy)
    constexpr int kCols = BN / 2;
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const uint32_t from = tmem + half * kCols + ((uint32_t)(quad * 32) << 16);
    const int nb = (p.K + kPackBlock - 1) / kPackBlock;
    int acc = 0;
    uint32_t acc_phase = 0;
    uint32_t seq = 0;  // stages before this tile
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
      if (lane == 0) arrive<CG>(&bar.acc_empty[acc]);
      acc ^= 1;
      acc_phase ^= acc == 0;
    };

    for (long long r0 = 0; r0 * units < total && ok; ++r0) {
      const long long t = dealt(r0, unit, units);
      if (t >= total) continue;
      // what outlives the tile's stages is kept few: the registers go to the sums
      float* out;
      int stages, m_left, len;
      bool k_in;
      int kb;
      const uint8_t* ex = nullptr;
      {
        const Tile x = tile_of(t);
        stages = x.stages;
        len = (int)(x.last - x.first);
        const int k = x.k0 + quad * 32 + lane, m0 = x.m0 + half * kCols;
        m_left = p.M - m0;
        k_in = k < p.K;
        out = weights_out(p, plan, x) + (size_t)m0 * p.K + k;
        if constexpr (X8) ex = p.x.exps + row_offset(x.first + ((threadIdx.x & 127) >> 1), nb) + x.k0 / kPackBlock + (threadIdx.x & 1) * 2;
        kb = x.k0 / kPackBlock + (threadIdx.x & 1) * 2;
      }
      const int parts = (stages + kPromote - 1) / kPromote;
#pragma unroll
      for (int j = 0; j < kCols; ++j) sum[j] = 0.0f;
      if constexpr (X8) {
        // Two teams of four warps widen alternate stages, so that one's barriers and fences overlap the other's work: a
        // thread takes a row and 64 columns (two blocks) of a stage.  The exponents of a thread's next four stages are on
        // their way while it works; the stages are unrolled so that a register waits for its own load only.
        constexpr int kOwn = kPromote / 2;
        const int tid = threadIdx.x & 127, crow = tid >> 1, ch = tid & 1;
        const int off = (half + seq) & 1;                 // this team's first stage of the tile
        const int rows = len - crow;  // rows of the chunk from this thread's first on
        const bool has0 = kb < nb, has1 = kb + 1 < nb;
        const uint32_t ex_step = (uint32_t)(kBK * nb);
        uint32_t e0[kOwn], e1[kOwn];
        auto exponents = [&](int i, int k) {
          const bool in = k * kBK < rows;
          e0[i] = in && has0 ? (uint32_t)__ldg(ex + (size_t)k * ex_step) : 127u;
          e1[i] = in && has1 ? (uint32_t)__ldg(ex + (size_t)k * ex_step + 1) : 127u;
        };
#pragma unroll
        for (int i = 0; i < kOwn; ++i) exponents(i, off + 2 * i);
        for (int part = 0; part <= parts; ++part) {
#pragma unroll
          for (int i = 0; i < kOwn; ++i) {
            const int k = part * kPromote + off + 2 * i;
            if (k >= stages) break;  // always for part = parts
            const uint32_t b0 = e0[i], b1 = e1[i];
            exponents(i, k + kPromote);
            const uint32_t stage = (seq + k) % R::kStages, phase = (seq + k) / R::kStages & 1;
            // every warp goes through the barriers below, also after a wait ran out (it then waits no more)
            if (ok) ok = __all_sync(kFull, tc::mbar_wait(&bar.full[stage], phase));
            uint8_t* st = ring + stage * R::kStage;
            uint4 q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)  // pieces in an order that spreads eight lanes over the banks
              q[j] = *reinterpret_cast<const uint4*>(st + crow * 128 + ch * 64 + (((j + (lane >> 1)) & 3) << 4));
            if (half == 0) asm volatile("bar.sync 1, 128;" ::: "memory");  // the codes are in registers: their place
            else asm volatile("bar.sync 2, 128;" ::: "memory");            // may be written
            const bool in = k * kBK < rows;  // past the chunk's end: zeros, in both operands
            // 2^e as bf16, twice; bf16 holds every exponent a checkpoint has
            const uint32_t s0 = b0 == kPackNan ? 0x7FC07FC0u : (b0 << 7) * 0x00010001u;
            const uint32_t s1 = b1 == kPackNan ? 0x7FC07FC0u : (b1 << 7) * 0x00010001u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int piece = (j + (lane >> 1)) & 3;  // 16 codes: two 16-byte pieces of the slab's row
              const uint32_t scale = piece < 2 ? s0 : s1;
              const uint32_t w[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint4 o = make_uint4(tc::codes_bf16x2(w[2 * h], 0, scale), tc::codes_bf16x2(w[2 * h], 1, scale),
                                     tc::codes_bf16x2(w[2 * h + 1], 0, scale), tc::codes_bf16x2(w[2 * h + 1], 1, scale));
                if (!in) o = make_uint4(0u, 0u, 0u, 0u);
                *reinterpret_cast<uint4*>(st + ch * 8192 + crow * 128 + (((piece * 2 + h) ^ (crow & 7)) << 4)) = o;
              }
            }
            if (!in) {
              for (int slab = 0; slab < kColsB / 64; ++slab)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  *reinterpret_cast<uint4*>(st + R::kStageA + slab * 8192 + crow * 128 + ch * 64 + c * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            tc::fence_async_proxy();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bar.ready[stage]);
          }
          // the part before this one: its products are done or nearly so, and this part's go on meanwhile
          if (part > 0 && ok) read_out();
        }
        seq += stages;
      } else {
        for (int part = 0; part < parts && ok; ++part) read_out();
      }
      if (!ok) break;
      // sum[j]: dW at column k0 + 32 quad + lane and row m0 + half kCols + j: 32 lanes write 128 bytes of a row
      size_t ld = p.K;
      asm volatile("" : "+l"(ld));  // keeps the compiler from holding a register per row's offset across the tiles
      if (k_in) {
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
          if (j < m_left) *out = sum[j];
          out += ld;
        }
      }
      __syncwarp();
    }
    if (!ok) latch_status(p.status, MT_ECUDA);
  }
  tc_end<BN, CG>(tmem);
}

// ---- host --------------------------------------------------------------------------------------------

// Tile width of a product with J columns and `row_tiles` row tiles: the widest that leaves no half of a tile idle and
// still gives every SM a tile.
int tile_width(int J, long long row_tiles) {
  int bn = J <= 64 ? 64 : (J <= 128 || (J % 256 != 0 && J % 256 <= 128 && J < 512) ? 128 : 256);
  while (bn > 64 && row_tiles * ((J + bn - 1) / bn) < sm_count()) bn >>= 1;
  return bn;
}

// Launches a kernel in clusters of `pair` blocks.
template <typename Kernel, typename Params>
cudaError_t launch_tc(Kernel kernel, int grid, int threads, size_t smem, int pair, cudaStream_t s, const CUtensorMap& a,
                      const CUtensorMap& b, const Params& p) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = pair;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pair > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a, b, p);
}

int tc_grid(long long tiles, int pair) { return (int)std::min<long long>(tiles, sm_count() / pair) * pair; }

template <int BN, bool B_MN, int CG>
cudaError_t rows_tc(const CUtensorMap& a, const CUtensorMap& w, LinearRows p, cudaStream_t s) {
  p.jtiles = (p.J + BN - 1) / BN;
  const long long tiles = (p.n / (kBM * CG) + p.groups) * p.jtiles;
  constexpr size_t ring = 1024 + Ring<BN, CG>::kBytes;  // the stages start on 1024 bytes
  static SmemLimit limit;
  const cudaError_t e = limit.allow(k_linear_rows_tc<BN, B_MN, CG>, ring + rows_smem(MT_MAX_GROUPS));
  if (e != cudaSuccess) return e;
  MT_LAUNCH("k_linear_rows_tc", s);
  return launch_tc(k_linear_rows_tc<BN, B_MN, CG>, tc_grid(tiles, CG), kWarpsTC * 32, ring + rows_smem(p.groups), CG, s, a, w, p);
}

template <int BN, bool X8, int CG>
cudaError_t weights_tc(const CUtensorMap& x, const CUtensorMap& dy, const LinearWeights& p, cudaStream_t s) {
  if (BN == 256) {  // the split of the registers needs the launch to bring them
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(k_linear_weights_tc<BN, X8, CG>));
    if (e != cudaSuccess) return e;
    if (a.numRegs < kRegsLaunch) return cudaErrorInvalidValue;
  }
  constexpr size_t ring = 1024 + Ring<BN, CG>::kStages * Ring<BN, CG>::kStage;
  static SmemLimit limit;
  const cudaError_t e = limit.allow(k_linear_weights_tc<BN, X8, CG>, ring + weights_smem(MT_MAX_GROUPS));
  if (e != cudaSuccess) return e;
  MT_LAUNCH("k_linear_weights_tc", s);
  return launch_tc(k_linear_weights_tc<BN, X8, CG>, weights_blocks(p) * CG, kWarpsW * 32, ring + weights_smem(p.groups), CG, s, x, dy, p);
}

template <bool X8>
cudaError_t weights_tc(const CUtensorMap& x, const CUtensorMap& dy, const LinearWeights& p, int bn, bool pair, cudaStream_t s) {
  if constexpr (!X8) {
    if (pair) return weights_tc<256, X8, 2>(x, dy, p, s);
  }
  return bn == 256 ? weights_tc<256, X8, 1>(x, dy, p, s) : bn == 128 ? weights_tc<128, X8, 1>(x, dy, p, s)
                                                                     : weights_tc<64, X8, 1>(x, dy, p, s);
}

}  // namespace

bool linear_rows_fits_tc(const LinearRows& p) {
  return p.I % 8 == 0 && p.J % 8 == 0 && p.lda % 8 == 0 && p.ldc % 8 == 0 && is_aligned(p.a, 16) && is_aligned(p.c, 16) &&
         is_aligned(p.w, 16);
}

// Pairs where the product is bound by its arithmetic, and tiles of 256 rows neither waste rows nor leave SMs without work.
// Measured, single blocks against pairs: one column tile (491,520 rows to 256 columns) from 256 columns 84 against 96 us,
// 384 106 against 109, 448 117 against 108, 512 127 against 117; several (327,680 to 512) from 128 74 against 74, 192 87
// against 83, 256 94 against 88.  Rows per group (65,536 x 1024 to 1024): 512 118 against 114, 256 144 against 141, 128
// 208 against 210; in 32 groups 103 against 93.
cudaError_t launch_linear_rows_tc(const LinearRows& p, cudaStream_t s) {
  const bool b_mn = p.wj == 1 && p.wi != 1;
  const int bn = tile_width(p.J, (p.n + kBM - 1) / kBM + p.groups - 1);
  const bool pair = bn == 256 && p.I > (p.J > 256 ? 2 : 6) * kBK && p.n / p.groups >= 256 && p.n / 256 * ((p.J + 255) / 256) >= sm_count() / 2;
  CUtensorMap a, w;
  if (!tc::encode_bf16(&a, 2, p.a, p.I, p.n, p.lda, 1, 0, kBK, kBM)) return cudaErrorInvalidValue;
  if (b_mn ? !tc::encode_bf16(&w, 3, p.w, p.J, p.I, p.J, p.groups, (uint64_t)p.I * p.J, 64, kBK)
           : !tc::encode_bf16(&w, 3, p.w, p.I, p.J, p.I, p.groups, (uint64_t)p.I * p.J, kBK, pair ? 128 : bn))
    return cudaErrorInvalidValue;
  if (pair) return b_mn ? rows_tc<256, true, 2>(a, w, p, s) : rows_tc<256, false, 2>(a, w, p, s);
  if (b_mn)
    return bn == 256 ? rows_tc<256, true, 1>(a, w, p, s) : bn == 128 ? rows_tc<128, true, 1>(a, w, p, s) : rows_tc<64, true, 1>(a, w, p, s);
  return bn == 256 ? rows_tc<256, false, 1>(a, w, p, s) : bn == 128 ? rows_tc<128, false, 1>(a, w, p, s) : rows_tc<64, false, 1>(a, w, p, s);
}

// 8-bit x lands by byte copies whose rows lie K bytes apart: K has to be a multiple of 16 there.
bool linear_weights_fits_tc(const LinearWeights& p) {
  if (p.K % 8 != 0 || p.M % 8 != 0 || p.lddy % 8 != 0 || !is_aligned(p.dy, 16)) return false;
  if (p.x.data == nullptr) return p.K % 16 == 0 && is_aligned(p.x.codes, 16);
  return p.x.ld % 8 == 0 && is_aligned(p.x.data, 16);
}

Cut cut_of(int64_t n, int32_t groups, int32_t k, int32_t m, bool pairs) {
  // the tiles' width goes by the chunks that the rows may make
  const long long chunks = groups + n / 4096;
  Cut c;
  c.bn = tile_width(m, chunks * ((k + kBM - 1) / kBM));
  // Whole calls, single blocks against pairs: 114,468 x 728 x 720 124 against 116 us, 65,536 x 1024 x 1024 in 8 groups 127
  // against 127.
  c.pair = pairs && c.bn == 256 && k > kBM && n / 512 * ((k + 255) / 256) * ((m + 255) / 256) >= sm_count() / 2;
  const int across = c.pair ? 2 * kBM : kBM;
  c.tiles = ((k + across - 1) / across) * ((m + c.bn - 1) / c.bn);
  c.units = std::max(1, sm_count() / (c.pair ? 2 : 1));
  return c;
}

cudaError_t launch_linear_weights_tc(const LinearWeights& p, const Cut& cut, cudaStream_t s) {
  CUtensorMap dy, x;
  if (!tc::encode_bf16(&dy, 2, p.dy, p.M, p.n, p.lddy, 1, 0, 64, kBK)) return cudaErrorInvalidValue;
  if (p.x.data == nullptr) {
    if (!tc::encode_u8(&x, p.x.codes, p.K, p.n, p.K, kBM, kBK)) return cudaErrorInvalidValue;
    return weights_tc<true>(x, dy, p, cut.bn, cut.pair, s);
  }
  if (!tc::encode_bf16(&x, 2, p.x.data, p.K, p.n, p.x.ld, 1, 0, 64, kBK)) return cudaErrorInvalidValue;
  return weights_tc<false>(x, dy, p, cut.bn, cut.pair, s);
}

}  // namespace mt
