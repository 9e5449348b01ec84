// Tiles of a bf16 matrix product on the tensor cores whose epilogue is the
// operator: the loop that the gated feed-forward part (mt_gated.cu) and the
// losses over a vocabulary (mt_vocab*.cu) share.
//
// C(i, j) = sum over k of A(i, k) B(j, k), 128 rows i (256 by a pair of blocks)
// and BN columns j per tile.  One persistent block per SM walks the units that
// its operator deals out (a row tile and a run of column tiles); one thread
// keeps a ring of stages filled by TMA, one issues the products into one of two or
// four accumulators in tensor memory, and two teams of four warps hand finished tiles
// to the operator while the next tile's products run: half of a tile's columns each,
// which leaves the accumulator soonest (the losses: 214 to 190 us, see there), or
// (kTeams) every other tile each.
//
// Bound: by the products from 512 columns of contraction on (7373 rows x 100,003
// entries x 512: 400 to 450 us, 1.7 to 1.9 PFLOP/s, the clock held down by power);
// shorter ones by what their epilogue does with a tile.  All of a warp issues
// products and copies by an elected lane: by lane 0 four products took 690 clocks,
// so 512.
//
// An operand lies with its contraction contiguous, or with its rows contiguous
// (A_MN, B_MN).  fp32 operands come as three bf16 parts side by side whose sum
// is the value (24 bits in three times 8); a tile then sums the six products of
// parts that reach 2^-24 of the whole, the small ones first, since the tensor
// core cuts its accumulator off towards zero at every step and the error goes by
// the accumulator's size (per 16 products 1.1e-9 of it on average over values of
// either sign; up to 2^-23 where all have one sign and size).
#pragma once

#include "mt_block.cuh"
#include "mt_tc.cuh"

namespace mt {
namespace tiles {

constexpr int kBM = 128;        // tile rows of a block: the lanes of tensor memory
constexpr int kBK = 64;         // contraction per stage: one 128-byte swizzled row of bf16
constexpr int kEpiWarps = 8;    // two for each 32 lanes of tensor memory: two teams
constexpr int kWarps = 4 + kEpiWarps;  // copies, products, two idle, epilogue
constexpr int kThreadsT = kWarps * 32;
// Where an epilogue needs more registers than the launch gives a thread (Op::kSplit), the block's (384 threads x 168 at launch
// = 64512) are split anew: 72 for a thread of the first four warps and 216 for one of the epilogue (128 x 72 + 256 x 216).
constexpr int kRegsLaunch = 168, kRegsControl = 72, kRegsEpi = 216;
static_assert(128 * kRegsControl + kEpiWarps * 32 * kRegsEpi <= kThreadsT * kRegsLaunch, "the split fits the launch");

// Shared memory of a block: stages of both operands (of a pair's block: its half of the columns), and where the epilogue
// turns its rows.  KEEP: A's tile (all of its contraction, up to kKept steps) is copied once per unit and stays, and the
// stages hold B alone.
constexpr int kKept = 8;
template <int BN, int CG, bool KEEP, bool TRI>  // TRI: a stage holds all three parts of both operands
struct Ring {
  static constexpr int kStageA = kBM * kBK * 2, kStageB = BN / CG * kBK * 2;
  static constexpr int kParts = TRI ? 3 : 1;
  static constexpr int kStage = kParts * (kStageB + (KEEP ? 0 : kStageA));
  static constexpr int kTotal = 196608;
  static __host__ __device__ constexpr int stages(int kept) {
    const int n = (kTotal - kept * kStageA) / kStage;
    return n < 8 ? n : 8;
  }
};

struct Barriers {
  uint64_t full[8], empty[8];          // a stage's copies have landed; its products are done
  uint64_t acc_full[4], acc_empty[4];  // an accumulator is finished; it has been read out
  uint64_t a_full, a_empty;            // a unit's kept A has landed; its products are done
  uint64_t done;                       // every product issued is done
  uint32_t tmem;
};

// The parts that pass q of `passes` multiplies, the smallest products first: of one pass the only parts, of two A's two parts
// with B's only one, of six those of three.
__device__ __forceinline__ int part_a(int passes, int q) { return passes == 1 ? 0 : passes == 2 ? 1 - q : (0x010120 >> (4 * q)) & 3; }
__device__ __forceinline__ int part_b(int passes, int q) { return passes <= 2 ? 0 : (0x001102 >> (4 * q)) & 3; }

// A unit of work: a row tile, column tiles [ct0, ct1) one after the other, contraction steps [k0, k1) of each pass.
struct Unit {
  int row0;  // first row of the (pair's) tile
  int end;   // rows of the tile end here
  int g;     // group (third coordinate of B)
  int ct0, ct1;
  int k0, k1;
  int slot;  // the operator's
};

// A finished accumulator as an epilogue warp sees it: its 32 lanes.
struct Acc {
  uint32_t from;
  uint64_t* empty;
  bool live;  // false: the contraction is empty, everything is zero
  // 32 columns from c on; tc::tmem_load_wait() before they are used
  __device__ __forceinline__ void load(int c, uint32_t (&v)[32]) const { tc::tmem_load32(from + c, v); }
  // the same where the contraction may be empty
  __device__ __forceinline__ void load_or_zero(int c, uint32_t (&v)[32]) const {
    if (live) {
      tc::tmem_load32(from + c, v);
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = 0u;
    }
  }
  // every load is done: the accumulator may be written again
  template <int CG>
  __device__ __forceinline__ void release(int lane) const {
    if (!live) return;
    tc::fence_before();
    __syncwarp();
    if (lane == 0) tc::arrive<CG>(empty);
  }
};

// Steps of A (of all parts) that stay.
template <class Op>
__device__ __forceinline__ int kept_of(const typename Op::Params& p) {
  if constexpr (Op::kKeep) return p.kept;
  else return 0;
}

// Op: what is computed.
//   kBN, kAMN, kBMN            tile columns; operands whose rows are contiguous
//   kTeams                     a team of epilogue warps takes every other tile (else half of the columns of each)
//   kKeep                      A's tile stays for the unit: parts x steps <= kKept
//   kTri                       every stage brings three parts of A and of B (passes is 1) and makes their six products
//   kTwoB                      (where B's contraction is contiguous) half of the columns b_second rows of B after the others
//   Params                     passes, a_part, b_part (columns between the parts), promote (stages an accumulator sums
//                              before it is handed over), status
//   Op(p, dynamic memory)      every thread; may synchronise the block
//   units(), unit(u)           the work
//   kStageOut                  bytes of shared memory for each epilogue warp (on 1024 bytes where they are a multiple of it)
//   warp(stage, quad, team, lane), finish()   once, epilogue warps: before the first unit, after the last
//   kAhead, ahead(x, ct)       before a tile is waited for
//   kSplit                     more registers for the epilogue
//   kSingle                    every unit is one tile of p.steps with one accumulator
//   begin(x), tile(x, ct, acc, first, last), end(x)   a unit; a column tile's accumulator, or (promote) the parts of it
template <class Op, int CG>
__global__ void __launch_bounds__(kThreadsT, 1)
k_tiles(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
        const __grid_constant__ typename Op::Params p) {
  constexpr int BN = Op::kBN;
  using R = Ring<BN, CG, Op::kKeep, Op::kTri>;
  constexpr int kCols = BN / CG;  // columns of B that a block copies
  constexpr int kAccs = BN >= 256 ? 2 : 4;
  extern __shared__ uint8_t s_raw[];
  __shared__ Barriers bar;
  uint8_t* ring = reinterpret_cast<uint8_t*>(((uintptr_t)s_raw + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % CG;  // in the pair
  const int kept = kept_of<Op>(p);
  const int stages = R::stages(kept);
  uint8_t* stages_at = ring + kept * R::kStageA;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 8; ++i) {
      tc::mbar_init(&bar.full[i], 1);
      tc::mbar_init(&bar.empty[i], 1);
    }
    tc::mbar_init(&bar.a_full, 1);
    tc::mbar_init(&bar.a_empty, 1);
    for (int i = 0; i < kAccs; ++i) {
      tc::mbar_init(&bar.acc_full[i], 1);
      tc::mbar_init(&bar.acc_empty[i], (Op::kTeams ? kEpiWarps / 2 : kEpiWarps) * CG);
    }
    tc::mbar_init(&bar.done, 1);
    tc::mbar_init_fence();
  }
  __syncwarp();
  if (warp == 1) tc::tmem_alloc<CG>(&bar.tmem, kAccs * BN);
  tc::fence_before();
  if constexpr (CG == 2) tc::cluster_sync();
  else __syncthreads();
  tc::fence_after();
  const uint32_t tmem = bar.tmem;
  lead();
  follow();
  Op op(p, ring + R::kTotal + kEpiWarps * Op::kStageOut, rank);
  const long long units = op.units(), u0 = blockIdx.x / CG, ustep = gridDim.x / CG;

  if (warp < 4) {
    if constexpr (Op::kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    if (warp == 0) {
      const bool one = tc::elect_one();
      tc::Slot s;
      long long issued = 0;
      uint32_t a_phase = 0;
      bool ok = true;
      // one step of A into `to`
      auto load_a = [&](uint8_t* to, uint64_t* full, int x, int r0, int k) {
        if constexpr (CG == 2) {
          const uint32_t at = tc::of_leader(full);
          if constexpr (Op::kAMN) {
#pragma unroll
            for (int c = 0; c < kBM / 64; ++c) tc::tma_load_2d_pair(to + c * 8192, &map_a, at, x + r0 + c * 64, k * kBK);
          } else {
            tc::tma_load_2d_pair(to, &map_a, at, x + k * kBK, r0);
          }
        } else {
          if constexpr (Op::kAMN) {
#pragma unroll
            for (int c = 0; c < kBM / 64; ++c) tc::tma_load_2d(to + c * 8192, &map_a, full, x + r0 + c * 64, k * kBK);
          } else {
            tc::tma_load_2d(to, &map_a, full, x + k * kBK, r0);
          }
        }
      };
      for (long long u = u0; u < units && ok; u += ustep) {
        const Unit x = op.unit(u);
        const int r0 = x.row0 + rank * kBM;
        if constexpr (Op::kKeep) {
          ok = tc::warp_wait(&bar.a_empty, a_phase ^ 1);
          if (!ok) break;
          a_phase ^= 1;
          if (one) {  // a pair's copies count on the first block's barrier
            if (rank == 0) tc::mbar_expect(&bar.a_full, CG * kept * R::kStageA);
            const int steps = x.k1 - x.k0;
            for (int i = 0; i < kept; ++i) load_a(ring + i * R::kStageA, &bar.a_full, i / steps * p.a_part, r0, x.k0 + i % steps);
          }
          __syncwarp();
        }
        for (int ct = x.ct0; ct < x.ct1 && ok; ++ct) {
          for (int q = 0; q < p.passes && ok; ++q) {
            const int ap = part_a(p.passes, q) * p.a_part, bp = part_b(p.passes, q) * p.b_part;
            for (int k = x.k0; k < x.k1; ++k) {
              ok = tc::warp_wait(&bar.empty[s.stage], s.phase ^ 1);
              if (!ok) break;
              uint8_t* st = stages_at + s.stage * R::kStage;
              uint8_t* sb = st + (Op::kKeep ? 0 : R::kParts * R::kStageA);
              if (one) {
                uint64_t* full = &bar.full[s.stage];
                if (rank == 0) tc::mbar_expect(full, CG * R::kStage);
                if constexpr (Op::kTri) {
                  static_assert(!Op::kTri || (CG == 1 && Op::kBMN && !Op::kKeep), "the only form with three parts at once");
#pragma unroll
                  for (int i = 0; i < 3; ++i) {
                    load_a(st + i * R::kStageA, full, i * p.a_part, r0, k);
#pragma unroll
                    for (int c = 0; c < kCols / 64; ++c)
                      tc::tma_load_2d(sb + i * R::kStageB + c * 8192, &map_b, full, i * p.b_part + ct * BN + c * 64, k * kBK);
                  }
                } else {
                if constexpr (!Op::kKeep) load_a(st, full, ap, r0, k);
                if constexpr (CG == 2) {
                  const uint32_t at = tc::of_leader(full);
                  if constexpr (Op::kBMN) {
#pragma unroll
                    for (int c = 0; c < kCols / 64; ++c)
                      tc::tma_load_2d_pair(sb + c * 8192, &map_b, at, bp + ct * BN + rank * kCols + c * 64, k * kBK);
                  } else if constexpr (Op::kTwoB) {  // the first block copies the first weights' columns, the second the second's
                    tc::tma_load_3d_pair(sb, &map_b, at, bp + k * kBK, ct * kCols + rank * p.b_second, x.g);
                  } else {
                    tc::tma_load_2d_pair(sb, &map_b, at, bp + k * kBK, ct * BN + rank * kCols);
                  }
                } else {
                  if constexpr (Op::kBMN) {
#pragma unroll
                    for (int c = 0; c < kCols / 64; ++c) tc::tma_load_2d(sb + c * 8192, &map_b, full, bp + ct * BN + c * 64, k * kBK);
                  } else if constexpr (Op::kTwoB) {
                    tc::tma_load_3d(sb, &map_b, full, bp + k * kBK, ct * (BN / 2), x.g);
                    tc::tma_load_3d(sb + R::kStageB / 2, &map_b, full, bp + k * kBK, ct * (BN / 2) + p.b_second, x.g);
                  } else {
                    tc::tma_load_2d(sb, &map_b, full, bp + k * kBK, ct * BN);
                  }
                }
                }
              }
              __syncwarp();
              ++issued;
              s.next(stages);
            }
          }
        }
      }
      ok = ok && tc::all_released(bar, s, issued, stages);
      // what the first block signals of its last products has to have arrived here before this block ends
      if (rank != 0) ok = tc::mbar_wait(&bar.done, 0) && ok;
      if (!ok) {
        if (one) tc::latch_status(p.status, MT_ECUDA);
        if (rank == 0) {
          tc::drain(bar, s, issued, stages);
          if (Op::kKeep && (issued > 0 || a_phase != 0)) tc::mbar_wait(&bar.a_full, a_phase ^ 1);
        }
      }
    } else if (warp == 1) {
      if (rank == 0) {
        constexpr uint32_t instr = tc::instr_bf16(kBM * CG, BN, Op::kAMN, Op::kBMN);
        // descriptors' low words: of the ring's (and the kept A's) first stage, from one stage to the next, from one 16 of the
        // contraction to the next
        constexpr uint32_t kLeadA = Op::kAMN ? 8192 : 16, kLeadB = Op::kBMN ? 8192 : 16;
        constexpr uint32_t kStepA = Op::kAMN ? 2048 >> 4 : 32 >> 4, kStepB = Op::kBMN ? 2048 >> 4 : 32 >> 4;
        const bool one = tc::elect_one();
        const uint32_t a0 = tc::desc_low(tc::smem_addr(Op::kKeep ? ring : stages_at), kLeadA);
        const uint32_t b0 = tc::desc_low(tc::smem_addr(stages_at + (Op::kKeep ? 0 : R::kParts * R::kStageA)), kLeadB);
        tc::Slot s;
        int acc = 0;
        uint32_t acc_phase = 0, a_phase = 0;
        bool ok = true;
        for (long long u = u0; u < units && ok; u += ustep) {
          Unit x;
          if constexpr (Op::kSingle) {  // nothing of a unit has to be found: it would hold the products up
            x.k0 = x.ct0 = 0;
            x.k1 = p.steps;
            x.ct1 = 1;
          } else {
            x = op.unit(u);
          }
          const int per_pass = x.k1 - x.k0;
          if constexpr (Op::kKeep) {
            ok = tc::warp_wait<CG == 2>(&bar.a_full, a_phase);
            a_phase ^= 1;
            if (!ok) break;
          }
          for (int ct = x.ct0; ct < x.ct1 && ok; ++ct) {
            int part = 0;  // stages that the accumulator has
            for (int q = 0; q < p.passes && ok; ++q) {
              uint32_t a_at = a0 + part_a(p.passes, q) * per_pass * (R::kStageA >> 4);  // (kept A)
              for (int k = 0; k < per_pass; ++k) {
                if (part == 0) {
                  ok = tc::warp_wait(&bar.acc_empty[acc], acc_phase ^ 1);
                  if (!ok) break;
                  tc::fence_after();
                }
                ok = tc::warp_wait<CG == 2>(&bar.full[s.stage], s.phase);
                if (!ok) break;
                tc::fence_after();
                const uint32_t b = b0 + s.stage * (R::kStage >> 4), a = Op::kKeep ? a_at : a0 + s.stage * (R::kStage >> 4);
                const bool closes = part + 1 == p.promote || (k + 1 == per_pass && q + 1 == p.passes);
                if (one) {
#pragma unroll
                  for (int q3 = 0; q3 < (Op::kTri ? 6 : 1); ++q3) {
                    const uint32_t aq = a + (Op::kTri ? part_a(6, q3) * (R::kStageA >> 4) : 0), bq = b + (Op::kTri ? part_b(6, q3) * (R::kStageB >> 4) : 0);
#pragma unroll
                    for (int i = 0; i < kBK / 16; ++i)
                      tc::mma_bf16<CG>(tmem + acc * BN, aq + i * kStepA, bq + i * kStepB, instr, part > 0 || i > 0 || q3 > 0);
                  }
                  tc::mma_commit<CG>(&bar.empty[s.stage]);
                  if (closes) tc::mma_commit<CG>(&bar.acc_full[acc]);
                }
                __syncwarp();
                a_at += R::kStageA >> 4;
                s.next(stages);
                ++part;
                if (closes) {
                  if (++acc == kAccs) {
                    acc = 0;
                    acc_phase ^= 1;
                  }
                  part = 0;
                }
              }
            }
          }
          if (Op::kKeep && ok && one) tc::mma_commit<CG>(&bar.a_empty);
          __syncwarp();
        }
        if (one) tc::mma_commit<CG>(&bar.done);  // tensor memory is freed only when no product writes it, also after a wait ran out
        __syncwarp();
        ok = tc::mbar_wait(&bar.done, 0) && ok;
        if (!ok && one) tc::latch_status(p.status, MT_ECUDA);
      }
    }
  } else {
    if constexpr (Op::kSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
    const int quad = warp & 3, team = (warp - 4) >> 2;
    op.warp(ring + R::kTotal + (warp - 4) * Op::kStageOut, quad, team, lane);
    uint32_t seq = 0;  // accumulators so far
    bool ok = true;
    for (long long u = u0; u < units && ok; u += ustep) {
      const Unit x = op.unit(u);
      op.begin(x);
      const int steps = (x.k1 - x.k0) * p.passes;
      const int parts = steps <= p.promote ? 1 : (steps + p.promote - 1) / p.promote;
      for (int ct = x.ct0; ct < x.ct1 && ok; ++ct) {
        for (int part = 0; part < parts; ++part) {
          const uint32_t b = seq % kAccs, parity = seq / kAccs & 1;
          if (Op::kTeams && (steps > 0 ? seq & 1 : 0) != team) {
            seq += steps > 0;
            continue;
          }
          seq += steps > 0;
          if constexpr (Op::kAhead) op.ahead(x, ct);
          if (steps > 0) {
            ok = __all_sync(kFull, tc::mbar_wait(&bar.acc_full[b], parity));
            if (!ok) break;
            tc::fence_after();
          }
          const Acc a{tmem + b * BN + ((uint32_t)(quad * 32) << 16), &bar.acc_empty[b], steps > 0};
          op.template tile<CG>(x, ct, a, part == 0, part + 1 == parts);
        }
      }
      if (ok) op.end(x);
    }
    op.finish();
    if (!ok) tc::latch_status(p.status, MT_ECUDA);
  }
  __syncwarp();
  tc::fence_before();
  if constexpr (CG == 2) tc::cluster_sync();
  else __syncthreads();
  tc::fence_after();
  if (warp == 1) tc::tmem_free<CG>(tmem, kAccs * BN);
}

// ---- rows through an epilogue warp's shared memory -------------------------------------------
//
// A lane holds its row's columns; global memory wants neighbouring lanes on
// neighbouring columns.  64 bytes of each of 32 rows go through shared memory as
// four 16-byte pieces, piece c of row r at c ^ ((r >> 1) & 3): writes and reads of
// eight neighbouring lanes then meet all banks.

__device__ __forceinline__ uint32_t piece_at(int row, int c) { return (uint32_t)(row * 64 + ((c ^ ((row >> 1) & 3)) << 4)); }

// How rows may be reached: by elements, in 16-byte pieces turned in shared memory, or in 32-byte sectors as they are.
enum Reach { kElements = 0, kPieces = 1, kSectors = 2 };
inline int reach_of(const void* data, int64_t ld, int64_t columns, size_t bytes) {
  const auto on = [&](size_t a) { return is_aligned(data, a) && ld * bytes % a == 0 && columns * bytes % a == 0; };
  return on(32) ? kSectors : on(16) ? kPieces : kElements;
}
__device__ __forceinline__ void store_sector(void* to, const uint32_t* w);

// Stores 64 bytes of each lane's row (w: 16 words; element j of the row is column col + j): rows [0, rows) of C from r0 on,
// columns below J.  In sectors where rows allow it: nothing passes through shared memory, whose bandwidth the products
// need.
template <typename T>
__device__ __forceinline__ void store_rows(uint8_t* stage, int lane, const uint32_t (&w)[16], T* C, size_t ldc, long long r0,
                                           int rows, int col, int J, int reach) {
  constexpr int kPer = 64 / sizeof(T);  // columns
  if (col >= J) return;
  if (reach == kSectors) {
    T* to = C + (size_t)(r0 + lane) * ldc + col;
    if (lane < rows) {
      store_sector(to, w);
      if (col + kPer / 2 < J) store_sector(to + kPer / 2, w + 8);
    }
    return;
  }
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<uint4*>(stage + piece_at(lane, c)) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  __syncwarp();
  if (reach == kPieces) {
    const int c = lane & 3, at = col + c * (16 / (int)sizeof(T));
    T* to = C + (size_t)r0 * ldc + at;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = q * 8 + (lane >> 2);
      if (r < rows && at < J) *reinterpret_cast<uint4*>(to + (size_t)r * ldc) = *reinterpret_cast<const uint4*>(stage + piece_at(r, c));
    }
  } else {
    const int j = lane % kPer;
    T* to = C + (size_t)(r0 + lane / kPer) * ldc + col + j;
#pragma unroll 8
    for (int r = lane / kPer; r < 32; r += 32 / kPer, to += (size_t)(32 / kPer) * ldc) {
      if (r < rows && col + j < J)
        *to = *reinterpret_cast<const T*>(stage + piece_at(r, j * (int)sizeof(T) / 16) + j * (int)sizeof(T) % 16);
    }
  }
}

// 32 bytes of a lane's row at once (sm_100 and later): a whole sector of global memory, so rows need no turning.
__device__ __forceinline__ void store_sector(void* to, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
               "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Loads 32 columns of each lane's row as fp32 (zeros outside): the reverse.
template <typename T>
__device__ __forceinline__ void load_rows(uint8_t* stage, int lane, float (&f)[32], const T* C, size_t ldc, long long r0, int rows,
                                          int col, int J, int reach) {
  if (reach != kElements) {
    const T* p = C + (size_t)(r0 + lane) * ldc + col;
    constexpr int kPer = 16 / sizeof(T);
#pragma unroll
    for (int c = 0; c < 32 / kPer; ++c) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (lane < rows && col + c * kPer < J) v = reinterpret_cast<const uint4*>(p)[c];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) {
          f[c * 4 + j] = __uint_as_float(w[j]);
        } else {
          f[c * 8 + 2 * j] = __uint_as_float(w[j] << 16);
          f[c * 8 + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
      }
    }
    return;
  }
  constexpr int kPer = 64 / sizeof(T);  // columns through the stage at a time
#pragma unroll
  for (int h = 0; h < 32 / kPer; ++h) {
    __syncwarp();
    const int j = lane % kPer, at = col + h * kPer + j;
    const T* from = C + (size_t)(r0 + lane / kPer) * ldc + at;
#pragma unroll 8
    for (int r = lane / kPer; r < 32; r += 32 / kPer, from += (size_t)(32 / kPer) * ldc) {
      T v = from_f<T>(0.0f);
      if (r < rows && at < J) v = *from;
      *reinterpret_cast<T*>(stage + piece_at(r, j * (int)sizeof(T) / 16) + j * (int)sizeof(T) % 16) = v;
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      f[h * kPer + j] = to_f<T>(*reinterpret_cast<const T*>(stage + piece_at(lane, j * (int)sizeof(T) / 16) + j * (int)sizeof(T) % 16));
  }
}

// The same words of 32 fp32 columns: rounded to bf16 (16 words), or half of them as they are.
__device__ __forceinline__ void narrow32(const float (&f)[32], uint32_t (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) w[j] = bf16x2_of(f[2 * j], f[2 * j + 1]);
}

// Stores 32 fp32 columns of each lane's row as T.
template <typename T>
__device__ __forceinline__ void store32(uint8_t* stage, int lane, const float (&f)[32], T* C, size_t ldc, long long r0, int rows,
                                        int col, int J, int reach) {
  uint32_t w[16];
  if constexpr (sizeof(T) == 2) {
    narrow32(f, w);
    store_rows<T>(stage, lane, w, C, ldc, r0, rows, col, J, reach);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(f[h * 16 + j]);
      store_rows<T>(stage, lane, w, C, ldc, r0, rows, col + h * 16, J, reach);
    }
  }
}

// ---- host ----------------------------------------------------------------------------------------

// Launches an operator over `units` units (at most), in clusters of CG blocks, following the kernel before it, with `extra` bytes of its own shared
// memory of at most `most`.
template <class Op, int CG>
cudaError_t launch(const char* name, const CUtensorMap& a, const CUtensorMap& b, const typename Op::Params& p, long long units,
                   size_t extra, size_t most, cudaStream_t s) {
  constexpr size_t ring = 1024 + Ring<Op::kBN, CG, Op::kKeep, Op::kTri>::kTotal + kEpiWarps * Op::kStageOut;  // the stages start on 1024 bytes
  static SmemLimit limit;
  // (a split of the registers needs the launch to bring them: a kernel that has one is compiled to the most that its launch
  // bounds leave a thread)
  const cudaError_t e = limit.allow(k_tiles<Op, CG>, ring + most, Op::kSplit ? kRegsLaunch : 0);
  if (e != cudaSuccess) return e;
  const int blocks = sm_count() / CG;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((units < blocks ? (units > 0 ? units : 1) : blocks) * CG));
  cfg.blockDim = dim3(kThreadsT);
  cfg.dynamicSmemBytes = ring + extra;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG > 1 ? 2 : 1;
  MT_LAUNCH(name, s);
  return cudaLaunchKernelEx(&cfg, k_tiles<Op, CG>, a, b, p);
}

}  // namespace tiles
}  // namespace mt
