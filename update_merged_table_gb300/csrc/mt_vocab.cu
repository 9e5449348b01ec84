// Losses of rows against a vocabulary whose logits are never kept: cross entropy,
// and distillation from a teacher's top logits.
//
//   k_vocab_mark   which rows take part (one bit each; few rows: k_vocab_rows sees to it)
//   k_vocab_rows   the rows that do, one after the other: their values as the
//                  tensor cores take them (bf16; fp32 in three parts), their targets
//                  in ascending order with their shares, for the backward the row's
//                  factors.  Rows that take no part cost nothing afterwards, and
//                  nothing of them can reach a sum.
//   k_logit_stats  (mt_vocab_logits.cu) largest logit, sum of exponentials, targets'
//                  logits, per row and run of the vocabulary
//   k_vocab_loss   joins the runs: lse and loss
//   k_logit_grad   the gradient of a piece of the logits
//   k_vocab_dx, k_vocab_dw  (mt_vocab_sums.cu) the products of that piece
//   k_vocab_fused_dx, k_vocab_fused_dw  (mt_vocab_fused.cu) both without the piece in memory, for narrow rows
//   k_vocab_dx_sum, k_vocab_dw_sum  partial products joined, rounded, put in place
#include <algorithm>

#include "mt_tiles.cuh"
#include "mt_vocab.cuh"

namespace mt {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

struct VocabRows {
  long long n;
  int vocab, dim, top;  // top: entries of a row's list (1: cross entropy)
  bool wide_ids, teacher16;
  const void* targets;
  const void* teacher;
  int32_t* status;
  float scale, smoothing, z_loss;
  const void* x;
  int64_t ldx;
  // made here
  uint32_t* mask;   // [ceil(n / 32)]
  int* live;        // [1]
  int* pos;         // [n] a row's place among the live ones, -1
  __nv_bfloat16* xs;  // [n][parts][dp]
  int dp;
  int* ids;
  float* share;
  float* entropy;   // [n] sum of share log share
  // backward
  const float* dloss;
  const float* lse;
  float4* coef;
};

__device__ __forceinline__ long long id_at(const VocabRows& p, long long i) {
  return p.wide_ids ? static_cast<const long long*>(p.targets)[i] : static_cast<const int*>(p.targets)[i];
}
__device__ __forceinline__ float teacher_at(const VocabRows& p, long long i) {
  return p.teacher16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.teacher)[i]) : static_cast<const float*>(p.teacher)[i];
}
template <bool DISTILL>
__device__ __forceinline__ bool pair_there(const VocabRows& p, long long i, long long id) {
  return id >= 0 && id < p.vocab && (!DISTILL || !(teacher_at(p, i) == -INFINITY));
}

// Whether a row has a pair that is there among every step-th from `first` on; what is outside the vocabulary is latched.
template <bool DISTILL>
__device__ __forceinline__ bool row_there(const VocabRows& p, long long row, int first = 0, int step = 1) {
  const int top = DISTILL ? p.top : 1;
  bool there = false, bad = false;
  for (int k = first; k < top; k += step) {
    const long long id = id_at(p, row * top + k);
    bad |= id >= p.vocab;
    there |= pair_there<DISTILL>(p, row * top + k, id);
  }
  if (bad && p.status != nullptr) atomicCAS(p.status, 0, MT_EINVAL);
  return there;
}

// A block per 32 rows: a thread per row where it has one target, else a warp.
template <bool DISTILL>
__global__ void __launch_bounds__(256) k_vocab_mark(const VocabRows p) {
  lead();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long words = (p.n + 31) / 32;
  if constexpr (!DISTILL) {
    for (long long w = (long long)blockIdx.x * 8 + warp; w < words; w += (long long)gridDim.x * 8) {
      const unsigned bits = __ballot_sync(kFull, w * 32 + lane < p.n && row_there<false>(p, w * 32 + lane));
      if (lane == 0) p.mask[w] = bits;
    }
  } else {
    __shared__ uint32_t s_bits;
    for (long long w = blockIdx.x; w < words; w += gridDim.x) {
      if (threadIdx.x == 0) s_bits = 0u;
      __syncthreads();
      for (int r = warp; r < 32; r += 8) {
        const long long row = w * 32 + r;
        bool there = false, bad = false;
        if (row < p.n) {
          for (int k = lane; k < p.top; k += 32) {
            const long long id = id_at(p, row * p.top + k);
            bad |= id >= p.vocab;
            there |= pair_there<true>(p, row * p.top + k, id);
          }
        }
        if (bad && p.status != nullptr) atomicCAS(p.status, 0, MT_EINVAL);
        if (__any_sync(kFull, there) && lane == 0) atomicOr(&s_bits, 1u << r);
      }
      __syncthreads();
      if (threadIdx.x == 0) p.mask[w] = s_bits;
      __syncthreads();
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

// A row's targets are put in order by a warp: up to kRankPairs of them each by how many others come before it (a step for each
// pair of targets), more by a bitonic sort in shared memory.  Forward against 8192 x 64, each way for both: 2 rows of 8 pairs
// 12.3 us (counted) and 14.4 (sorted), of 64 16.4 and 16.0, of 128 25 and 17.7, of 1024 606 and 60; 4096 rows of 8 27 and 34,
// of 64 44.7 and 47.2, of 128 82 and 67, of 1024 1862 and 451.
constexpr int kRankPairs = 64;
__host__ __device__ inline int sorted_pairs(int top) {  // places that the sort needs: a power of two
  int size = kRankPairs;
  while (size < top) size *= 2;
  return size;
}
// Shared memory of a warp: the targets to be put in order, and their shares.
inline size_t list_bytes(int top) { return top > kRankPairs ? (size_t)sorted_pairs(top) * 12 : (size_t)top * 8; }

__device__ __forceinline__ void warp_sort(unsigned long long* s, int size, int lane) {
  constexpr int kOnce = 2;  // pairs a lane has loaded before it stores any (4: 64 registers, 5224 rows of 2 pairs 23.9 to 25.8 us)
  for (int k = 2; k <= size; k *= 2) {
    for (int j = k / 2; j > 0; j /= 2) {
      __syncwarp();
      for (int i0 = lane; i0 < size / 2; i0 += 32 * kOnce) {
        unsigned long long x[kOnce], y[kOnce];
        int at[kOnce];
#pragma unroll
        for (int q = 0; q < kOnce; ++q) {
          const int i = i0 + 32 * q;
          at[q] = 2 * i - (i & (j - 1));
          if (i < size / 2) {
            x[q] = s[at[q]];
            y[q] = s[at[q] + j];
          }
        }
#pragma unroll
        for (int q = 0; q < kOnce; ++q) {
          if (i0 + 32 * q < size / 2 && (x[q] > y[q]) == ((at[q] & k) == 0)) {
            s[at[q]] = y[q];
            s[at[q] + j] = x[q];
          }
        }
      }
    }
  }
  __syncwarp();
}

// MARK: few rows, of up to kMarkRows targets or kMarkPairs pairs, which every block looks through itself (no k_vocab_mark before it): a
// thread to a row of up to kLanePairs, else eight lanes, or 32 from 65 on.  Forward in us, so, with k_vocab_mark, and by a
// thread to any row: against 32,771 x 320, 37 rows of 8 pairs 16.9, 19.0 and 16.9, 200 of 9 24 (thread) or 27 (lanes) and 26,
// 64 of 32 18.8, 20.4 and 28.3, 16 of 128 23.8, 25.0 and 38, 2 of 1024 56, 63 and 111; against 8192 x 64, 256 targets 13.1 and
// 13.7, 1024 15.4 and 15.2, 2048 17.6 and 16.2, 1024 rows of 2 pairs 18.3 and 19.2.
constexpr int kMarkRows = 1024, kMarkPairs = 2048, kLanePairs = 16;

constexpr int kRowBlocks = 4;  // blocks to 32 rows: a warp has one row at most

// A quarter of 32 rows' live ones per block, a warp each; the last block writes how many there are and puts zeros behind them up to the
// next 128 rows (steps of dW's contraction).  T: the rows' type; AL: they can be read in 16-byte vectors.
// LIST: what a row has, kTarget one target, kCounted and kSorted a teacher's pairs (each form by itself: all in one took a few
// rows' call a microsecond or two longer).
enum List { kTarget, kCounted, kSorted };
template <typename T, bool AL, bool MARK, int LIST>
__global__ void __launch_bounds__(256) k_vocab_rows(const VocabRows p) {
  lead();
  if (!MARK) follow();
  constexpr int kParts = sizeof(T) == 4 ? 3 : 1;
  constexpr bool DISTILL = LIST != kTarget;
  extern __shared__ __align__(16) uint8_t s_mem[];
  __shared__ int s_base;
  __shared__ uint32_t s_mask[MARK && DISTILL ? kMarkPairs / (kLanePairs + 1) / 32 + 1 : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long words = (p.n + 31) / 32, all = words * kRowBlocks, per = (all + gridDim.x - 1) / gridDim.x;
  const long long q0 = blockIdx.x * per, q1 = min(q0 + per, all);  // a block's quarters lie one after the other
  if (q0 >= q1) return;
  // the live rows before the block's first word
  int before = 0;
  const bool wide = MARK && DISTILL && p.top > kLanePairs;
  if (threadIdx.x == 0) s_base = 0;
  if (wide) {
    if (threadIdx.x < words) s_mask[threadIdx.x] = 0u;
    __syncthreads();
    const int rows = (int)min(p.n, ((q1 - 1) / kRowBlocks + 1) * 32);  // up to the block's last one
    const int shift = p.top > 64 ? 5 : 3;
    for (int r0 = 0; r0 < rows; r0 += 256 >> shift) {
      const int row = r0 + ((int)threadIdx.x >> shift);
      const bool there = row < rows && row_there<DISTILL>(p, row, threadIdx.x & ((1 << shift) - 1), 1 << shift);
      const unsigned bits = __reduce_or_sync(kFull, there ? 1u << (row & 31) : 0u);  // a warp's rows are of one word
      if (lane == 0 && bits != 0u) atomicOr(&s_mask[row >> 5], bits);
    }
  }
  __syncthreads();
  if (wide) {
    for (long long i = threadIdx.x; i < q0 / kRowBlocks; i += blockDim.x) before += __popc(s_mask[i]);
    __syncwarp();
  } else if constexpr (MARK) {
    for (long long i = threadIdx.x; i < q0 / kRowBlocks * 32; i += blockDim.x) before += row_there<DISTILL>(p, i);
    __syncwarp();
  } else {
    for (long long i = threadIdx.x; i < q0 / kRowBlocks; i += blockDim.x) before += __popc(p.mask[i]);
  }
  before = __reduce_add_sync(kFull, before);
  if (lane == 0) atomicAdd(&s_base, before);
  __syncthreads();
  int base = s_base;
  for (long long q = q0; q < q1; ++q) {
    const long long w = q / kRowBlocks;
    const int share = (int)(q % kRowBlocks);
    uint32_t bits;
    if constexpr (MARK) bits = wide ? s_mask[w] : __ballot_sync(kFull, w * 32 + lane < p.n && row_there<DISTILL>(p, w * 32 + lane));
    else bits = p.mask[w];
    const int own = __popc(bits);
    if (share == 0 && threadIdx.x < 32 && w * 32 + lane < p.n)
      p.pos[w * 32 + lane] = bits >> lane & 1 ? base + __popc(bits & ((1u << lane) - 1u)) : -1;
    for (int k = share * 8 + warp; k < own; k += 8 * kRowBlocks) {
      const long long row = w * 32 + __fns(bits, 0, k + 1);
      const size_t at = (size_t)base + k;
      // the row's values
      __nv_bfloat16* to = p.xs + at * ((size_t)kParts * p.dp);
      const Rows x{const_cast<T*>(static_cast<const T*>(p.x) + row * p.ldx), 0, nullptr, nullptr};
      for (int v = lane; v < p.dp / 8; v += 32) {
        const Raw8<T> raw = load8<T, AL>(x, 0, v, p.dim);
        if constexpr (kParts == 1) {
          *reinterpret_cast<uint4*>(to + v * 8) = raw.a;
        } else {
          float f[8];
          widen8<T>(raw, false, f);
          uint32_t q[3][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            __nv_bfloat16 a[3], b[3];
            split3(f[2 * j], a[0], a[1], a[2]);
            split3(f[2 * j + 1], b[0], b[1], b[2]);
#pragma unroll
            for (int i = 0; i < 3; ++i) q[i][j] = bf16_bits(a[i], b[i]);
          }
#pragma unroll
          for (int i = 0; i < 3; ++i) *reinterpret_cast<uint4*>(to + (size_t)i * p.dp + v * 8) = make_uint4(q[i][0], q[i][1], q[i][2], q[i][3]);
        }
      }
      // its targets and their shares
      if constexpr (!DISTILL) {
        if (lane == 0) {
          p.ids[at] = (int)id_at(p, row);
          p.share[at] = 1.0f - p.smoothing;
        }
      } else {
        // (the differences are scaled, not the logits: a type's lowest or largest value times the scale may be no number)
        const int size = LIST == kSorted ? sorted_pairs(p.top) : p.top;
        unsigned long long* s_key = reinterpret_cast<unsigned long long*>(s_mem) + warp * size;  // kSorted: the id, then its place among the pairs
        int* s_id = reinterpret_cast<int*>(s_mem) + warp * size;                                 // kCounted
        float* s_t = reinterpret_cast<float*>(s_mem + (size_t)8 * size * (LIST == kSorted ? 8 : 4)) + warp * size;
        float top = -INFINITY;
        for (int j = lane; j < p.top; j += 32) {
          const long long id = id_at(p, row * p.top + j);
          const bool there = pair_there<true>(p, row * p.top + j, id);
          const int key = there ? (int)id : 0x7FFFFFFF;  // ids that are not there come last, with a share of zero
          if constexpr (LIST == kSorted) s_key[j] = (unsigned long long)(unsigned)key << 32 | (unsigned)j;
          else s_id[j] = key;
          s_t[j] = there ? teacher_at(p, row * p.top + j) : -INFINITY;
          top = fmaxf(top, s_t[j]);
        }
        top = warp_max(top);
        float sum = 0.0f;
        for (int j = lane; j < p.top; j += 32) sum += expf(p.scale * (s_t[j] - top));
        sum = warp_sum(sum);
        const float inv = 1.0f / sum, log_sum = logf(sum);
        float entropy = 0.0f;
        __syncwarp();
        for (int j = lane; j < p.top; j += 32) {
          const float d = p.scale * (s_t[j] - top), t = expf(d) * inv;
          if (t != 0.0f) entropy += t * (d - log_sum);
          if constexpr (LIST == kSorted) {
            s_t[j] = t;
          } else {
            const int id = s_id[j];
            int rank = 0;
            for (int i = 0; i < p.top; ++i) rank += s_id[i] < id || (s_id[i] == id && i < j);
            p.ids[at * p.top + rank] = id;
            p.share[at * p.top + rank] = t;
          }
        }
        if constexpr (LIST == kSorted) {
          for (int j = p.top + lane; j < size; j += 32) s_key[j] = ~0ull;
          warp_sort(s_key, size, lane);
          for (int j = lane; j < p.top; j += 32) {
            const unsigned long long key = s_key[j];
            p.ids[at * p.top + j] = (int)(key >> 32);
            p.share[at * p.top + j] = s_t[(unsigned)key];
          }
        }
        entropy = warp_sum(entropy);
        if (lane == 0) p.entropy[at] = entropy;
        __syncwarp();
      }
      if (p.coef != nullptr && lane == 0) {
        const float lse = p.lse[row], g = p.dloss[row] * p.scale;
        p.coef[at] = make_float4(lse * kLog2e, g * (1.0f + 2.0f * p.z_loss * lse), g * p.smoothing / (float)p.vocab, g);
      }
    }
    if (q + 1 == all) {
      const int live = base + own;
      if (threadIdx.x == 0) *p.live = live;
      const size_t width = (size_t)kParts * p.dp;
      const size_t first = (size_t)live * width, last = (size_t)((live + 127) / 128 * 128) * width;
      for (size_t i = first / 8 + threadIdx.x; i < last / 8; i += blockDim.x) reinterpret_cast<uint4*>(p.xs)[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    if (share == kRowBlocks - 1) base += own;
  }
}

struct VocabLoss {
  long long n;
  int vocab, top;
  const int* pos;
  const float2* part;
  const float* sum_z;
  size_t stride;
  const int* chunks;
  int teams;             // partial statistics of a run
  const float* picked;
  const float* share;
  const float* entropy;  // NULL: cross entropy
  float scale, smoothing, z_loss;
  float* loss;
  float* lse;
};

// A warp per row: the runs' statistics joined.
__global__ void __launch_bounds__(256) k_vocab_loss(const VocabLoss p) {
  lead();
  follow();
  const int lane = threadIdx.x & 31;
  const int slots = p.teams * *p.chunks;
  for (long long row = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5; row < p.n; row += ((long long)gridDim.x * blockDim.x) >> 5) {
    const int at = p.pos[row];
    if (at < 0) {
      if (lane == 0) p.loss[row] = p.lse[row] = 0.0f;
      continue;
    }
    // the runs' largest logit first (their loads do not wait for one another), then their sums brought to it
    float top = -INFINITY;
#pragma unroll 4
    for (int k = lane; k < slots; k += 32) top = fmaxf(top, p.part[(size_t)k * p.stride + at].x);
    top = warp_max(top);
    const float off = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f, z = 0.0f, told = 0.0f;
#pragma unroll 4
    for (int k = lane; k < slots; k += 32) {
      const float2 q = p.part[(size_t)k * p.stride + at];
      sum += q.y * exp2f(q.x - off);
      if (p.sum_z != nullptr) z += p.sum_z[(size_t)k * p.stride + at];
    }
    for (int k = lane; k < p.top; k += 32) {
      const float t = p.share[(size_t)at * p.top + k];
      if (t != 0.0f) told += t * p.picked[(size_t)at * p.top + k];
    }
    sum = warp_sum(sum);
    told = warp_sum(told);
    const float lse = fmaf(top, 0.693147181f, logf(sum));
    float loss = fmaf(-p.scale, told, lse);
    if (p.sum_z != nullptr) loss = fmaf(-p.smoothing / (float)p.vocab * p.scale, warp_sum(z), loss);
    if (lane == 0) {
      if (p.entropy != nullptr) loss += p.entropy[at];
      p.loss[row] = fmaf(p.z_loss * lse, lse, loss);
      p.lse[row] = lse;
    }
  }
}

// The sum of `runs` values `step` apart, in their order, four loads under way.  The kernel before wrote them, so they come from
// L2 (ordinary loads, whichever way they were grouped: backward of 64 rows x 100,003 x 256, dx alone, 94 to 102 us, so 87).
__device__ __forceinline__ float4 sum_runs(const float4* from, size_t step, int runs) {
  constexpr int kOnce = 4;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add = [&](const float4& v) { s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w); };
  int k = 0;
  for (; k + kOnce <= runs; k += kOnce, from += kOnce * step) {
    float4 v[kOnce];
#pragma unroll
    for (int q = 0; q < kOnce; ++q) v[q] = __ldcg(from + q * step);
#pragma unroll
    for (int q = 0; q < kOnce; ++q) add(v[q]);
  }
  float4 v[kOnce - 1];
#pragma unroll
  for (int q = 0; q < kOnce - 1; ++q)
    if (k + q < runs) v[q] = __ldcg(from + q * step);
#pragma unroll
  for (int q = 0; q < kOnce - 1; ++q)
    if (k + q < runs) add(v[q]);
  return s;
}

// dx in its rows' places; zeros for rows that take no part.  The live rows from cut[0] on come in cut[1] runs.  FOUR: four
// columns a thread.
template <typename T, bool FOUR>
__global__ void __launch_bounds__(256) k_vocab_dx_sum(const float* part, size_t stride, const int* pos, long long n, int d, T* dx,
                                                      int64_t lddx, const int* cut) {
  lead();
  follow();
  constexpr int kPer = FOUR ? 4 : 1;
  const int per_row = d / kPer;
  const long long total = n * per_row;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (long long)gridDim.x * blockDim.x) {
    const long long row = i / per_row;
    const int j = (int)(i - row * per_row) * kPer, at = pos[row];
    const float* from = part + (size_t)at * d + j;
    const int runs = at >= cut[0] ? cut[1] : 1;
    T* to = dx + row * lddx + j;
    if constexpr (FOUR) {
      const float4 s = sum_runs(reinterpret_cast<const float4*>(from), stride * d / 4, at >= 0 ? runs : 0);
      if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(to) = s;
      else *reinterpret_cast<uint2*>(to) = make_uint2(bf16x2_of(s.x, s.y), bf16x2_of(s.z, s.w));
    } else {
      float s = 0.0f;
      if (at >= 0)
        for (int k = 0; k < runs; ++k) s += from[(size_t)k * stride * d];
      *to = from_f<T>(s);
    }
  }
}
// The rows of dW from cut[0] on, which came in cut[1] runs.  FOUR: four values a thread.
template <typename T, bool FOUR>
__global__ void __launch_bounds__(256) k_vocab_dw_sum(const float* part, size_t stride, const int* cut, long long rows, int d, T* dw) {
  lead();
  follow();
  constexpr int kPer = FOUR ? 4 : 1;
  const int runs = cut[1];
  const size_t first = (size_t)cut[0] * d;
  const long long values = (rows * d - (long long)first) / kPer;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < values; i += (long long)gridDim.x * blockDim.x) {
    if constexpr (FOUR) {
      const float4 s = sum_runs(reinterpret_cast<const float4*>(part) + i, stride * d / 4, runs);
      if constexpr (sizeof(T) == 4) reinterpret_cast<float4*>(dw + first)[i] = s;
      else reinterpret_cast<uint2*>(dw + first)[i] = make_uint2(bf16x2_of(s.x, s.y), bf16x2_of(s.z, s.w));
    } else {
      float s = 0.0f;
      for (int k = 0; k < runs; ++k) s += part[(size_t)k * stride * d + i];
      dw[first + i] = from_f<T>(s);
    }
  }
}

// `rows` rows of dW, at most `tail` of them in runs.
cudaError_t launch_dw_sum(const float* part, size_t stride, const int* cut, long long rows, long long tail, int d, int dtype, void* dw,
                          cudaStream_t s) {
  const bool four = d % 4 == 0 && is_aligned(dw, 4 * elem_bytes(dtype));
  const int grid = grid_for(tail * d / (four ? 4 : 1), 256, 8);
  MT_LAUNCH("k_vocab_dw_sum", s);
  auto go = [&](auto kernel, auto* to) { return launch_following(kernel, grid, 256, 0, s, part, stride, cut, rows, d, to); };
  if (dtype == MT_F32) return four ? go(k_vocab_dw_sum<float, true>, static_cast<float*>(dw)) : go(k_vocab_dw_sum<float, false>, static_cast<float*>(dw));
  return four ? go(k_vocab_dw_sum<__nv_bfloat16, true>, static_cast<__nv_bfloat16*>(dw))
              : go(k_vocab_dw_sum<__nv_bfloat16, false>, static_cast<__nv_bfloat16*>(dw));
}

// ---- host --------------------------------------------------------------------------------------

// Bytes of dz at a time, a 64th of the GPU's memory.  Every piece starts and ends three kernels and adds dx up in memory once
// more.  Measured with 1, 2, 4 and 8 GiB: backward of 262,144 x 100,003 x 256 36.8, 33.5, 32.4 and 31.0 ms, of 65,536 x 131,072 x
// 512 17.6, 16.9, 16.4 and 16.2; with 64 MiB, which the second-level cache would hold, 3.1 ms for 8192 x 100,003 x 512 against 1.9.
constexpr size_t kPieceBytes = (size_t)4 << 30;

struct Layout {
  int parts, dp, wp;          // parts of an operand; columns of a part of x and of W
  int dz_parts;
  bool copy_w, fused;         // fused: the gradients without dz in memory
  int whole;                  // fused: dW's tiles that need no partial products
  int runs_dx, runs_dw;       // room for runs
  int64_t rows;               // n in multiples of 256
  int top, max_chunks;
  int64_t piece;              // entries of the vocabulary at a time, a multiple of 256
  int64_t dw_rows;            // rows of dW's partial products
  size_t mask, live, chunks, cut, pos, xs, ids, share, entropy, w, picked, part, sum_z, coef, dz, dx, dw, total;
};

// dz of up to this many bf16 rows comes in two bf16 parts.  Its rounding (up to 2^-8 of a value) is one of many terms of dx and dw and
// adds about what their own rounding does; with few rows single terms show (one row: dw's row of the target is one product).
// Measured, relative error of dw with one part and with two: 2 rows 0.0029 and 0.0014 (its rounding alone 0.0014), 200 rows
// 0.0022 and 0.0016; backward of 16 x 100,003 x 256 91 and 112 us, of 200 x 100,003 x 64 54 and 95.  The rule goes by all rows,
// those that take no part among them: how many do is known on the device only, and what is laid out and launched is not.
constexpr int64_t kFewRowsTwice = 64;

int64_t tiles_of(int64_t n, int64_t of) { return (n + of - 1) / of; }

// Pairs of blocks where the product is bound by its arithmetic and there are tiles enough for every pair.
bool pair_rows(int64_t n, int64_t tiles, int64_t steps) { return steps > 2 && n >= 256 && n / 256 * tiles >= sm_count() / 2; }

Layout layout_of(const mt_vocab_loss& c, bool backward) {
  Layout l{};
  l.parts = c.dtype == MT_F32 ? 3 : 1;
  l.dp = l.wp = (int)part_columns(c.dim, l.parts);
  l.copy_w = c.dtype == MT_F32 || c.dim % 8 != 0 || (c.vocab > 1 && c.ldw % 8 != 0) || !is_aligned(c.w, 16);
  l.rows = tiles_of(c.n, 256) * 256;
  l.top = c.top > 0 ? c.top : 1;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align_up(bytes, 256);
    return here;
  };
  l.mask = take((size_t)tiles_of(c.n, 32) * 4);
  l.live = take(4);
  l.chunks = take(8);
  l.cut = take(16);
  l.pos = take((size_t)c.n * 4);
  l.xs = take((size_t)l.rows * l.parts * l.dp * 2);
  l.ids = take((size_t)c.n * l.top * 4);
  l.share = take((size_t)c.n * l.top * 4);
  l.entropy = take(c.top > 0 ? (size_t)c.n * 4 : 0);
  if (l.copy_w) l.w = take((size_t)c.vocab * l.parts * l.wp * 2);
  const int sms = std::max(1, sm_count());
  const int64_t runs_v = tiles_of(c.vocab, kLongest), runs_n = tiles_of(c.n, kLongest);  // what the sums over them are cut into at least
  if (!backward) {
    l.max_chunks = (int)(16 * sms / (l.rows / 128) + 1);
    l.picked = take((size_t)c.n * l.top * 4);
    l.part = take((size_t)kNarrowTeams * l.max_chunks * l.rows * 8);
    if (c.smoothing > 0.0f) l.sum_z = take((size_t)kNarrowTeams * l.max_chunks * l.rows * 4);
  } else if (c.dtype == MT_BF16 && c.dim <= kFusedColumns && c.n > kFewRowsTwice) {
    // room for as many runs as give every block eight units, of the tiles that are cut at all
    l.fused = true;
    const int64_t rt = tiles_of(c.n, kFusedTile), vt = tiles_of(c.vocab, kFusedTile);
    l.coef = take((size_t)c.n * 16);
    // (cut for kLongest: up to 32 runs within 256 MiB, so that their last round is a full one)
    const auto cuts = [&](int64_t least, int64_t rows) {
      return least > 1 ? std::max(least, std::min<int64_t>(32, (int64_t)((256 << 20) / ((size_t)rows * c.dim * 4)))) : 1;
    };
    l.runs_dx = (int)std::max(std::min<int64_t>(vt, rt < sms ? 8 * sms / rt + 1 : 4), cuts(runs_v, l.rows));
    l.dx = take((size_t)l.runs_dx * l.rows * c.dim * 4);
    l.whole = runs_n > 1 ? 0 : (int)(vt / sms * sms);
    l.runs_dw = vt > l.whole ? (int)std::max(std::min<int64_t>(rt, 8 * sms / (vt - l.whole) + 1), cuts(runs_n, vt * kFusedTile)) : 0;
    l.dw = take((size_t)l.runs_dw * (vt - l.whole) * kFusedTile * c.dim * 4);
  } else {
    l.dz_parts = c.dtype == MT_F32 ? 3 : c.n <= kFewRowsTwice ? 2 : 1;
    l.max_chunks = 1 << 30;
    const int64_t most = std::max<int64_t>(1, (int64_t)(kPieceBytes / ((size_t)l.rows * l.dz_parts * 512)));
    const int64_t pieces = tiles_of(tiles_of(c.vocab, 256), most);
    l.piece = tiles_of(tiles_of(c.vocab, 256), pieces) * 256;
    l.coef = take((size_t)c.n * 16);
    l.dz = take((size_t)l.rows * l.dz_parts * l.piece * 2);
    const int bn = sum_width(c.dim, c.dtype == MT_F32);
    const int64_t ct = tiles_of(c.dim, bn);
    // room for runs of the contraction: eight units a block, no run shorter than 8 steps, 256 MiB of dx; and as many as kLongest
    // asks for (a piece's rows times its entries are bounded, so these take 256 MiB for 8192 columns too)
    const int64_t rt = l.rows / 128;
    l.runs_dx = (int)std::max<int64_t>(1, std::min({8 * sms / (rt * ct) + 1, l.piece / 512, (int64_t)((256 << 20) / ((size_t)l.rows * c.dim * 4))}));
    l.runs_dx = (int)std::max<int64_t>(l.runs_dx, tiles_of(l.piece, kLongest));
    l.dx = take((size_t)l.runs_dx * l.rows * c.dim * 4);
    // dW: only of the tiles behind the whole rounds, fewer than there are blocks
    const int64_t tail = std::min<int64_t>(l.piece / 128 * ct, sms + ct);
    l.runs_dw = (int)std::max<int64_t>(1, std::min<int64_t>(8 * sms / tail + 1, tiles_of(c.n, 512)));
    l.dw_rows = std::min<int64_t>(l.piece, tiles_of(tail, ct) * 256);
    if (runs_n > 1) {  // all of the piece comes in runs
      l.dw_rows = l.piece;
      l.runs_dw = (int)std::max(runs_n, std::min<int64_t>(l.runs_dw, (int64_t)((256 << 20) / ((size_t)l.piece * c.dim * 4))));
    }
    l.dw = take((size_t)l.runs_dw * l.dw_rows * c.dim * 4);
  }
  l.total = at;
  return l;
}

int check(const mt_vocab_loss* c) {
  if (c == nullptr || (c->dtype != MT_F32 && c->dtype != MT_BF16)) return MT_EINVAL;
  if (c->n < 0 || c->n > MT_MAX_BLOCK_ROWS || c->vocab < 1 || c->vocab > MT_MAX_BLOCK_ROWS) return MT_EINVAL;
  if (c->dim < 1 || c->dim > MT_MAX_BLOCK_DIM || c->top < 0 || c->top > MT_MAX_TOP) return MT_EINVAL;
  if (!(c->scale > 0.0f && c->scale <= 1e30f) || !(c->smoothing >= 0.0f && c->smoothing < 1.0f) || !(c->z_loss >= 0.0f && c->z_loss <= 1e30f))
    return MT_EINVAL;
  if (c->top > 0 && (c->smoothing != 0.0f || c->z_loss != 0.0f)) return MT_EINVAL;
  if (c->id_bytes != 4 && c->id_bytes != 8) return MT_EINVAL;
  if (c->top > 0 && c->teacher_dtype != MT_F32 && c->teacher_dtype != MT_BF16) return MT_EINVAL;
  if (!is_aligned(c->status, 4) || !rows_ok(c->w, c->ldw, c->dim, c->dtype)) return MT_EINVAL;
  if (c->n > 0) {
    if (!rows_ok(c->x, c->ldx, c->dim, c->dtype) || c->targets == nullptr || !is_aligned(c->targets, c->id_bytes)) return MT_EINVAL;
    if (c->top > 0 && (c->teacher == nullptr || !is_aligned(c->teacher, elem_bytes(c->teacher_dtype)))) return MT_EINVAL;
  }
  return MT_OK;
}

void inputs_of(const mt_vocab_loss& c, Regions& all) {
  all.in(Rows{const_cast<void*>(c.x), c.ldx, nullptr, nullptr}, c.n, c.dim, c.dtype);
  all.in(Rows{const_cast<void*>(c.w), c.ldw, nullptr, nullptr}, c.vocab, c.dim, c.dtype);
  const size_t pairs = (size_t)c.n * (c.top > 0 ? c.top : 1);
  all.in(whole_region(c.targets, pairs * c.id_bytes));
  if (c.top > 0) all.in(whole_region(c.teacher, pairs * elem_bytes(c.teacher_dtype)));
}

// The rows that take part, and W as the tensor cores take it.
cudaError_t launch_rows(const mt_vocab_loss& c, const Layout& l, char* ws, const float* dloss, const float* lse, cudaStream_t s) {
  VocabRows r{};
  r.n = c.n;
  r.vocab = c.vocab;
  r.dim = c.dim;
  r.top = l.top;
  r.wide_ids = c.id_bytes == 8;
  r.teacher16 = c.teacher_dtype == MT_BF16;
  r.targets = c.targets;
  r.teacher = c.teacher;
  r.status = c.status;
  r.scale = c.scale;
  r.smoothing = c.smoothing;
  r.z_loss = c.z_loss;
  r.x = c.x;
  r.ldx = c.ldx;
  r.mask = reinterpret_cast<uint32_t*>(ws + l.mask);
  r.live = reinterpret_cast<int*>(ws + l.live);
  r.pos = reinterpret_cast<int*>(ws + l.pos);
  r.xs = reinterpret_cast<__nv_bfloat16*>(ws + l.xs);
  r.dp = l.dp;
  r.ids = reinterpret_cast<int*>(ws + l.ids);
  r.share = reinterpret_cast<float*>(ws + l.share);
  r.entropy = reinterpret_cast<float*>(ws + l.entropy);
  r.dloss = dloss;
  r.lse = lse;
  r.coef = dloss != nullptr ? reinterpret_cast<float4*>(ws + l.coef) : nullptr;
  const bool mark = c.top > 0 ? c.n * l.top <= kMarkPairs : c.n <= kMarkRows;
  cudaError_t e = cudaSuccess;
  if (!mark) {
    MT_LAUNCH("k_vocab_mark", s);
    if (c.top > 0) k_vocab_mark<true><<<grid_for(tiles_of(c.n, 32) * 256, 256, 8), 256, 0, s>>>(r);
    else k_vocab_mark<false><<<grid_for(c.n, 256, 8), 256, 0, s>>>(r);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  {
    const bool al = rows_wide(Rows{const_cast<void*>(c.x), c.n <= 1 ? c.dim : c.ldx, nullptr, nullptr}, c.dim, c.dtype);
    const size_t smem = c.top > 0 ? 8 * list_bytes(c.top) : 0;
    const int grid = grid_for(tiles_of(c.n, 32) * kRowBlocks * 256, 256, 8);
    static SmemLimit limit[24];
    auto go = [&](auto kernel, int i) {
      const cudaError_t le = limit[i].allow(kernel, 8 * list_bytes(MT_MAX_TOP));
      if (le != cudaSuccess) return le;
      MT_LAUNCH("k_vocab_rows", s);
      if (!mark) return launch_following(kernel, grid, 256, smem, s, r);
      kernel<<<grid, 256, smem, s>>>(r);
      return cudaGetLastError();
    };
    auto of = [&](auto few, auto list) {
      constexpr bool M = decltype(few)::value;
      constexpr int L = decltype(list)::value, at = M + 2 * L;
      if (c.dtype == MT_F32) return al ? go(k_vocab_rows<float, true, M, L>, at) : go(k_vocab_rows<float, false, M, L>, 6 + at);
      return al ? go(k_vocab_rows<__nv_bfloat16, true, M, L>, 12 + at) : go(k_vocab_rows<__nv_bfloat16, false, M, L>, 18 + at);
    };
    auto by_list = [&](auto few) {
      if (c.top == 0) return of(few, std::integral_constant<int, kTarget>{});
      return c.top <= kRankPairs ? of(few, std::integral_constant<int, kCounted>{}) : of(few, std::integral_constant<int, kSorted>{});
    };
    e = mark ? by_list(std::true_type{}) : by_list(std::false_type{});
  }
  if (e == cudaSuccess && l.copy_w)
    e = launch_parts(c.w, c.vocab <= 1 ? c.dim : c.ldw, 1, c.vocab, c.vocab, c.dim, c.dtype, reinterpret_cast<__nv_bfloat16*>(ws + l.w), s);
  return e;
}

struct Weights {
  const char* data;
  uint64_t width, ld;  // columns and stride, elements
};
Weights weights_of(const mt_vocab_loss& c, const Layout& l, const char* ws) {
  const uint64_t width = (uint64_t)l.parts * l.wp;
  if (l.copy_w) return {ws + l.w, width, width};
  return {static_cast<const char*>(c.w), width, c.vocab <= 1 ? width : (uint64_t)c.ldw};
}

LogitParams logits_of(const mt_vocab_loss& c, const Layout& l, char* ws) {
  LogitParams p{};
  p.passes = l.parts == 3 ? 6 : 1;
  p.a_part = l.dp;
  p.b_part = l.wp;
  p.promote = 1 << 30;
  p.steps = (int)tiles_of(l.dp, 64);
  p.kept = l.parts * p.steps <= kLogitKept ? l.parts * p.steps : 0;
  p.status = c.status;
  p.rows = LiveRows{reinterpret_cast<int*>(ws + l.live), reinterpret_cast<int*>(ws + l.ids), reinterpret_cast<float*>(ws + l.share), l.top};
  p.max_chunks = l.max_chunks;
  p.scale2 = c.scale * kLog2e;
  p.stride = l.rows;
  return p;
}

}  // namespace
}  // namespace mt

extern "C" {

size_t mt_vocab_loss_workspace_bytes(const mt_vocab_loss* c, int backward) {
  using namespace mt;
  if (check(c) != MT_OK) return 0;
  if (c->n == 0) return 256;
  return layout_of(*c, backward != 0).total;
}

int mt_vocab_loss_forward(const mt_vocab_loss* c, float* loss, float* lse, void* ws, size_t ws_bytes, mt_stream stream) {
  using namespace mt;
  const int rc = check(c);
  if (rc != MT_OK) return rc;
  if (c->n == 0) return MT_OK;
  if (loss == nullptr || lse == nullptr || !is_aligned(loss, 4) || !is_aligned(lse, 4)) return MT_EINVAL;
  const Layout l = layout_of(*c, false);
  if (ws == nullptr || !is_aligned(ws, 256) || ws_bytes < l.total) return MT_ENOSPACE;
  Regions all;
  inputs_of(*c, all);
  all.out(whole_region(loss, (size_t)c->n * 4));
  all.out(whole_region(lse, (size_t)c->n * 4));
  all.out(whole_region(ws, l.total));
  if (all.clash()) return MT_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* base = static_cast<char*>(ws);
  cudaError_t e = launch_rows(*c, l, base, nullptr, nullptr, s);
  if (e != cudaSuccess) return MT_ECUDA;
  LogitParams p = logits_of(*c, l, base);
  p.v0 = 0;
  p.columns = c->vocab;
  p.tiles = (int)tiles_of(c->vocab, 256);
  p.part = reinterpret_cast<float2*>(base + l.part);
  p.sum_z = c->smoothing > 0.0f ? reinterpret_cast<float*>(base + l.sum_z) : nullptr;
  p.picked = reinterpret_cast<float*>(base + l.picked);
  p.chunks = reinterpret_cast<int*>(base + l.chunks);
  const bool narrow = c->dtype == MT_BF16 && c->dim <= kFusedColumns;
  const bool pair = !narrow && c->dtype == MT_BF16 && pair_rows(c->n, tiles_of(c->vocab, 256), p.steps);
  const Weights w = weights_of(*c, l, base);
  CUtensorMap a, b;
  const uint64_t width = (uint64_t)l.parts * l.dp;
  if (!tc::encode_bf16(&a, 2, base + l.xs, width, l.rows, width, 1, 0, 64, 128)) return MT_ECUDA;
  if (!tc::encode_bf16(&b, 2, w.data, w.width, c->vocab, w.ld, 1, 0, 64, pair || narrow ? 128 : 256)) return MT_ECUDA;
  if (narrow) {
    FusedParams f{};
    f.status = c->status;
    f.rows = p.rows;
    f.vocab = c->vocab;
    f.columns = c->dim;
    f.max_chunks = l.max_chunks;
    f.scale2 = p.scale2;
    f.stats = p.part;
    f.sum_z = p.sum_z;
    f.picked = p.picked;
    f.stride = l.rows;
    f.cut = p.chunks;
    e = launch_narrow_stats(f, a, b, tiles_of(c->n, kFusedTile) * std::min<int64_t>(l.max_chunks, tiles_of(c->vocab, kFusedTile)), s);
  } else {
    e = launch_logit_stats(p, a, b, tiles_of(c->n, pair ? 256 : 128), pair, s);
  }
  if (e != cudaSuccess) return MT_ECUDA;
  VocabLoss q{};
  q.n = c->n;
  q.vocab = c->vocab;
  q.top = l.top;
  q.pos = reinterpret_cast<int*>(base + l.pos);
  q.part = p.part;
  q.sum_z = p.sum_z;
  q.stride = l.rows;
  q.chunks = p.chunks;
  q.teams = narrow ? kNarrowTeams : 2;
  q.picked = p.picked;
  q.share = p.rows.share;
  q.entropy = c->top > 0 ? reinterpret_cast<float*>(base + l.entropy) : nullptr;
  q.scale = c->scale;
  q.smoothing = c->smoothing;
  q.z_loss = c->z_loss;
  q.loss = loss;
  q.lse = lse;
  MT_LAUNCH("k_vocab_loss", s);
  return launch_following(k_vocab_loss, grid_for(c->n * 32, 256, 8), 256, 0, s, q) == cudaSuccess ? MT_OK : MT_ECUDA;
}

int mt_vocab_loss_backward(const mt_vocab_loss* c, const float* dloss, const float* lse, void* dx, int64_t lddx, void* dw, void* ws,
                           size_t ws_bytes, mt_stream stream) {
  using namespace mt;
  const int rc = check(c);
  if (rc != MT_OK) return rc;
  if (dx == nullptr && dw == nullptr) return MT_EINVAL;
  if (c->n > 0) {
    if (dloss == nullptr || lse == nullptr || !is_aligned(dloss, 4) || !is_aligned(lse, 4)) return MT_EINVAL;
    if (dx != nullptr && !rows_ok(dx, lddx, c->dim, c->dtype)) return MT_EINVAL;
  }
  const size_t el = elem_bytes(c->dtype), weights = (size_t)c->vocab * c->dim * el;
  if (!is_aligned(dw, el)) return MT_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (c->n == 0) {
    if (dw == nullptr) return MT_OK;
    Regions all;
    inputs_of(*c, all);
    all.out(whole_region(dw, weights));
    if (all.clash()) return MT_EINVAL;
    return cudaMemsetAsync(dw, 0, weights, s) == cudaSuccess ? MT_OK : MT_ECUDA;
  }
  const Layout l = layout_of(*c, true);
  if (ws == nullptr || !is_aligned(ws, 256) || ws_bytes < l.total) return MT_ENOSPACE;
  Regions all;
  inputs_of(*c, all);
  all.in(whole_region(dloss, (size_t)c->n * 4));
  all.in(whole_region(lse, (size_t)c->n * 4));
  if (dx != nullptr) all.out(Rows{dx, lddx, nullptr, nullptr}, c->n, c->dim, c->dtype);
  if (dw != nullptr) all.out(whole_region(dw, weights));
  all.out(whole_region(ws, l.total));
  if (all.clash()) return MT_EINVAL;
  char* base = static_cast<char*>(ws);
  cudaError_t e = launch_rows(*c, l, base, dloss, lse, s);
  const bool fp32 = c->dtype == MT_F32;
  const Weights w = weights_of(*c, l, base);
  const uint64_t xw = (uint64_t)l.parts * l.dp;
  const int bn = sum_width(c->dim, fp32);
  const int ct = (int)tiles_of(c->dim, bn);
  const int reach = dw != nullptr ? tiles::reach_of(dw, c->dim, c->dim, el) : 0, reach_part = tiles::reach_of(base, c->dim, c->dim, 4);
  int* cut = reinterpret_cast<int*>(base + l.cut);  // of dx, of dW
  if (l.fused && e == cudaSuccess) {
    FusedParams f{};
    f.status = c->status;
    f.rows = logits_of(*c, l, base).rows;
    f.vocab = c->vocab;
    f.columns = c->dim;
    f.scale2 = c->scale * kLog2e;
    f.coef = reinterpret_cast<float4*>(base + l.coef);
    f.reach = reach;
    f.reach_part = reach_part;
    f.out = static_cast<__nv_bfloat16*>(dw);
    CUtensorMap a, b;
    if (!tc::encode_bf16(&a, 2, base + l.xs, xw, l.rows, xw, 1, 0, 64, kFusedTile)) return MT_ECUDA;
    if (!tc::encode_bf16(&b, 2, w.data, w.width, c->vocab, w.ld, 1, 0, 64, kFusedTile)) return MT_ECUDA;
    const int64_t rt = tiles_of(c->n, kFusedTile), vt = tiles_of(c->vocab, kFusedTile);
    if (dx != nullptr) {
      f.max_chunks = l.runs_dx;
      f.cut = cut;
      f.part = reinterpret_cast<float*>(base + l.dx);
      f.stride = l.rows;
      e = launch_fused(false, f, a, b, rt * l.runs_dx, s);
    }
    if (dw != nullptr && e == cudaSuccess) {
      f.max_chunks = std::max(1, l.runs_dw);
      f.whole = l.whole;
      f.cut = cut + 2;
      f.part = reinterpret_cast<float*>(base + l.dw);
      f.stride = (size_t)(vt - l.whole) * kFusedTile;
      e = launch_fused(true, f, a, b, l.whole + (vt - l.whole) * l.runs_dw, s);
      const int64_t tail = c->vocab - (int64_t)l.whole * kFusedTile;
      if (tail > 0 && e == cudaSuccess) e = launch_dw_sum(f.part, f.stride, f.cut, c->vocab, tail, c->dim, c->dtype, dw, s);
    }
  }
  for (int64_t v0 = 0; !l.fused && v0 < c->vocab && e == cudaSuccess; v0 += l.piece) {
    const int64_t columns = std::min<int64_t>(l.piece, c->vocab - v0);
    const char* wv = w.data + (size_t)v0 * w.ld * 2;
    LogitParams p = logits_of(*c, l, base);
    p.v0 = (int)v0;
    if (p.kept > kGradKept) p.kept = 0;
    p.columns = (int)columns;
    p.tiles = (int)tiles_of(columns, 256);
    p.coef = reinterpret_cast<float4*>(base + l.coef);
    p.dz = reinterpret_cast<__nv_bfloat16*>(base + l.dz);
    p.width = (int)(tiles_of(columns, 64) * 64);
    const uint64_t zw = (uint64_t)l.dz_parts * p.width;
    CUtensorMap a, b;
    {
      const bool pair = l.dz_parts == 1 && pair_rows(c->n, tiles_of(columns, 256), p.steps);
      if (!tc::encode_bf16(&a, 2, base + l.xs, xw, l.rows, xw, 1, 0, 64, 128)) return MT_ECUDA;
      if (!tc::encode_bf16(&b, 2, wv, w.width, columns, w.ld, 1, 0, 64, pair ? 128 : 256)) return MT_ECUDA;
      if (l.dz_parts == 1 && !tc::encode_bf16(&p.map_dz, 2, p.dz, zw, l.rows, zw, 1, 0, 64, 32)) return MT_ECUDA;
      e = launch_logit_grad(p, l.dz_parts, a, b, tiles_of(c->n, pair ? 256 : 128), pair, s);
    }
    SumParams q{};
    q.passes = l.dz_parts == 2 ? 2 : 1;
    q.promote = fp32 ? 1 : 1 << 30;
    q.status = c->status;
    q.live = p.rows.count;
    q.a_part = p.width;
    q.columns = c->dim;
    q.ctiles = ct;
    q.reach = reach;
    q.reach_part = reach_part;
    if (dx != nullptr && e == cudaSuccess) {
      const bool pair = bn == 256 && pair_rows(c->n, (int64_t)ct * l.runs_dx, l.piece / 64);  // (the same for every piece)
      if (!tc::encode_bf16(&a, 2, base + l.dz, zw, l.rows, zw, 1, 0, 64, 128)) return MT_ECUDA;
      if (!tc::encode_bf16(&b, 2, wv, w.width, columns, w.ld, 1, 0, 64, 64)) return MT_ECUDA;
      q.b_part = l.wp;
      q.steps = p.width / 64;
      q.usual = (int)(l.piece / 64);
      q.max_runs = l.runs_dx;
      q.cut = cut;
      q.part = reinterpret_cast<float*>(base + l.dx);
      q.stride = l.rows;
      q.add = v0 > 0;
      e = launch_rows_sum(q, fp32, a, b, tiles_of(c->n, pair ? 256 : 128), pair, s);
    }
    if (dw != nullptr && e == cudaSuccess) {
      const bool pair = bn == 256 && pair_rows(columns, (int64_t)ct * l.runs_dw, tiles_of(c->n, 64));
      if (!tc::encode_bf16(&a, 2, base + l.dz, zw, l.rows, zw, 1, 0, 64, 64)) return MT_ECUDA;
      if (!tc::encode_bf16(&b, 2, base + l.xs, xw, l.rows, xw, 1, 0, 64, 64)) return MT_ECUDA;
      q.b_part = l.dp;
      q.rows = (int)columns;
      q.max_runs = l.runs_dw;
      q.cut = cut + 2;
      q.part = reinterpret_cast<float*>(base + l.dw);
      q.stride = l.dw_rows;
      q.add = false;
      q.out = static_cast<char*>(dw) + (size_t)v0 * c->dim * el;
      e = launch_vocab_sum(q, fp32, a, b, tiles_of(columns, pair ? 256 : 128), pair, s);
      if (e == cudaSuccess) e = launch_dw_sum(q.part, q.stride, q.cut, columns, std::min<int64_t>(columns, l.dw_rows), c->dim, c->dtype, q.out, s);
    }
  }
  if (dx != nullptr && e == cudaSuccess) {
    const float* part = reinterpret_cast<const float*>(base + l.dx);
    const int* pos = reinterpret_cast<const int*>(base + l.pos);
    const bool four = c->dim % 4 == 0 && (c->n <= 1 || lddx % 4 == 0) && is_aligned(dx, 4 * el);
    const int grid = grid_for(c->n * (four ? c->dim / 4 : c->dim), 256, 8);
    auto go = [&](auto kernel, auto* to) { return launch_following(kernel, grid, 256, 0, s, part, l.rows, pos, c->n, c->dim, to, lddx, cut); };
    MT_LAUNCH("k_vocab_dx_sum", s);
    if (fp32) e = four ? go(k_vocab_dx_sum<float, true>, static_cast<float*>(dx)) : go(k_vocab_dx_sum<float, false>, static_cast<float*>(dx));
    else e = four ? go(k_vocab_dx_sum<__nv_bfloat16, true>, static_cast<__nv_bfloat16*>(dx)) : go(k_vocab_dx_sum<__nv_bfloat16, false>, static_cast<__nv_bfloat16*>(dx));
  }
  return e == cudaSuccess ? MT_OK : MT_ECUDA;
}

}  // extern "C"
