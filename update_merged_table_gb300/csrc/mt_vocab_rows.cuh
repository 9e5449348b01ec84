// What an epilogue thread knows of its row of logits: device code that the kernels
// of mt_vocab_logits.cu and mt_vocab_fused.cu share.
#pragma once

#include "mt_vocab.cuh"

namespace mt {

__device__ __forceinline__ float exp2_of(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The first `left` of 32 columns, as bits.
__device__ __forceinline__ uint32_t below(int left) { return left >= 32 ? kFull : left <= 0 ? 0u : (1u << left) - 1u; }

// Runs of column tiles for `rt` row tiles on `blocks` blocks (pairs): as many as end the last block soonest, a run's start
// and end counted as `extra` half tiles, and `least` at least.  Every thread calls it.
__device__ __forceinline__ int choose_chunks(int rt, int tiles, int most, int blocks, int extra, int least = 1) {
  __shared__ unsigned long long s_best;
  if (threadIdx.x == 0) s_best = ~0ull;
  __syncthreads();
  unsigned long long best = ~0ull;
  for (int c = threadIdx.x + least; c <= max(least, min(most, tiles)); c += blockDim.x) {
    const long long rounds = ((long long)rt * c + blocks - 1) / blocks;
    const unsigned long long cost = (unsigned long long)rounds * (2 * ((tiles + c - 1) / c) + extra);
    best = min(best, cost << 32 | (unsigned)c);
  }
  if (best != ~0ull) atomicMin(&s_best, best);
  __syncthreads();
  return (int)(uint32_t)s_best;
}

// A row's targets, which lie in ascending order, as its columns come by: one comparison per 32 columns finds them.
struct RowTargets {
  int row, pos, next;  // the next target and its place in the list

  __device__ __forceinline__ void start(const LiveRows& r, int of, int live, int first) {
    row = of;
    pos = 0;
    next = 0x7FFFFFFF;
    if (row >= live) return;
    const int* ids = r.ids + (size_t)row * r.top;
    int lo = 0, hi = r.top;  // targets before `lo` are below `first`, those from `hi` on are not
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (ids[mid] < first) lo = mid + 1;
      else hi = mid;
    }
    pos = lo;
    if (pos < r.top) next = ids[pos];
  }
  __device__ __forceinline__ void advance(const LiveRows& r) {
    ++pos;
    next = pos < r.top ? r.ids[(size_t)row * r.top + pos] : 0x7FFFFFFF;
  }
  // The logits of targets among the 32 columns from col on go to picked.
  __device__ __forceinline__ void pick(const LiveRows& r, int col, const uint32_t (&v)[32], float* picked) {
    while (__any_sync(kFull, next < col + 32)) {
      if (next < col + 32) {
        if (next >= col) {
          const int at = next - col;
          uint32_t z = v[0];
#pragma unroll
          for (int j = 1; j < 32; ++j) z = at == j ? v[j] : z;
          picked[(size_t)row * r.top + pos] = __uint_as_float(z);
        }
        advance(r);
      }
    }
  }
  // Their shares, times `factor`, are taken off the gradients.
  __device__ __forceinline__ void take(const LiveRows& r, int col, float factor, float (&f)[32]) {
    while (__any_sync(kFull, next < col + 32)) {
      if (next < col + 32) {
        if (next >= col) {
          const int at = next - col;
          const float off = factor * r.share[(size_t)row * r.top + pos];
#pragma unroll
          for (int j = 0; j < 32; ++j) f[j] -= at == j ? off : 0.0f;
        }
        advance(r);
      }
    }
  }
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// A row's statistics over the columns it has seen: the largest logit (in base 2) and the sum of 2^(z - that), and (SMOOTH) the
// sum of the logits before the scale.
template <bool SMOOTH>
struct RowStats {
  float top, sum, total;

  __device__ __forceinline__ void clear() {
    top = -INFINITY;
    sum = total = 0.0f;
  }
  // N x 32 columns: their largest, then one exponential each; only the first `left` count.
  template <int N>
  __device__ __forceinline__ void add(uint32_t (&v)[N][32], float scale2, int left) {
    if constexpr (SMOOTH) {
      f32x2 t[2] = {0ull, 0ull};
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 32; j += 2)  // (columns that are not there are zero)
          t[j >> 1 & 1] = add2(t[j >> 1 & 1], pk(__uint_as_float(v[i][j]), __uint_as_float(v[i][j + 1])));
      total += pair_sum(add2(t[0], t[1]));
    }
    if (left < N * 32) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t there = below(left - i * 32);
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (!(there >> j & 1)) v[i][j] = 0xFF800000u;
      }
    }
    float m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = __uint_as_float(v[0][i * 8]);
#pragma unroll
      for (int j = 1; j < 7; j += 2) m[i] = max3(m[i], __uint_as_float(v[0][i * 8 + j]), __uint_as_float(v[0][i * 8 + j + 1]));
      m[i] = fmaxf(m[i], __uint_as_float(v[0][i * 8 + 7]));
#pragma unroll
      for (int n = 1; n < N; ++n)
#pragma unroll
        for (int j = 0; j < 8; j += 2) m[i] = max3(m[i], __uint_as_float(v[n][i * 8 + j]), __uint_as_float(v[n][i * 8 + j + 1]));
    }
    const float now = max3(top, fmaxf(m[0], m[1]) * scale2, fmaxf(m[2], m[3]) * scale2);
    const float off = now == -INFINITY ? 0.0f : now;
    const f32x2 s2 = both(scale2), o2 = both(-off);
    f32x2 s[2] = {0ull, 0ull};
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        const float2 e = upk(fma2(pk(__uint_as_float(v[i][j]), __uint_as_float(v[i][j + 1])), s2, o2));
        s[j >> 1 & 1] = add2(s[j >> 1 & 1], pk(exp2_of(e.x), exp2_of(e.y)));
      }
    sum = fmaf(sum, exp2_of(top - off), pair_sum(add2(s[0], s[1])));
    top = now;
  }
  __device__ __forceinline__ void add(uint32_t (&v)[32], float scale2, int left) {
    add<1>(reinterpret_cast<uint32_t(&)[1][32]>(v), scale2, left);
  }
};

}  // namespace mt
