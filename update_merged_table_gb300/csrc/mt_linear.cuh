// Parameter blocks of the grouped matrix products.
#pragma once

#include "mt_block.cuh"

namespace mt {

constexpr int kMinChunk = 256;  // fewest rows that a group is split into

// C[row, j] = sum over i < I of A[row, i] * w[g * wg + i * wi + j * wj], for the rows of group g; rows in no group
// become zeros.
struct LinearRows {
  long long n;
  int groups;
  const long long* offsets;
  int32_t* status;
  const void* a;
  long long lda;
  const void* w;
  size_t wg, wi, wj;
  void* c;
  long long ldc;
  int I, J, jtiles;
};

// dW[g][m][k] = sum over the rows r of group g of dy[r][m] * x[r][k].
struct LinearWeights {
  long long n;
  int groups;
  const long long* offsets;
  int32_t* status;
  const void* dy;
  long long lddy;
  Rows x;
  int K, M;
  int chunks;     // most chunks the rows are split into (at least the groups)
  int slots;      // most of them that belong to groups of several
  float* part;    // [slots][M][K]: partial products of the groups that have several chunks
  float* dw;      // [groups][M][K]
};

inline size_t weights_smem(int groups) { return (size_t)(groups + 1) * (8 + 4 + 4); }

// The rows of a chunk: the least multiple of 64 (and at least kMinChunk) with which the groups' rows make no more than
// p.chunks chunks and need no more than p.slots partial products.  The kernels give every SM (or pair) the same number
// of chunk tiles, so the chunks' number has to fit a whole number of rounds however ragged the groups are; equal chunks
// then make equal rounds.  Every thread calls it.
__device__ __forceinline__ int choose_chunk(const LinearWeights& p, const long long* s_off, int* s_value) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x, G = p.groups;
    int longest = 0;
    for (int i = lane; i < G; i += 32) longest = max(longest, (int)((s_off[i + 1] - s_off[i] + 63) / 64));
    longest = __reduce_max_sync(kFull, longest);
    int lo = kMinChunk / 64, hi = max(lo, longest);  // in units of 64 rows; hi always fits (one chunk per group)
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      int count = 0, split = 0;
      for (int i = lane; i < G; i += 32) {
        const int c = ((int)((s_off[i + 1] - s_off[i] + 63) / 64) + mid - 1) / mid;
        count += c;
        split += c > 1 ? c : 0;
      }
      count = __reduce_add_sync(kFull, count);
      split = __reduce_add_sync(kFull, split);
      if (count <= p.chunks && split <= p.slots) hi = mid;
      else lo = mid + 1;
    }
    if (lane == 0) *s_value = lo * 64;
  }
  __syncthreads();
  return *s_value;
}

// s_slot[g]: partial products of the groups before g that have more than one chunk; after count_tiles, by every thread.
__device__ __forceinline__ void count_slots(const int* s_cum, int G, int* s_slot) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int carry = 0;
    for (int i0 = 0; i0 < G; i0 += 32) {
      const int i = i0 + lane;
      const int c = i < G ? s_cum[i + 1] - s_cum[i] : 0;
      const int t = c > 1 ? c : 0;
      const int inc = warp_sum_scan(t, lane);
      if (i < G) s_slot[i] = carry + inc - t;
      carry += __shfl_sync(kFull, inc, 31);
    }
    if (lane == 0) s_slot[G] = carry;
  }
  __syncthreads();
}

// Where chunk c (of group g) puts its product: dW itself when the group has no other chunk, else its slot.
__device__ __forceinline__ float* weights_out(const LinearWeights& p, const int* s_cum, const int* s_slot, int g, int c) {
  const size_t size = (size_t)p.M * p.K;
  if (s_cum[g + 1] - s_cum[g] == 1) return p.dw + (size_t)g * size;
  return p.part + (size_t)(s_slot[g] + c - s_cum[g]) * size;
}

// Zeros for the rows in no group, by the threads [0, threads) of every block.
template <typename T>
__device__ __forceinline__ void zero_outside(const long long* s_off, int G, long long n, T* c, long long ldc, int J,
                                             int threads, int thread) {
  const long long before = s_off[0], outside = before + (n - s_off[G]);
  for (long long q = (long long)blockIdx.x * threads + thread; q < outside * J; q += (long long)gridDim.x * threads) {
    const long long o = q / J;
    const long long row = o < before ? o : o - before + s_off[G];
    c[row * ldc + (q - o * J)] = from_f<T>(0.0f);
  }
}

// The tensor-core forms (mt_linear_tc.cu): bf16, widths and strides in multiples of 8, rows on 16 bytes.
bool linear_rows_fits_tc(const LinearRows& p);
cudaError_t launch_linear_rows_tc(const LinearRows& p, cudaStream_t s);
bool linear_weights_fits_tc(const LinearWeights& p);
cudaError_t launch_linear_weights_tc(const LinearWeights& p, cudaStream_t s);

}  // namespace mt
