// Parameter blocks of the grouped matrix products.
#pragma once

#include "mt_block.cuh"

namespace mt {

constexpr int kMinChunk = 256;  // fewest rows of a chunk that a group is split into
constexpr int kSplits = 32;     // ways of splitting that choose_chunk weighs at a time

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
  int tiles;        // tiles of dW (of the kernel that runs)
  int units;        // blocks (pairs) that there are to walk over them
  float slot_cost, round_cost, sums_cost;  // what a partial product, a tile's end and the sums' launch cost, in units of
                                           // 64 rows of a tile
  int slots;        // partial products there is room for
  int* chosen;      // [1] workspace: the rows of a chunk, as the products chose them, for their sums
  float* part;    // [slots][M][K]: partial products of the groups that have several chunks
  float* dw;      // [groups][M][K]
};

// Dynamic shared memory for the offsets and what is derived from them.
inline size_t rows_smem(int groups) { return (size_t)(groups + 1) * (8 + 4); }
inline size_t weights_smem(int groups) { return (size_t)(groups + 1) * (8 + 4 * 4); }

// The rows of a chunk.  A group may be split into chunks whose products are summed afterwards, so that every block (pair)
// gets about the same work however ragged the groups are; a partial product costs a write and a read of dW's size.  What
// is weighed is the longest group in 1, 2, ... kSplits equal chunks, by the time of the last block in units of 64 rows:
// rounds of tiles of that many rows, or what a block has on average plus a part of a tile where the rounds differ in
// length (plan_chunks deals them out by length), and per round the tile's last read-out and store.  Where kSplits chunks of
// the longest group are still longer than that average (a long group, few tiles), as many finer splits follow, in even ratios
// up to the partial products that there is room for: one group of 1,970,003 x 64 x 64 398 us with kSplits chunks, 128 with
// these.  Every thread calls it, after load_offsets.
struct ChunkChoice {
  int count[kSplits], split[kSplits];  // chunks; those of groups that have several
  int longest, rows, chunk;            // in units of 64 rows, and in rows
  bool finer;
};
__device__ __forceinline__ int choose_chunk(const LinearWeights& p, const long long* s_off, ChunkChoice& c) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  auto units_of = [&](int g) { return (int)((s_off[g + 1] - s_off[g] + 63) / 64); };
  if (warp == 0) {
    int longest = 0, rows = 0;
    for (int g = lane; g < p.groups; g += 32) {
      const int u = units_of(g);
      longest = max(longest, u);
      rows += u;
    }
    longest = __reduce_max_sync(kFull, longest);
    rows = __reduce_add_sync(kFull, rows);
    c.count[lane] = c.split[lane] = 0;
    if (lane == 0) {
      c.longest = longest;
      c.rows = rows;
    }
  }
  float least = 3.0e38f;  // what the chunk chosen so far costs
  for (int pass = 0; pass < 2; ++pass) {
    __syncthreads();
    const int parts = pass == 0 ? lane + 1 : (int)(kSplits * exp2f(log2f((float)p.slots / kSplits) * (float)(lane + 1) / 32.0f));
    const int s = max(kMinChunk / 64, (c.longest + parts - 1) / parts);  // this lane's chunk
    const float inv = 1.0f / (float)s;
    int count = 0, split = 0;
    for (int g = warp; g < p.groups; g += warps) {
      const int u = units_of(g);
      int k = (int)((float)u * inv);  // within one of u / s
      k += (k + 1) * s <= u;
      k -= k * s > u;
      k += k * s < u;  // rounded up
      count += k;
      split += k > 1 ? k : 0;
    }
    atomicAdd(&c.count[lane], count);  // integers: any order gives the same sum
    atomicAdd(&c.split[lane], split);
    __syncthreads();
    if (warp == 0) {
      const float rounds = ceilf((float)c.count[lane] * (float)p.tiles / (float)p.units);
      const float mean = (float)c.rows * (float)p.tiles / (float)p.units;
      const int sp = c.split[lane];
      float cost = fmaxf(fmaxf(mean, (float)min(s, c.longest)), fminf(rounds * (float)s, mean + 0.35f * (float)s)) + rounds * p.round_cost +
                   (float)sp * p.slot_cost + (sp > 0 ? p.sums_cost : 0.0f);
      if (sp > p.slots) cost = 3.0e38f;  // lane 0 of the first pass splits nothing: it always has room
      int best = lane;
      for (int o = 16; o > 0; o >>= 1) {  // the cheapest, of equals the one that splits least
        const float oc = __shfl_xor_sync(kFull, cost, o);
        const int ob = __shfl_xor_sync(kFull, best, o);
        if (oc < cost || (oc == cost && ob < best)) {
          cost = oc;
          best = ob;
        }
      }
      const int chosen = __shfl_sync(kFull, s, best) * 64;
      const int finest = __shfl_sync(kFull, s, 31);
      c.count[lane] = c.split[lane] = 0;
      if (lane == 0) {
        if (cost < least) c.chunk = chosen;
        c.finer = p.slots > kSplits && finest > kMinChunk / 64 && (float)finest > mean;
      }
      least = fminf(least, cost);
    }
    __syncthreads();
    if (!c.finer) break;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.chosen = c.chunk;
  return c.chunk;
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

// The chunks of dW's rows and the order in which their tiles are dealt out.  A group's chunks are equal; the groups come
// by the length of their chunks, longest first, and every other round of tiles is dealt backwards, so that the blocks'
// sums come out near one another.
constexpr int kSortGroups = 256;  // more groups than this make tiles enough to even out as they come
struct Plan {
  const long long* off;  // [groups + 1] rows
  int* cum;              // [groups + 1] chunks before each group
  int* slot;             // [groups + 1] partial products before each group
  int* order;            // [groups] the groups as they are dealt
  int* ocum;             // [groups + 1] chunks before each place of the order
};
struct Chunk {
  int g, index;          // its group, and which of the group's chunks it is
  long long first, last; // its rows
};

__device__ __forceinline__ Plan plan_in(long long* s_off, int G) {
  int* p = reinterpret_cast<int*>(s_off + G + 1);
  return Plan{s_off, p, p + (G + 1), p + 2 * (G + 1), p + 3 * (G + 1)};
}
// Units of 64 rows in each of group g's chunks.
__device__ __forceinline__ int chunk_units(const Plan& q, int g) {
  const int c = q.cum[g + 1] - q.cum[g], u = (int)((q.off[g + 1] - q.off[g] + 63) / 64);
  return c > 0 ? (u + c - 1) / c : 0;
}

// Fills the plan (q.off is there already); every thread calls it.
__device__ __forceinline__ void plan_chunks(const LinearWeights& p, const Plan& q, ChunkChoice& choice) {
  const int G = p.groups, chunk = choose_chunk(p, q.off, choice);
  if (G <= 32) {  // a lane per group: all in one warp, without waiting for the others in between
    if (threadIdx.x < 32) {
      const int lane = threadIdx.x;
      const bool on = lane < G;
      const int u = on ? (int)((q.off[lane + 1] - q.off[lane] + 63) / 64) : 0, s = chunk / 64;
      const int c = (u + s - 1) / s, split = c > 1 ? c : 0;
      const int before = warp_sum_scan(c, lane), slots = warp_sum_scan(split, lane);
      const int e = on ? (c > 0 ? (u + c - 1) / c : 0) : -1;
      int rank = 0;
      for (int j = 0; j < G; ++j) {
        const int ej = __shfl_sync(kFull, e, j);
        rank += ej > e || (ej == e && j < lane);
      }
      if (on) {
        q.cum[lane] = before - c;
        q.slot[lane] = slots - split;
        q.order[rank] = lane;
        q.ocum[rank] = c;
      }
      if (lane == 31) {
        q.cum[G] = q.ocum[G] = before;
        q.slot[G] = slots;
      }
      __syncwarp();
      const int oc = on ? q.ocum[lane] : 0, obefore = warp_sum_scan(oc, lane);
      __syncwarp();
      if (on) q.ocum[lane] = obefore - oc;
    }
    __syncthreads();
    return;
  }
  count_tiles(q.off, G, chunk, q.cum);
  count_slots(q.cum, G, q.slot);
  if (G <= kSortGroups) {
    for (int g = threadIdx.x; g < G; g += blockDim.x) q.ocum[g] = chunk_units(q, g);
    __syncthreads();
    for (int g = threadIdx.x; g < G; g += blockDim.x) {
      const int e = q.ocum[g];
      int rank = 0;
      for (int j = 0; j < G; ++j) rank += q.ocum[j] > e || (q.ocum[j] == e && j < g);
      q.order[rank] = g;
    }
  } else {
    for (int g = threadIdx.x; g < G; g += blockDim.x) q.order[g] = g;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int carry = 0;
    for (int i0 = 0; i0 < G; i0 += 32) {
      const int i = i0 + lane, g = i < G ? q.order[i] : 0;
      const int c = i < G ? q.cum[g + 1] - q.cum[g] : 0;
      const int inc = warp_sum_scan(c, lane);
      if (i < G) q.ocum[i] = carry + inc - c;
      carry += __shfl_sync(kFull, inc, 31);
    }
    if (lane == 0) q.ocum[G] = carry;
  }
  __syncthreads();
}

// The c-th chunk as they are dealt.
__device__ __forceinline__ Chunk chunk_of(const Plan& q, int G, int c) {
  const int place = tile_group(q.ocum, G, c), g = q.order[place];
  Chunk x;
  x.g = g;
  x.index = c - q.ocum[place];
  const int rows = chunk_units(q, g) * 64;
  x.first = q.off[g] + (long long)x.index * rows;
  x.last = min(x.first + rows, q.off[g + 1]);
  return x;
}

// The tile that block `unit` of `units` takes in round r (it may lie past the last one).
__device__ __forceinline__ long long dealt(long long r, int unit, int units) {
  return r * units + ((r & 1) != 0 ? units - 1 - unit : unit);
}

// Where a chunk puts its product: dW itself when the group has no other chunk, else its slot.
__device__ __forceinline__ float* weights_out(const LinearWeights& p, const Plan& q, const Chunk& c) {
  const size_t size = (size_t)p.M * p.K;
  if (q.cum[c.g + 1] - q.cum[c.g] == 1) return p.dw + (size_t)c.g * size;
  return p.part + (size_t)(q.slot[c.g] + c.index) * size;
}

// Blocks (pairs) of a launch: no more than there can be tiles (each then has one, as it would of a larger launch).
inline int weights_blocks(const LinearWeights& p) {
  const long long chunks = (p.n < p.groups ? p.n : p.groups) + p.n / kMinChunk;  // at most
  return (int)(chunks * p.tiles < p.units ? chunks * p.tiles : p.units);
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

// How a dW of this shape is cut into tiles, and over how many blocks (pairs, if it may be pairs) they are dealt.
struct Cut {
  int bn;        // columns of dy in a tile (rows of dW)
  bool pair;     // tiles of 256 columns of x by pairs of blocks, else of 128
  int tiles, units;
};
Cut cut_of(int64_t n, int32_t groups, int32_t k, int32_t m, bool pairs);

// The tensor-core forms (mt_linear_tc.cu): bf16, widths and strides in multiples of 8, rows on 16 bytes.
bool linear_rows_fits_tc(const LinearRows& p);
cudaError_t launch_linear_rows_tc(const LinearRows& p, cudaStream_t s);
bool linear_weights_fits_tc(const LinearWeights& p);
cudaError_t launch_linear_weights_tc(const LinearWeights& p, const Cut& cut, cudaStream_t s);

}  // namespace mt
