// Matrix products grouped by ragged row segments (features, or experts):
//
//   forward   y_i  = W_g x_i             W [groups, out, in]
//   backward  dx_i = W_g^T dy_i          dW_g = sum over the group's rows of dy_i x_i^T
//
// This file holds the entry points and the kernels that take every type, width,
// stride and alignment on the fp32 pipes:
//  k_linear_rows     forward and dx: a 128 x 64 tile of one group's rows per
//                    block, both operands staged in shared memory as fp32.
//  k_linear_few      forward of a row or two per group.
//  k_linear_weights  dW: a 128 x 64 tile of one group's dW over one chunk of its
//                    rows; x may come in 8 bits (its values are read as they
//                    stand, exact in fp32).
//  k_linear_sums     dW of the groups whose rows were split over several chunks,
//                    from the chunks' partial products in chunk order (no
//                    atomics: the sum has one order), and zeros for empty groups.
//
// The fp32 pipes bound the tiles (200,000 x 128 to 256 in fp32: 305 us, 43
// TFLOP/s; dW 260 us, 50, and 35 of sums), shared memory and its latency where
// the contraction is short (65,536 x 32 to 128: 22 us).  Alignment chooses the VEC
// form: 53,166 x 32 to 207 columns 45 us, to 208 columns 31.
#include <algorithm>

#include "mt_linear.cuh"

namespace mt {
namespace {

constexpr int kTM = 128, kTN = 64;  // a tile: rows (of C, or of dW) by columns
constexpr int kI = 16;              // contraction per step
constexpr int kThreadsL = 256;      // a thread holds 8 x 4 values of the tile

// Both operands of a step in shared memory, contraction first.
struct Steps {
  float a[kI][kTM + 4], b[kI][kTN + 4];
};

// acc += a^T b over one step.  A thread's eight rows are four pairs (one instruction for two products); its four columns
// come one by one.
__device__ __forceinline__ void multiply(const Steps& s, int tx, int ty, f32x2 (&acc)[4][4]) {
#pragma unroll
  for (int i = 0; i < kI; ++i) {
    const ulonglong2 a0 = *reinterpret_cast<const ulonglong2*>(&s.a[i][ty * 8]);
    const ulonglong2 a1 = *reinterpret_cast<const ulonglong2*>(&s.a[i][ty * 8 + 4]);
    const float4 b = *reinterpret_cast<const float4*>(&s.b[i][tx * 4]);
    const f32x2 a[4] = {a0.x, a0.y, a1.x, a1.y}, c[4] = {both(b.x), both(b.y), both(b.z), both(b.w)};
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[u][v] = fma2(a[u], c[v], acc[u][v]);
  }
}

// Four neighbouring elements of a row (zeros from `left` on); VEC: one access.
template <typename T, bool VEC>
__device__ __forceinline__ float4 load4(const T* p, int left) {
  float f[4];
  if (VEC) {
    if (left <= 0) return make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if constexpr (sizeof(T) == 4) return __ldg(reinterpret_cast<const float4*>(p));
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xFFFF0000u));
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = j < left ? to_f<T>(__ldg(p + j)) : 0.0f;
  return make_float4(f[0], f[1], f[2], f[3]);
}

// ---- forward and dx ----------------------------------------------------------------
//
// C[row, j] = sum over i < I of A[row, i] * W_g(i, j), with W_g(i, j) = w[g * wg + i * wi + j * wj]; one of wi and wj is
// 1.  The next step's operands are on their way to registers while one is multiplied.  VEC: widths and strides are
// multiples of four elements and everything starts on four.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreadsL) k_linear_rows(const LinearRows p) {
  extern __shared__ long long s_off[];
  __shared__ __align__(16) Steps s;
  int* s_cum = reinterpret_cast<int*>(s_off + p.groups + 1);
  load_offsets(p.offsets, p.groups, p.n, s_off, p.status);
  count_tiles(s_off, p.groups, kTM, s_cum);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const T* A = static_cast<const T*>(p.a);
  T* C = static_cast<T*>(p.c);
  const bool across = p.wi != 1;  // W's rows run along j (else along i)

  zero_outside<T>(s_off, p.groups, p.n, C, p.ldc, p.J, kThreadsL, tid);

  const long long total = (long long)s_cum[p.groups] * p.jtiles;
  for (long long t = blockIdx.x; t < total; t += gridDim.x) {
    const int rt = (int)(t / p.jtiles), j0 = (int)(t - (long long)rt * p.jtiles) * kTN;
    const int g = tile_group(s_cum, p.groups, rt);
    const long long r0 = s_off[g] + (long long)(rt - s_cum[g]) * kTM;
    const int rows = (int)min((long long)kTM, s_off[g + 1] - r0);
    const T* W = static_cast<const T*>(p.w) + (size_t)g * p.wg;
    // this thread's four-element pieces: two of A (rows ar and ar + 64), one of W
    const int ar = tid >> 2, ai = (tid & 3) * 4;
    const int wr = across ? tid >> 4 : tid >> 2, wc = across ? (tid & 15) * 4 : (tid & 3) * 4;  // W: row i or j, place in it
    float4 ra[2], rw;
    auto fetch = [&](int i0) {
#pragma unroll
      for (int q = 0; q < 2; ++q)
        ra[q] = load4<T, VEC>(A + row_offset(r0 + ar + q * 64, p.lda) + i0 + ai, ar + q * 64 < rows ? p.I - i0 - ai : 0);
      if (across) rw = load4<T, VEC>(W + (size_t)(i0 + wr) * p.wi + j0 + wc, i0 + wr < p.I ? p.J - j0 - wc : 0);
      else rw = load4<T, VEC>(W + (size_t)(j0 + wr) * p.wj + i0 + wc, j0 + wr < p.J ? p.I - i0 - wc : 0);
    };
    f32x2 acc[4][4] = {};
    fetch(0);
    for (int i0 = 0; i0 < p.I; i0 += kI) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        s.a[ai][ar + q * 64] = ra[q].x;
        s.a[ai + 1][ar + q * 64] = ra[q].y;
        s.a[ai + 2][ar + q * 64] = ra[q].z;
        s.a[ai + 3][ar + q * 64] = ra[q].w;
      }
      if (across) {
        *reinterpret_cast<float4*>(&s.b[wr][wc]) = rw;
      } else {
        s.b[wc][wr] = rw.x;
        s.b[wc + 1][wr] = rw.y;
        s.b[wc + 2][wr] = rw.z;
        s.b[wc + 3][wr] = rw.w;
      }
      __syncthreads();
      if (i0 + kI < p.I) fetch(i0 + kI);
      multiply(s, tx, ty, acc);
      __syncthreads();
    }
    const int col = j0 + tx * 4;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float2 f[4] = {upk(acc[u][0]), upk(acc[u][1]), upk(acc[u][2]), upk(acc[u][3])};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = ty * 8 + u * 2 + h;
        if (r >= rows) continue;
        T* c = C + row_offset(r0 + r, p.ldc) + col;
        const float4 v = h ? make_float4(f[0].y, f[1].y, f[2].y, f[3].y) : make_float4(f[0].x, f[1].x, f[2].x, f[3].x);
        if (VEC && sizeof(T) == 4) {
          if (col < p.J) *reinterpret_cast<float4*>(c) = v;
        } else if (VEC) {
          if (col < p.J) *reinterpret_cast<uint2*>(c) = make_uint2(bf16x2_of(v.x, v.y), bf16x2_of(v.z, v.w));
        } else {
          const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (col + j < p.J) c[j] = from_f<T>(x[j]);
        }
      }
    }
  }
}

// ---- forward of a few rows --------------------------------------------------------------
//
// A few tokens being served: every weight of the groups that have a row is read once and multiplied by a row or two, so
// the weights' bytes and the latency of one load are all there is.  A warp takes kOuts neighbouring rows of W_g (32 lanes
// by eight columns a step, the loads in flight together) against kFewRows rows of x at once; lanes then join by shuffles.
// A group's further rows are tasks of their own, so a batch costs the same whichever groups its rows are in (512 rows to
// 64 groups of 256 x 128 in fp32 10.4 us, all to one 10.0).  The SMs hold every block at once, three an SM: four would leave
// 64 registers a thread and spills (8 tokens on 8 experts of 512 x 1024 in bf16 5.0 against 4.1 us), and more blocks than
// fit would each read the offsets anew (128 tokens on 64 experts 21.0 against 18.4).
constexpr int kFewRows = 2, kOuts = 4, kFewBlocks = 3;

template <typename T>
__global__ void __launch_bounds__(256, kFewBlocks) k_linear_few(const LinearRows p) {
  extern __shared__ long long s_off[];
  int* s_cum = reinterpret_cast<int*>(s_off + p.groups + 1);
  load_offsets(p.offsets, p.groups, p.n, s_off, p.status);
  count_tiles(s_off, p.groups, kFewRows, s_cum);
  const int lane = threadIdx.x & 31;
  T* C = static_cast<T*>(p.c);
  zero_outside<T>(s_off, p.groups, p.n, C, p.ldc, p.J, blockDim.x, threadIdx.x);
  const int per_tile = (p.J + kOuts - 1) / kOuts;
  const int warps = (gridDim.x * blockDim.x) >> 5;
  for (int t = (blockIdx.x * blockDim.x + threadIdx.x) >> 5; t < s_cum[p.groups] * per_tile; t += warps) {
    const int q = t / per_tile, j0 = (t - q * per_tile) * kOuts, g = tile_group(s_cum, p.groups, q);
    const T* W = static_cast<const T*>(p.w) + (size_t)g * p.wg + (size_t)j0 * p.wj;
    const int outs = min(kOuts, p.J - j0);
    const int r0 = (int)s_off[g] + (q - s_cum[g]) * kFewRows, rows = min(kFewRows, (int)s_off[g + 1] - r0);
    f32x2 acc[kFewRows][kOuts] = {};
#pragma unroll 2
    for (int i = lane * 8; i < p.I; i += 256) {
      Raw8<T> w[kOuts], x[kFewRows];  // every load of the step issued before the first is used
#pragma unroll
      for (int o = 0; o < kOuts; ++o)
        w[o] = load8<T, true>(Rows{const_cast<T*>(W), (int64_t)p.wj, nullptr, nullptr}, o < outs ? o : 0, i >> 3, p.I);
#pragma unroll
      for (int r = 0; r < kFewRows; ++r)
        if (r < rows) x[r] = load8<T, true>(Rows{const_cast<void*>(p.a), p.lda, nullptr, nullptr}, r0 + r, i >> 3, p.I);
#pragma unroll
      for (int r = 0; r < kFewRows; ++r) {
        if (r >= rows) break;
        f32x2 v[4];
        widen8<T>(x[r], false, v);
#pragma unroll
        for (int o = 0; o < kOuts; ++o) {
          f32x2 f[4];
          widen8<T>(w[o], false, f);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[r][o] = fma2(v[j], f[j], acc[r][o]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kFewRows; ++r) {
      if (r >= rows) break;
#pragma unroll
      for (int o = 0; o < kOuts; ++o) {
        float s = pair_sum(acc[r][o]);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
        if (lane == o && o < outs) C[row_offset(r0 + r, p.ldc) + j0 + o] = from_f<T>(s);
      }
    }
  }
}

// ---- dW ---------------------------------------------------------------------------
//
// A sum of r unit normal products that grows row by row in fp32 is about 1.7e-8 * sqrt(r) of its size off (4.3e-6 measured
// at 61,600 rows), so it starts anew every kFold rows and is added to what the tile has so far, in memory, as the registers
// are full: 5.3e-7 for 1,970,003 rows x 16 x 16, 5.7e-7 for 200,000 x 128 x 256.  It costs nothing that shows (65,536 x 512
// x 512 in 8 groups 709 us without, 699 with).
constexpr int kFold = 1024;

__device__ __forceinline__ void add4(float4& s, const float4& v) {
  s.x += v.x;
  s.y += v.y;
  s.z += v.z;
  s.w += v.w;
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreadsL) k_linear_weights(const LinearWeights p) {
  extern __shared__ long long s_off[];
  __shared__ __align__(16) Steps s;
  __shared__ ChunkChoice s_choice;
  load_offsets(p.offsets, p.groups, p.n, s_off, p.status);
  const Plan plan = plan_in(s_off, p.groups);
  plan_chunks(p, plan, s_choice);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const T* DY = static_cast<const T*>(p.dy);
  const T* X = static_cast<const T*>(p.x.data);
  const int nb = (p.K + kPackBlock - 1) / kPackBlock;
  const bool is_wide = ((uintptr_t)p.dw & 15) == 0;  // (partial products always are)
  const int kt = (p.K + kTN - 1) / kTN, tiles = (p.M + kTM - 1) / kTM * kt;
  const long long total = (long long)plan.ocum[p.groups] * tiles;
  for (long long round = 0; round * gridDim.x < total; ++round) {
    const long long t = dealt(round, blockIdx.x, gridDim.x);
    if (t >= total) continue;
    const int c = (int)(t / tiles), q0 = (int)(t - (long long)c * tiles);
    const int m0 = q0 / kt * kTM, k0 = (q0 - q0 / kt * kt) * kTN;
    const Chunk x = chunk_of(plan, p.groups, c);
    const long long first = x.first, last = x.last;
    // this thread's four-element pieces: two of dy (rows yr and yr + 8), one of x
    const int yr = tid >> 5, yc = (tid & 31) * 4, xr = tid >> 4, xc = (tid & 15) * 4;
    float4 ry[2], rx;
    auto fetch = [&](long long r0) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const long long r = r0 + yr + q * 8;
        ry[q] = load4<T, VEC>(DY + row_offset(r, p.lddy) + m0 + yc, r < last ? p.M - m0 - yc : 0);
      }
      const long long r = r0 + xr;
      const int k = k0 + xc, left = r < last ? p.K - k : 0;
      if (X != nullptr) {
        rx = load4<T, VEC>(X + row_offset(r, p.x.ld) + k, left);
      } else {
        float f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)  // four columns never straddle a block of 32
          f[j] = j < left ? (float)p.x.codes[row_offset(r, p.K) + k + j] : 0.0f;
        const float scale = left > 0 ? pack_scale(p.x.exps[row_offset(r, nb) + k / kPackBlock]) : 0.0f;
        rx = make_float4(f[0] * scale, f[1] * scale, f[2] * scale, f[3] * scale);
        if (left < 4) {  // a block that is not finite makes its columns NaN, not the columns past K
          if (left < 1) rx.x = 0.0f;
          if (left < 2) rx.y = 0.0f;
          if (left < 3) rx.z = 0.0f;
          rx.w = 0.0f;
        }
      }
    };
    float* out = weights_out(p, plan, x);
    const int k = k0 + tx * 4;
    fetch(first);
    for (long long part = first; part < last; part += kFold) {
      const long long end = min(part + kFold, last);
      f32x2 acc[4][4] = {};
      for (long long r0 = part; r0 < end; r0 += kI) {
        *reinterpret_cast<float4*>(&s.a[yr][yc]) = ry[0];
        *reinterpret_cast<float4*>(&s.a[yr + 8][yc]) = ry[1];
        *reinterpret_cast<float4*>(&s.b[xr][xc]) = rx;
        __syncthreads();
        if (r0 + kI < last) fetch(r0 + kI);
        multiply(s, tx, ty, acc);
        __syncthreads();
      }
      const bool more = part > first;  // a thread adds to what it has written itself
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float2 f[4] = {upk(acc[u][0]), upk(acc[u][1]), upk(acc[u][2]), upk(acc[u][3])};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int m = m0 + ty * 8 + u * 2 + h;
          if (m >= p.M) continue;
          float* o = out + (size_t)m * p.K + k;
          float4 v = h ? make_float4(f[0].y, f[1].y, f[2].y, f[3].y) : make_float4(f[0].x, f[1].x, f[2].x, f[3].x);
          if (VEC && is_wide) {
            if (k >= p.K) continue;
            if (more) add4(v, *reinterpret_cast<const float4*>(o));
            *reinterpret_cast<float4*>(o) = v;
          } else {
            const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (k + j < p.K) o[j] = more ? o[j] + x[j] : x[j];
          }
        }
      }
    }
  }
}

constexpr int kSumSlices = 8;                 // warps of a block
constexpr int kSumTask = 32 * kSumSlices * 4;  // values of dW a block sums at a time
__host__ __device__ inline int sum_tasks(size_t size) { return (int)((size + kSumTask - 1) / kSumTask); }
__global__ void __launch_bounds__(32 * kSumSlices) k_linear_sums(const LinearWeights p) {
  extern __shared__ long long s_off[];
  __shared__ float4 s_sum[kSumSlices][32];
  __shared__ int s_active;
  int* s_cum = reinterpret_cast<int*>(s_off + p.groups + 1);
  int* s_slot = s_cum + p.groups + 1;
  load_offsets(p.offsets, p.groups, p.n, s_off, p.status);
  count_tiles(s_off, p.groups, *p.chosen, s_cum);
  count_slots(s_cum, p.groups, s_slot);
  const size_t size = (size_t)p.M * p.K;
  const bool four = size % 4 == 0 && ((uintptr_t)p.dw & 15) == 0;  // four values at once
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  // the groups with work: all but those whose only chunk wrote dW itself
  int* s_group = s_slot + p.groups + 1;
  if (threadIdx.x < 32) {
    int active = 0;
    for (int g0 = 0; g0 < p.groups; g0 += 32) {
      const int g = g0 + lane;
      const bool on = g < p.groups && s_cum[g + 1] - s_cum[g] != 1;
      const unsigned mask = __ballot_sync(kFull, on);
      if (on) s_group[active + __popc(mask & ((1u << lane) - 1u))] = g;
      active += __popc(mask);
    }
    if (lane == 0) s_active = active;
  }
  __syncthreads();
  // a block's task: a group's next kSumTask values
  const int per_group = sum_tasks(size);
  for (long long t = blockIdx.x; t < (long long)s_active * per_group; t += gridDim.x) {
    const int a = (int)(t / per_group), q = (int)(t - (long long)a * per_group), g = s_group[a];
    const int c = s_cum[g + 1] - s_cum[g];
    const float* part = p.part + (size_t)s_slot[g] * size;
    float* out = p.dw + (size_t)g * size;
    const size_t end = size < (size_t)(q + 1) * kSumTask ? size : (size_t)(q + 1) * kSumTask;
    if (four && c >= 2 * kSumSlices) {  // many chunks: the block's warps take every kSumSlices-th, joined in their order
      for (size_t b = (size_t)q * kSumTask / 4; b < end / 4; b += 32) {
        const size_t i = b + lane;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (i < end / 4) {
#pragma unroll 4
          for (int k = slice; k < c; k += kSumSlices) add4(s, __ldg(reinterpret_cast<const float4*>(part + (size_t)k * size) + i));
        }
        s_sum[slice][lane] = s;
        __syncthreads();
        if (slice == 0 && i < end / 4) {
          for (int k = 1; k < kSumSlices; ++k) add4(s, s_sum[k][lane]);
          reinterpret_cast<float4*>(out)[i] = s;
        }
        __syncthreads();
      }
    } else if (four) {
      const size_t i = (size_t)q * kSumTask / 4 + threadIdx.x;
      if (i < end / 4) {
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int k = 0; k < c; ++k) add4(s, __ldg(reinterpret_cast<const float4*>(part + (size_t)k * size) + i));
        reinterpret_cast<float4*>(out)[i] = s;
      }
    } else {
      for (size_t i = (size_t)q * kSumTask + threadIdx.x; i < end; i += blockDim.x) {
        float s = 0.0f;
#pragma unroll 4
        for (int k = 0; k < c; ++k) s += __ldg(part + (size_t)k * size + i);
        out[i] = s;
      }
    }
  }
}

// Partial products of dW there is room for: as many as give every block (pair) kRounds tiles, if the rows allow any split
// (a split leaves chunks of kMinChunk rows and more, so a group of one more than that makes two).
constexpr int kRounds = 4;
int slots_of(int64_t n, int32_t groups, int32_t k, int32_t m) {
  const Cut c = cut_of(n, groups, k, m, true);
  const long long want = std::max<long long>(2, (long long)kRounds * c.units / c.tiles);
  return (int)std::min<long long>(want, 2 * (n / kMinChunk));
}
size_t partial_bytes(int64_t n, int32_t groups, int32_t k, int32_t m) {
  return align_up((size_t)slots_of(n, groups, k, m) * k * m * 4 + 256, 256);
}

size_t weights_bytes(int32_t groups, int32_t k, int32_t m, int dtype) { return (size_t)groups * k * m * elem_bytes(dtype); }

// The shapes, offsets and types that both directions share.
int linear_check(const int64_t* offsets, int32_t groups, int64_t n, int32_t k, int32_t m, int dtype,
                 const int32_t* status) {
  if (dtype != MT_F32 && dtype != MT_BF16) return MT_EINVAL;
  if (n < 0 || n > MT_MAX_BLOCK_ROWS || groups < 1 || groups > MT_MAX_GROUPS) return MT_EINVAL;
  if (k < 1 || k > MT_MAX_BLOCK_DIM || m < 1 || m > MT_MAX_BLOCK_DIM) return MT_EINVAL;
  if (offsets == nullptr || !is_aligned(offsets, 8) || !is_aligned(status, 4)) return MT_EINVAL;
  return MT_OK;
}

// The forward of few rows goes to k_linear_few: of up to kFewTc rows per group on average (against the tensor cores) or
// kFewPipes (against the fp32 pipes), as long as each warp that the SMs hold has no more than kTasksTc or kTasksPipes tasks.
// Each further pair of a group's rows reads its weights again (from L2), where the tiles read them once.  Measured, warm and
// with weights from HBM, against the tiles: bf16 512 x 1024, 8 tokens on 8 experts 4.1 and 10.2 us against 7.7 and 12.3, 64
// on 32 (3.4 tasks a warp) 10.2 and 18.4 against 11.7 and 18.5, 128 on 64 (6.7) 18.4 and 26.7 against 10.8 and 24.6; 16 on 8
// of 2048 x 2048 15.7 against 33.7.  fp32: 64 on 8 of 512 x 1024 14.2 against 34.4, 8192 on 1024 of 128 x 128 (40 tasks) 103
// against 109.
constexpr int kFewTc = 2, kFewPipes = 8, kTasksTc = 3, kTasksPipes = 12;

cudaError_t launch_linear_rows(LinearRows p, int dtype, cudaStream_t s) {
  const bool tc = dtype == MT_BF16 && linear_rows_fits_tc(p);
  const long long few_tiles = (p.n + std::min<long long>(p.n, p.groups) * (kFewRows - 1)) / kFewRows;  // at most
  const long long tasks = few_tiles * ((p.J + kOuts - 1) / kOuts), held = (long long)sm_count() * kFewBlocks * 8;
  if (p.n <= (long long)(tc ? kFewTc : kFewPipes) * p.groups && tasks <= (tc ? kTasksTc : kTasksPipes) * held && p.wi == 1 &&
      p.I % 8 == 0 && (p.lda * elem_bytes(dtype)) % 16 == 0 && is_aligned(p.a, 16) && is_aligned(p.w, 16)) {
    const int grid = grid_for(tasks * 32, 256, kFewBlocks);
    MT_LAUNCH("k_linear_few", s);
    if (dtype == MT_F32) k_linear_few<float><<<grid, 256, rows_smem(p.groups), s>>>(p);
    else k_linear_few<__nv_bfloat16><<<grid, 256, rows_smem(p.groups), s>>>(p);
    return cudaGetLastError();
  }
  if (tc) return launch_linear_rows_tc(p, s);
  p.jtiles = (p.J + kTN - 1) / kTN;
  const long long tiles = (p.n / kTM + p.groups) * p.jtiles;
  const int grid = (int)std::min<long long>(tiles, (long long)sm_count() * 4);
  const size_t four = 4 * elem_bytes(dtype);
  const bool vec = p.I % 4 == 0 && p.J % 4 == 0 && p.lda % 4 == 0 && p.ldc % 4 == 0 && is_aligned(p.a, four) &&
                   is_aligned(p.w, four) && is_aligned(p.c, four);
  MT_LAUNCH("k_linear_rows", s);
  if (dtype == MT_F32) {
    if (vec) k_linear_rows<float, true><<<grid, kThreadsL, rows_smem(p.groups), s>>>(p);
    else k_linear_rows<float, false><<<grid, kThreadsL, rows_smem(p.groups), s>>>(p);
  } else {
    if (vec) k_linear_rows<__nv_bfloat16, true><<<grid, kThreadsL, rows_smem(p.groups), s>>>(p);
    else k_linear_rows<__nv_bfloat16, false><<<grid, kThreadsL, rows_smem(p.groups), s>>>(p);
  }
  return cudaGetLastError();
}

// The rest of p is filled in here: the sums go by it too.
cudaError_t launch_linear_weights(LinearWeights& p, int dtype, cudaStream_t s) {
  const Cut cut = cut_of(p.n, p.groups, p.K, p.M, p.x.data != nullptr);
  const bool tc = dtype == MT_BF16 && linear_weights_fits_tc(p);
  p.slots = slots_of(p.n, p.groups, p.K, p.M);
  // Measured: 64 rows of a tile take 0.42 us on the tensor cores and 6 us on the fp32 pipes, a tile's end 6 us, the sums'
  // launch 5 us; a partial product is written and read once, at about 4 TB/s.
  const float unit = tc ? 0.42f : 6.0f;
  p.slot_cost = (float)((double)p.K * p.M * 8 / 4e6) / unit;
  p.round_cost = 6.0f / unit;
  p.sums_cost = 5.0f / unit;
  p.tiles = tc ? cut.tiles : ((p.M + kTM - 1) / kTM) * ((p.K + kTN - 1) / kTN);
  p.units = tc ? cut.units : sm_count() * 4;
  if (p.n > 0 && tc) return launch_linear_weights_tc(p, cut, s);
  if (p.n > 0) {
    const int grid = weights_blocks(p);
    MT_LAUNCH("k_linear_weights", s);
    const size_t four = 4 * elem_bytes(dtype);
    const bool vec = p.K % 4 == 0 && p.M % 4 == 0 && p.lddy % 4 == 0 && is_aligned(p.dy, four) &&
                     (p.x.data == nullptr || (p.x.ld % 4 == 0 && is_aligned(p.x.data, four)));
    if (dtype == MT_F32) {
      if (vec) k_linear_weights<float, true><<<grid, kThreadsL, weights_smem(p.groups), s>>>(p);
      else k_linear_weights<float, false><<<grid, kThreadsL, weights_smem(p.groups), s>>>(p);
    } else {
      if (vec) k_linear_weights<__nv_bfloat16, true><<<grid, kThreadsL, weights_smem(p.groups), s>>>(p);
      else k_linear_weights<__nv_bfloat16, false><<<grid, kThreadsL, weights_smem(p.groups), s>>>(p);
    }
  }
  return cudaGetLastError();
}

cudaError_t launch_linear_sums(const LinearWeights& p, cudaStream_t s) {
  if (p.n == 0) return cudaMemsetAsync(p.dw, 0, (size_t)p.groups * p.M * p.K * 4, s);
  MT_LAUNCH("k_linear_sums", s);
  const long long tasks = (long long)p.groups * sum_tasks((size_t)p.M * p.K);
  k_linear_sums<<<grid_for(tasks * 256, 256, 8), 256, weights_smem(p.groups) + (size_t)p.groups * 4, s>>>(p);
  return cudaGetLastError();
}

// 8-bit x whose rows do not lie a multiple of 16 bytes apart cannot be copied as it is: it is widened to bf16 rows in
// the workspace first (one more pass over x, 3 bytes per value).
bool widened_first(int32_t k) { return k % 16 == 8; }

}  // namespace
}  // namespace mt

extern "C" {

int mt_group_linear_forward(const void* x, int64_t ldx, const void* w, const int64_t* offsets, int32_t groups,
                            int64_t n, int32_t in_dim, int32_t out_dim, int dtype, void* y, int64_t ldy,
                            int32_t* status, mt_stream stream) {
  using namespace mt;
  const int rc = linear_check(offsets, groups, n, in_dim, out_dim, dtype, status);
  if (rc != MT_OK) return rc;
  if (w == nullptr || !is_aligned(w, elem_bytes(dtype))) return MT_EINVAL;
  if (n == 0) return MT_OK;
  if (!rows_ok(x, ldx, in_dim, dtype) || !rows_ok(y, ldy, out_dim, dtype)) return MT_EINVAL;
  Regions all;
  all.in(Rows{const_cast<void*>(x), ldx, nullptr, nullptr}, n, in_dim, dtype);
  all.in(whole_region(w, weights_bytes(groups, in_dim, out_dim, dtype)));
  all.in(whole_region(offsets, (size_t)(groups + 1) * 8));
  all.out(Rows{y, ldy, nullptr, nullptr}, n, out_dim, dtype);
  if (all.clash()) return MT_EINVAL;
  LinearRows p{};
  p.n = n;
  p.groups = groups;
  p.offsets = reinterpret_cast<const long long*>(offsets);
  p.status = status;
  p.a = x;
  p.lda = ldx;
  p.w = w;
  p.wg = (size_t)in_dim * out_dim;
  p.wi = 1;
  p.wj = in_dim;
  p.c = y;
  p.ldc = ldy;
  p.I = in_dim;
  p.J = out_dim;
  return launch_linear_rows(p, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MT_OK : MT_ECUDA;
}

size_t mt_group_linear_workspace_bytes(int64_t n, int32_t groups, int32_t in_dim, int32_t out_dim) {
  using namespace mt;
  if (n < 0 || n > MT_MAX_BLOCK_ROWS || groups < 1 || groups > MT_MAX_GROUPS || in_dim < 1 || in_dim > MT_MAX_BLOCK_DIM || out_dim < 1 || out_dim > MT_MAX_BLOCK_DIM)
    return 0;
  return partial_bytes(n, groups, in_dim, out_dim) + (widened_first(in_dim) ? align_up((size_t)n * in_dim * 2, 256) : 0);
}

int mt_group_linear_backward(const void* dy, int64_t lddy, const mt_rows* x, const void* w, const int64_t* offsets,
                             int32_t groups, int64_t n, int32_t in_dim, int32_t out_dim, int dtype, void* dx,
                             int64_t lddx, float* dw, int32_t* status, void* ws, size_t ws_bytes, mt_stream stream) {
  using namespace mt;
  const int rc = linear_check(offsets, groups, n, in_dim, out_dim, dtype, status);
  if (rc != MT_OK) return rc;
  if (dx == nullptr && dw == nullptr) return MT_EINVAL;
  if (n > 0 && !rows_ok(dy, lddy, out_dim, dtype)) return MT_EINVAL;
  if (dx != nullptr) {
    if (w == nullptr || !is_aligned(w, elem_bytes(dtype))) return MT_EINVAL;
    if (n > 0 && !rows_ok(dx, lddx, in_dim, dtype)) return MT_EINVAL;
  }
  if (dw != nullptr) {
    if (!is_aligned(dw, 4) || x == nullptr) return MT_EINVAL;
    const bool packed = x->data == nullptr;
    if (n > 0 && (packed ? x->codes == nullptr || x->exps == nullptr : !rows_ok(x->data, x->ld, in_dim, dtype)))
      return MT_EINVAL;
    if (ws == nullptr || !is_aligned(ws, 256) || ws_bytes < mt_group_linear_workspace_bytes(n, groups, in_dim, out_dim))
      return MT_ENOSPACE;
  }
  Regions all;
  all.in(Rows{const_cast<void*>(dy), lddy, nullptr, nullptr}, n, out_dim, dtype);
  all.in(whole_region(offsets, (size_t)(groups + 1) * 8));
  if (dx != nullptr) {
    all.in(whole_region(w, weights_bytes(groups, in_dim, out_dim, dtype)));
    all.out(Rows{dx, lddx, nullptr, nullptr}, n, in_dim, dtype);
  }
  if (dw != nullptr) {
    all.in(x->data != nullptr ? Rows{x->data, x->ld, nullptr, nullptr} : *x, n, in_dim, dtype);
    all.out(whole_region(dw, weights_bytes(groups, in_dim, out_dim, MT_F32)));
    all.out(whole_region(ws, mt_group_linear_workspace_bytes(n, groups, in_dim, out_dim)));
  }
  if (all.clash()) return MT_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (dx != nullptr && n > 0) {
    LinearRows p{};
    p.n = n;
    p.groups = groups;
    p.offsets = reinterpret_cast<const long long*>(offsets);
    p.status = status;
    p.a = dy;
    p.lda = lddy;
    p.w = w;
    p.wg = (size_t)in_dim * out_dim;
    p.wi = in_dim;
    p.wj = 1;
    p.c = dx;
    p.ldc = lddx;
    p.I = out_dim;
    p.J = in_dim;
    e = launch_linear_rows(p, dtype, s);
  }
  if (dw != nullptr && e == cudaSuccess) {
    LinearWeights p{};
    p.n = n;
    p.groups = groups;
    p.offsets = reinterpret_cast<const long long*>(offsets);
    p.status = status;
    p.dy = dy;
    p.lddy = lddy;
    p.x = *x;
    p.K = in_dim;
    p.M = out_dim;
    p.chosen = static_cast<int*>(ws);
    p.part = static_cast<float*>(ws) + 64;
    p.dw = dw;
    if (dtype == MT_BF16 && x->data == nullptr && widened_first(in_dim) && n > 0) {
      LinearWeights q = p;
      q.x = Rows{static_cast<char*>(ws) + partial_bytes(n, groups, in_dim, out_dim), in_dim, nullptr, nullptr};
      if (linear_weights_fits_tc(q)) {
        const int rc8 = mt_unpack8(x->codes, x->exps, n, in_dim, dtype, q.x.data, in_dim, stream);
        if (rc8 != MT_OK) return rc8;
        p = q;
      }
    }
    e = launch_linear_weights(p, dtype, s);
    if (e == cudaSuccess) e = launch_linear_sums(p, s);
  }
  return e == cudaSuccess ? MT_OK : MT_ECUDA;
}

}  // extern "C"
