// Tiles of logits x W^T, 128 rows (256 by a pair of blocks) by 256 entries of the
// vocabulary, that never leave the chip:
//
//  the statistics   a thread has one row and half of a tile's columns.  It keeps
//                   the largest logit so far and the sum of 2^(z - largest) over a
//                   run of tiles (an online softmax in base 2, one exponential a
//                   logit), and picks the logits of the row's targets as they come
//                   by: the targets lie in ascending order, so one comparison per
//                   32 columns finds them.
//  their gradient   with the row's log sum known, dz = a p - b less the targets'
//                   shares, rounded to bf16 (fp32 rows: three bf16 parts), a piece
//                   of the vocabulary at a time.
#include "mt_tiles.cuh"
#include "mt_vocab.cuh"

namespace mt {
namespace {

using tiles::Acc;
using tiles::Unit;

__device__ __forceinline__ float exp2_of(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Runs of column tiles for `rt` row tiles on `blocks` blocks (pairs): as many as end the last block soonest, a run's start
// counted as half a tile.  Every thread calls it.
__device__ __forceinline__ int choose_chunks(int rt, int tiles, int most, int blocks) {
  __shared__ unsigned long long s_best;
  if (threadIdx.x == 0) s_best = ~0ull;
  __syncthreads();
  unsigned long long best = ~0ull;
  for (int c = threadIdx.x + 1; c <= min(most, tiles); c += blockDim.x) {
    const long long rounds = ((long long)rt * c + blocks - 1) / blocks;
    const unsigned long long cost = (unsigned long long)rounds * (2 * ((tiles + c - 1) / c) + 1);
    best = min(best, cost << 32 | (unsigned)c);
  }
  if (best != ~0ull) atomicMin(&s_best, best);
  __syncthreads();
  return (int)(uint32_t)s_best;
}

// What both kernels share: rows tiles fastest, so that blocks at work at the same time read the same entries of W.
template <int CG>
struct Logits {
  using Params = LogitParams;
  static constexpr int kBN = 256;
  static constexpr bool kAMN = false, kBMN = false, kTwoB = false;
  const Params& p;
  int rank, live, rt, chunks;
  uint8_t* stage;
  int half, lane, row, pos, next;  // the thread's row; its next target

  __device__ Logits(const Params& params, uint8_t*, int r) : p(params), rank(r) {
    live = *p.rows.count;
    rt = (live + tiles::kBM * CG - 1) / (tiles::kBM * CG);
    chunks = choose_chunks(rt, p.tiles, p.max_chunks, gridDim.x / CG);
  }
  __device__ long long units() const { return (long long)rt * chunks; }
  __device__ Unit unit(long long u) const {
    const int c = (int)(u / rt), r = (int)(u - (long long)c * rt);
    Unit x;
    x.g = 0;
    x.row0 = r * (tiles::kBM * CG);
    x.end = live;
    x.ct0 = (int)((long long)c * p.tiles / chunks);
    x.ct1 = (int)((long long)(c + 1) * p.tiles / chunks);
    x.k0 = 0;
    x.k1 = p.steps;
    x.slot = c;
    return x;
  }
  int quad;
  __device__ void warp(uint8_t* s, int q, int h, int l) {
    stage = s;
    quad = q;
    half = h;
    lane = l;
  }
  __device__ void start(const Unit& x) {
    row = x.row0 + rank * tiles::kBM + quad * 32 + lane;
    pos = 0;
    next = 0x7FFFFFFF;
    if (row >= live) return;
    const int first = p.v0 + x.ct0 * kBN;
    const int* ids = p.rows.ids + (size_t)row * p.rows.top;
    int lo = 0, hi = p.rows.top;  // targets before `lo` are below `first`, those from `hi` on are not
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (ids[mid] < first) lo = mid + 1;
      else hi = mid;
    }
    pos = lo;
    if (pos < p.rows.top) next = ids[pos];
  }
  __device__ __forceinline__ void advance() {
    ++pos;
    next = pos < p.rows.top ? p.rows.ids[(size_t)row * p.rows.top + pos] : 0x7FFFFFFF;
  }
};

template <bool SMOOTH, int CG>
struct Stats : Logits<CG> {
  using Base = Logits<CG>;
  float top, sum, total;
  __device__ Stats(const LogitParams& p, uint8_t* mem, int r) : Base(p, mem, r) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.chunks = this->chunks;
  }
  __device__ void begin(const Unit& x) {
    this->start(x);
    top = -INFINITY;
    sum = total = 0.0f;
  }
  __device__ void end(const Unit& x) {
    if (this->row >= this->live) return;
    const size_t at = (size_t)(x.slot * 2 + this->half) * this->p.stride + this->row;
    this->p.part[at] = make_float2(top, sum);
    if constexpr (SMOOTH) this->p.sum_z[at] = total;
  }
  template <int G>
  __device__ __forceinline__ void tile(const Unit&, int ct, const Acc& acc, bool, bool) {
    const LogitParams& p = this->p;
    const int left = p.columns - ct * 256 - this->half * 128;  // columns of this half that there are
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
      uint32_t v[32];
      acc.load(this->half * 128 + c, v);
      tc::tmem_load_wait(v);
      if (c == 96) acc.release<G>(this->lane);
      const int col = p.v0 + ct * 256 + this->half * 128 + c;
      while (__any_sync(kFull, this->next < col + 32)) {
        if (this->next < col + 32) {
          if (this->next >= col) {
            const int at = this->next - col;
            uint32_t z = v[0];
#pragma unroll
            for (int j = 1; j < 32; ++j) z = at == j ? v[j] : z;
            p.picked[(size_t)this->row * p.rows.top + this->pos] = __uint_as_float(z);
          }
          this->advance();
        }
      }
      if (left < c + 32) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (c + j >= left) v[j] = 0xFF800000u;
      }
      float m = __uint_as_float(v[0]);
#pragma unroll
      for (int j = 1; j < 32; ++j) m = fmaxf(m, __uint_as_float(v[j]));
      const float now = fmaxf(top, m * p.scale2);
      const float off = now == -INFINITY ? 0.0f : now;
      const f32x2 s2 = both(p.scale2), o2 = both(-off);
      float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        const float2 e = upk(fma2(pk(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), s2, o2));
        s[j & 2] += exp2_of(e.x);
        s[(j & 2) + 1] += exp2_of(e.y);
      }
      sum = fmaf(sum, exp2_of(top - off), (s[0] + s[1]) + (s[2] + s[3]));
      top = now;
      if constexpr (SMOOTH) {
        float t = 0.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (c + j < left) t += __uint_as_float(v[j]);
        total += t;
      }
    }
  }
};

template <int PARTS, int CG>
struct Grad : Logits<CG> {
  using Base = Logits<CG>;
  float4 k;
  __device__ Grad(const LogitParams& p, uint8_t* mem, int r) : Base(p, mem, r) {}
  __device__ void begin(const Unit& x) {
    this->start(x);
    k = this->row < this->live ? this->p.coef[this->row] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  __device__ void end(const Unit&) {}
  template <int G>
  __device__ __forceinline__ void tile(const Unit& x, int ct, const Acc& acc, bool, bool) {
    const LogitParams& p = this->p;
    const int left = p.columns - ct * 256 - this->half * 128;
    const bool dead = this->row >= this->live;  // a row behind the last: whatever it holds, zeros
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
      uint32_t v[32];
      acc.load(this->half * 128 + c, v);
      tc::tmem_load_wait(v);
      if (c == 96) acc.release<G>(this->lane);
      const int at0 = ct * 256 + this->half * 128 + c, col = p.v0 + at0;
      float f[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) f[j] = fmaf(exp2_of(fmaf(__uint_as_float(v[j]), p.scale2, -k.x)), k.y, -k.z);
      while (__any_sync(kFull, this->next < col + 32)) {
        if (this->next < col + 32) {
          if (this->next >= col) {
            const int at = this->next - col;
            const float take = k.w * p.rows.share[(size_t)this->row * p.rows.top + this->pos];
#pragma unroll
            for (int j = 0; j < 32; ++j) f[j] -= at == j ? take : 0.0f;
          }
          this->advance();
        }
      }
      if (dead || left < c + 32) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (dead || c + j >= left) f[j] = 0.0f;
      }
      const long long r0 = x.row0 + this->rank * tiles::kBM + this->quad * 32;
      if constexpr (PARTS == 1) {
        tiles::store32<__nv_bfloat16>(this->stage, this->lane, f, p.dz, p.width, r0, 32, at0, p.width, true);
      } else {
        uint32_t w[3][16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          __nv_bfloat16 a[3], b[3];
          split3(f[2 * j], a[0], a[1], a[2]);
          split3(f[2 * j + 1], b[0], b[1], b[2]);
#pragma unroll
          for (int q = 0; q < 3; ++q) w[q][j] = bf16_bits(a[q], b[q]);
        }
#pragma unroll
        for (int q = 0; q < 3; ++q)
          tiles::store_rows<__nv_bfloat16>(this->stage, this->lane, w[q], p.dz + (size_t)q * p.width, (size_t)3 * p.width, r0, 32, at0, p.width, true);
      }
    }
  }
};

}  // namespace

cudaError_t launch_logit_stats(const LogitParams& p, const CUtensorMap& a, const CUtensorMap& b, long long row_tiles, bool pair,
                               cudaStream_t s) {
  const long long units = row_tiles * (p.tiles < p.max_chunks ? p.tiles : p.max_chunks);
  const char* name = "k_logit_stats";
  if (p.sum_z != nullptr)
    return pair ? tiles::launch<Stats<true, 2>, 2>(name, a, b, p, units, 0, 0, s) : tiles::launch<Stats<true, 1>, 1>(name, a, b, p, units, 0, 0, s);
  return pair ? tiles::launch<Stats<false, 2>, 2>(name, a, b, p, units, 0, 0, s) : tiles::launch<Stats<false, 1>, 1>(name, a, b, p, units, 0, 0, s);
}

cudaError_t launch_logit_grad(const LogitParams& p, int parts, const CUtensorMap& a, const CUtensorMap& b, long long row_tiles, bool pair,
                              cudaStream_t s) {
  const long long units = row_tiles * (p.tiles < p.max_chunks ? p.tiles : p.max_chunks);
  const char* name = "k_logit_grad";
  if (parts == 3) return tiles::launch<Grad<3, 1>, 1>(name, a, b, p, units, 0, 0, s);
  return pair ? tiles::launch<Grad<1, 2>, 2>(name, a, b, p, units, 0, 0, s) : tiles::launch<Grad<1, 1>, 1>(name, a, b, p, units, 0, 0, s);
}

}  // namespace mt
