// Tiles of logits x W^T, 128 rows (256 by a pair of blocks) by 256 entries of the
// vocabulary, that never leave the chip.  Where the rows are short (KEEP) a block
// keeps its rows of x for a whole run of the vocabulary, which halves what it reads
// from L2.
//
//  the statistics   a thread has one row of half of each tile.  It keeps the largest
//                   logit so far and the sum of 2^(z - largest) over a run of tiles (an online softmax in base 2, one exponential a
//                   logit), and picks the logits of the row's targets as they come
//                   by: the targets lie in ascending order, so one comparison per
//                   32 columns finds them.
//  their gradient   with the row's log sum known, dz = a p - b less the targets'
//                   shares, rounded to bf16 (few rows: two bf16 parts, fp32 rows:
//                   three), a piece of the vocabulary at a time.
//
// Bound: by the tensor cores from 512 columns on (7373 live rows x 100,003 x 512: statistics 400 to 450 us, 1.7 to 1.9
// PFLOP/s; gradient 545, with 1.5 GB written), below by exponentials and their latency (32,769 live rows x 16,384 x 256:
// 170 us, 1.6 PFLOP/s, and 244 us).
#include <algorithm>

#include "mt_tiles.cuh"
#include "mt_vocab.cuh"
#include "mt_vocab_rows.cuh"

namespace mt {
namespace {

using tiles::Acc;
using tiles::Unit;

// Columns of a tile that a team of epilogue warps has.  Both teams at one tile leave its accumulator twice as soon as teams in
// turns, and all columns of a row in registers have one largest value and one chain of sums.  Measured with teams in turns and
// 32 columns at a time, with halves, and with halves at once: 32,769 of 65,537 rows x 16,384 x 256 statistics 214, 190 and 170 us,
// gradient 284, 252 and 244; 4096 x 131,072 x 1024, bound by the products, 609, 609 and 630, and 719, 633 and 654.
constexpr int kHalf = 128;

// What both kernels share: rows tiles fastest, so that blocks at work at the same time read the same entries of W.
template <int CG, bool KEEP>
struct Logits {
  using Params = LogitParams;
  static constexpr int kBN = 256;
  static constexpr bool kAMN = false, kBMN = false, kTwoB = false, kTeams = false, kKeep = KEEP, kAhead = false, kSplit = true, kSingle = false, kTri = false;
  static constexpr int kStageOut = 4096;  // 32 rows x 128 bytes
  const Params& p;
  int rank, live, rt, chunks;
  uint8_t* stage;
  int quad, team, lane, row;  // the thread's row
  RowTargets to;

  __device__ Logits(const Params& params, uint8_t*, int r) : p(params), rank(r) {
    live = *p.rows.count;
    rt = (live + tiles::kBM * CG - 1) / (tiles::kBM * CG);
    chunks = choose_chunks(rt, p.tiles, p.max_chunks, gridDim.x / CG, KEEP ? 6 : 1);
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
  __device__ void warp(uint8_t* s, int q, int h, int l) {
    stage = s;
    quad = q;
    team = h;
    lane = l;
  }
  // A warp's columns of a tile, all at once: the accumulator is free for the next products before the arithmetic begins.
  template <int G>
  __device__ __forceinline__ void load(const Acc& acc, uint32_t (&v)[kHalf / 32][32]) const {
#pragma unroll
    for (int i = 0; i < kHalf / 32; ++i) acc.load(team * kHalf + i * 32, v[i]);
    tc::tmem_load_wait(v[0]);
#pragma unroll
    for (int i = 1; i < kHalf / 32; ++i) tc::tmem_loaded(v[i]);
    acc.release<G>(lane);
  }
  __device__ void start(const Unit& x) {
    row = x.row0 + rank * tiles::kBM + quad * 32 + lane;
    to.start(p.rows, row, live, p.v0 + x.ct0 * kBN);
  }
};

template <bool SMOOTH, int CG, bool KEEP>
struct Stats : Logits<CG, KEEP> {
  using Base = Logits<CG, KEEP>;
  RowStats<SMOOTH> stats;
  __device__ Stats(const LogitParams& p, uint8_t* mem, int r) : Base(p, mem, r) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.chunks = this->chunks;
  }
  __device__ void begin(const Unit& x) {
    this->start(x);
    stats.clear();
  }
  __device__ void end(const Unit& x) {
    if (this->row >= this->live) return;
    const size_t at = (size_t)(x.slot * 2 + this->team) * this->p.stride + this->row;
    this->p.part[at] = make_float2(stats.top, stats.sum);
    if constexpr (SMOOTH) this->p.sum_z[at] = stats.total;
  }
  __device__ void finish() {}
  template <int G>
  __device__ __forceinline__ void tile(const Unit&, int ct, const Acc& acc, bool, bool) {
    const LogitParams& p = this->p;
    const int at = ct * Base::kBN + this->team * kHalf, left = p.columns - at;
    // there may be targets among the columns, or columns that are not there
    const bool some = left < kHalf || __any_sync(kFull, this->to.next < p.v0 + at + kHalf);
    uint32_t v[kHalf / 32][32];
    this->template load<G>(acc, v);
    if (some) {
#pragma unroll
      for (int i = 0; i < kHalf / 32; ++i) this->to.pick(p.rows, p.v0 + at + i * 32, v[i], p.picked);
    }
    stats.add(v, p.scale2, some ? left : kHalf);
  }
};

template <int PARTS, int CG, bool KEEP>  // of dz, bf16 each
struct Grad : Logits<CG, KEEP> {
  using Base = Logits<CG, KEEP>;
  float4 k;
  __device__ Grad(const LogitParams& p, uint8_t* mem, int r) : Base(p, mem, r) {}
  __device__ void begin(const Unit& x) {
    this->start(x);
    k = this->row < this->live ? this->p.coef[this->row] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  __device__ void end(const Unit&) {}
  __device__ void finish() {
    if (PARTS == 1 && this->lane == 0) tc::bulk_done();
  }
  // dz of 32 columns
  __device__ __forceinline__ void columns(const uint32_t (&v)[32], int at0, int left, bool some, float (&f)[32]) {
    const LogitParams& p = this->p;
    const int col = p.v0 + at0;
    const f32x2 s2 = both(p.scale2), x2 = both(-k.x), y2 = both(k.y), z2 = both(-k.z);
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const float2 e = upk(fma2(pk(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), s2, x2));
      const float2 d = upk(fma2(pk(exp2_of(e.x), exp2_of(e.y)), y2, z2));
      f[j] = d.x;
      f[j + 1] = d.y;
    }
    if (some) {
      this->to.take(p.rows, col, k.w, f);
      // zeros behind the piece's last column, and in a row behind the last, whatever it holds
      const uint32_t there = this->row < this->live ? below(left) : 0u;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (!(there >> j & 1)) f[j] = 0.0f;
    }
  }
  // bf16: 32 columns into their half of the warp's 32 rows x 128 bytes (piece c of row r at c ^ (r & 7), as copies with the
  // 128-byte swizzle have it), which leave by one copy: the warps neither turn rows nor wait for their stores.
  __device__ __forceinline__ void to_stage(const float (&f)[32], int half) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<uint4*>(this->stage + this->lane * 128 + (((half * 4 + q) ^ (this->lane & 7)) << 4)) =
          make_uint4(bf16x2_of(f[q * 8], f[q * 8 + 1]), bf16x2_of(f[q * 8 + 2], f[q * 8 + 3]), bf16x2_of(f[q * 8 + 4], f[q * 8 + 5]),
                     bf16x2_of(f[q * 8 + 6], f[q * 8 + 7]));
  }
  __device__ __forceinline__ void put_parts(const float (&f)[32], int at0, long long r0) {
    const LogitParams& p = this->p;
    uint32_t w[3][16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      uint32_t t[3];
      split3_pair(f[2 * j], f[2 * j + 1], t);
#pragma unroll
      for (int q = 0; q < 3; ++q) w[q][j] = t[q];
    }
#pragma unroll
    for (int q = 0; q < PARTS; ++q)
      tiles::store_rows<__nv_bfloat16>(this->stage, this->lane, w[q], p.dz + (size_t)q * p.width, (size_t)PARTS * p.width, r0, 32, at0, p.width, tiles::kSectors);
  }
  template <int G>
  __device__ __forceinline__ void tile(const Unit& x, int ct, const Acc& acc, bool, bool) {
    const int at = ct * Base::kBN + this->team * kHalf, left = this->p.columns - at;
    const int r0 = x.row0 + this->rank * tiles::kBM + this->quad * 32;
    const bool some = left < kHalf || __any_sync(kFull, this->to.next < this->p.v0 + at + kHalf || this->row >= this->live);
    uint32_t v[kHalf / 32][32];
    this->template load<G>(acc, v);
#pragma unroll
    for (int i = 0; i < kHalf / 32; ++i) {
      float f[32];
      const int c = i * 32;
      columns(v[i], at + c, left - c, some, f);
      if constexpr (PARTS > 1) {
        put_parts(f, at + c, r0);
      } else {
        if (i % 2 == 0) {
          if (this->lane == 0) tc::bulk_read();  // the last 64 columns' copy has read them
          __syncwarp();
        }
        to_stage(f, i % 2);
        if (i % 2 == 1) {
          tc::fence_async_proxy();
          __syncwarp();
          if (this->lane == 0 && at + c - 32 < this->p.width) tc::tma_store_2d(&this->p.map_dz, this->stage, at + c - 32, r0);
        }
      }
    }
  }
};

}  // namespace

namespace {
template <class Op, int CG>
cudaError_t launch_op(const char* name, const LogitParams& p, const CUtensorMap& a, const CUtensorMap& b, long long row_tiles, cudaStream_t s) {
  return tiles::launch<Op, CG>(name, a, b, p, row_tiles * std::min(p.tiles, p.max_chunks), 0, 0, s);
}
}  // namespace

cudaError_t launch_logit_stats(const LogitParams& p, const CUtensorMap& a, const CUtensorMap& b, long long row_tiles, bool pair,
                               cudaStream_t s) {
  const char* name = "k_logit_stats";
  auto go = [&](auto smooth) {
    constexpr bool S = decltype(smooth)::value;
    if (p.kept > 0)
      return pair ? launch_op<Stats<S, 2, true>, 2>(name, p, a, b, row_tiles, s) : launch_op<Stats<S, 1, true>, 1>(name, p, a, b, row_tiles, s);
    return pair ? launch_op<Stats<S, 2, false>, 2>(name, p, a, b, row_tiles, s) : launch_op<Stats<S, 1, false>, 1>(name, p, a, b, row_tiles, s);
  };
  return p.sum_z != nullptr ? go(std::true_type{}) : go(std::false_type{});
}
cudaError_t launch_logit_grad(const LogitParams& p, int parts, const CUtensorMap& a, const CUtensorMap& b, long long row_tiles, bool pair,
                              cudaStream_t s) {
  const char* name = "k_logit_grad";
  auto single = [&](auto n) {
    constexpr int N = decltype(n)::value;
    return p.kept > 0 ? launch_op<Grad<N, 1, true>, 1>(name, p, a, b, row_tiles, s) : launch_op<Grad<N, 1, false>, 1>(name, p, a, b, row_tiles, s);
  };
  if (parts == 3) return single(std::integral_constant<int, 3>{});
  if (parts == 2) return single(std::integral_constant<int, 2>{});
  if (!pair) return single(std::integral_constant<int, 1>{});
  return p.kept > 0 ? launch_op<Grad<1, 2, true>, 2>(name, p, a, b, row_tiles, s) : launch_op<Grad<1, 2, false>, 2>(name, p, a, b, row_tiles, s);
}

}  // namespace mt
