// The gradients of the losses over a vocabulary from a piece of dz, the gradient
// of its logits:
//
//   dx = dz W    rows of x by columns of W, the contraction over the piece; fp32
//                sums, which the next pieces add to
//   dW = dz^T x  entries of the piece by columns of x, the contraction over the live
//                rows, rounded and done
//
// fp32 rows: a step brings all parts of both operands and makes their six products
// (part by part, each pass over the operands again was bound by L2: dW of 10,007 x
// 128 from 1639 rows 45 us, with all at once 33).  The accumulator starts anew
// every step (`promote`) and is added up in registers, rounding to nearest, since the
// tensor core cuts it off towards zero at every product.
#include "mt_tiles.cuh"
#include "mt_vocab.cuh"
#include "mt_vocab_rows.cuh"

namespace mt {
namespace {

using tiles::Acc;
using tiles::Unit;

// BN: columns of a tile.  FP32: operands in three parts, sums kept in registers between parts of the contraction.  VOCAB:
// rows are entries of the piece and the contraction is over the live rows (dW), else the other way round (dx).
template <int BN, bool FP32, bool VOCAB, int CG>
struct Sum {
  using Params = SumParams;
  static constexpr int kBN = BN;
  static constexpr bool kAMN = VOCAB, kBMN = true, kTeams = !FP32, kKeep = false, kAhead = false, kSplit = false, kSingle = false, kTri = FP32;
  static constexpr int kStageOut = 2048;  // 32 rows x 64 bytes
  const Params& p;
  int rank, rows, rt, steps, whole, runs, quad, half, lane;  // whole: row tiles with the whole contraction
  uint8_t* stage;
  float sum[FP32 ? BN / 2 : 1];

  __device__ Sum(const Params& params, uint8_t*, int r) : p(params), rank(r) {
    const int live = *p.live;
    rows = VOCAB ? p.rows : live;
    steps = VOCAB ? (live + tiles::kBK - 1) / tiles::kBK : p.steps;
    rt = (rows + tiles::kBM * CG - 1) / (tiles::kBM * CG);
    const int blocks = gridDim.x / CG;
    const int least = max(1, ((VOCAB ? steps : p.usual) + kLongest / tiles::kBK - 1) / (kLongest / tiles::kBK));
    whole = least > 1 ? 0 : rt * p.ctiles / blocks * blocks / p.ctiles;
    // (a partial product is written and read again, which takes about as long as 24 steps, or 4 of six products each)
    runs = choose_chunks((rt - whole) * p.ctiles, VOCAB ? steps : p.usual, p.max_runs, blocks, FP32 ? 8 : 48, least);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      p.cut[0] = whole * (tiles::kBM * CG);
      p.cut[1] = runs;
    }
  }
  __device__ long long units() const { return ((long long)whole + (long long)(rt - whole) * runs) * p.ctiles; }
  __device__ Unit unit(long long u) const {  // columns fastest: the tiles of a row tile read the same rows of dz
    const unsigned q = (unsigned)u / (unsigned)p.ctiles;  // (fewer than 2^32: at most eight a block beside the whole tiles)
    const int c = (int)((unsigned)u - q * (unsigned)p.ctiles);
    int r = (int)q, s = 0, n = 1;
    if (r >= whole) {
      const int rest = rt - whole;
      s = (r - whole) / rest;
      r = whole + (r - whole) - s * rest;
      n = runs;
    }
    Unit x;
    x.g = 0;
    x.row0 = r * (tiles::kBM * CG);
    x.end = rows;
    x.ct0 = c;
    x.ct1 = c + 1;
    x.k0 = (int)((long long)s * steps / n);
    x.k1 = (int)((long long)(s + 1) * steps / n);
    x.slot = s;
    return x;
  }
  __device__ void warp(uint8_t* s, int q, int h, int l) {
    stage = s;
    quad = q;
    half = h;
    lane = l;
  }
  __device__ void begin(const Unit&) {}
  __device__ void finish() {}
  __device__ void end(const Unit&) {}

  // 32 columns of each lane's row to the unit's partial product, or added to it
  __device__ __forceinline__ void put(float (&f)[32], const Unit& x, int col) {
    const long long r0 = x.row0 - (VOCAB ? whole * (tiles::kBM * CG) : 0) + rank * tiles::kBM + quad * 32;
    const int n = min(32, x.end - (x.row0 + rank * tiles::kBM + quad * 32));
    float* C = p.part + (size_t)x.slot * p.stride * p.columns;
    if (!VOCAB && p.add) {
      float old[32];
      tiles::load_rows<float>(stage, lane, old, C, p.columns, r0, n, col, p.columns, p.reach_part);
#pragma unroll
      for (int j = 0; j < 32; ++j) f[j] += old[j];
    }
    tiles::store32<float>(stage, lane, f, C, p.columns, r0, n, col, p.columns, p.reach_part);
  }

  __device__ __forceinline__ void store(float (&f)[32], const Unit& x, int col) {
    if (!VOCAB || x.row0 >= whole * (tiles::kBM * CG)) {
      put(f, x, col);
      return;
    }
    using T = std::conditional_t<FP32, float, __nv_bfloat16>;
    const int r0 = x.row0 + rank * tiles::kBM + quad * 32;
    tiles::store32<T>(stage, lane, f, static_cast<T*>(p.out), p.columns, r0, min(32, x.end - r0), col, p.columns, p.reach);
  }

  template <int G>
  __device__ __forceinline__ void tile(const Unit& x, int ct, const Acc& acc, bool first, bool last) {
    constexpr int kMine = kTeams ? BN : BN / 2;  // columns of this warp
    const int from = kTeams ? 0 : half * kMine, col0 = ct * BN + from;
#pragma unroll
    for (int c = 0; c < kMine; c += 32) {
      uint32_t v[32];
      acc.load_or_zero(from + c, v);
      tc::tmem_load_wait(v);
      if (c + 32 == kMine) acc.release<G>(lane);
      if constexpr (FP32) {
#pragma unroll
        for (int j = 0; j < 32; ++j) sum[c + j] = first ? __uint_as_float(v[j]) : sum[c + j] + __uint_as_float(v[j]);
      } else {
        float f[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(v[j]);
        store(f, x, col0 + c);
      }
    }
    if constexpr (FP32) {
      if (last) {
#pragma unroll
        for (int c = 0; c < kMine; c += 32) {
          float f[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) f[j] = sum[c + j];
          store(f, x, col0 + c);
        }
      }
    }
  }
};

template <bool VOCAB>
cudaError_t launch_sum(const char* name, const SumParams& p, bool fp32, const CUtensorMap& a, const CUtensorMap& b, long long row_tiles,
                       bool pair, cudaStream_t s) {
  const long long units = row_tiles * p.ctiles * p.max_runs;
  const int bn = sum_width(p.columns, fp32);
  if (fp32)
    return bn == 64 ? tiles::launch<Sum<64, true, VOCAB, 1>, 1>(name, a, b, p, units, 0, 0, s)
                    : tiles::launch<Sum<128, true, VOCAB, 1>, 1>(name, a, b, p, units, 0, 0, s);
  if (bn == 64) return tiles::launch<Sum<64, false, VOCAB, 1>, 1>(name, a, b, p, units, 0, 0, s);
  if (bn == 128) return tiles::launch<Sum<128, false, VOCAB, 1>, 1>(name, a, b, p, units, 0, 0, s);
  return pair ? tiles::launch<Sum<256, false, VOCAB, 2>, 2>(name, a, b, p, units, 0, 0, s)
              : tiles::launch<Sum<256, false, VOCAB, 1>, 1>(name, a, b, p, units, 0, 0, s);
}

}  // namespace

cudaError_t launch_rows_sum(const SumParams& p, bool fp32, const CUtensorMap& a, const CUtensorMap& b, long long row_tiles, bool pair,
                            cudaStream_t s) {
  return launch_sum<false>("k_vocab_dx", p, fp32, a, b, row_tiles, pair, s);
}
cudaError_t launch_vocab_sum(const SumParams& p, bool fp32, const CUtensorMap& a, const CUtensorMap& b, long long row_tiles, bool pair,
                             cudaStream_t s) {
  return launch_sum<true>("k_vocab_dw", p, fp32, a, b, row_tiles, pair, s);
}

}  // namespace mt
