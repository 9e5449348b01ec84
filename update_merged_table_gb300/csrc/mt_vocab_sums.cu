// The gradients of the losses over a vocabulary from a piece of dz, the gradient
// of its logits:
//
//   dx = dz W    rows of x by columns of W, the contraction over the piece, cut into
//                runs where there are few rows; fp32 partial products, one per run,
//                which the next pieces add to
//   dW = dz^T x  entries of the piece by columns of x, the contraction over the live
//                rows; the only product where the piece has entries enough, else cut
//
// fp32 rows: the accumulator starts anew every 512 products (`promote`) and is
// added up in registers, rounding to nearest, since the tensor core cuts it off
// towards zero at every step.
#include "mt_tiles.cuh"
#include "mt_vocab.cuh"

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
  static constexpr bool kAMN = VOCAB, kBMN = true, kTeams = !FP32, kKeep = false;
  const Params& p;
  int rank, rows, rt, steps, quad, half, lane;
  uint8_t* stage;
  float sum[FP32 ? BN / 2 : 1];

  __device__ Sum(const Params& params, uint8_t*, int r) : p(params), rank(r) {
    const int live = *p.live;
    rows = VOCAB ? p.rows : live;
    steps = VOCAB ? (live + tiles::kBK - 1) / tiles::kBK : p.steps;
    rt = (rows + tiles::kBM * CG - 1) / (tiles::kBM * CG);
  }
  __device__ long long units() const { return (long long)rt * p.ctiles * p.splits; }
  __device__ Unit unit(long long u) const {  // columns fastest: the tiles of a row tile read the same rows of dz
    const int c = (int)(u % p.ctiles);
    const long long q = u / p.ctiles;
    const int r = (int)(q % rt), s = (int)(q / rt);
    Unit x;
    x.g = 0;
    x.row0 = r * (tiles::kBM * CG);
    x.end = rows;
    x.ct0 = c;
    x.ct1 = c + 1;
    x.k0 = (int)((long long)s * steps / p.splits);
    x.k1 = (int)((long long)(s + 1) * steps / p.splits);
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
  __device__ void end(const Unit&) {}

  // 16 columns of each lane's row, added to what is there where p.add
  __device__ __forceinline__ void put(const float (&f)[32], const Unit& x, int col, bool first_half) {
    const long long r0 = x.row0 + rank * tiles::kBM + quad * 32;
    const int n = min(32, x.end - (int)r0);
    float* C = p.part + (size_t)x.slot * p.stride * p.columns;
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(first_half ? f[j] : f[16 + j]);
    if (!p.add) {
      tiles::store_rows<float>(stage, lane, w, C, p.columns, r0, n, col, p.columns, p.columns % 4 == 0);
      return;
    }
    if (col >= p.columns) return;
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<uint4*>(stage + tiles::piece_at(lane, c)) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    __syncwarp();
    if (p.columns % 4 == 0) {
      const int c = lane & 3, at = col + c * 4;
      float4 old[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = q * 8 + (lane >> 2);
        if (r < n && at < p.columns) old[q] = *reinterpret_cast<const float4*>(C + (size_t)(r0 + r) * p.columns + at);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = q * 8 + (lane >> 2);
        if (r < n && at < p.columns) {
          const float4 v = *reinterpret_cast<const float4*>(stage + tiles::piece_at(r, c));
          *reinterpret_cast<float4*>(C + (size_t)(r0 + r) * p.columns + at) =
              make_float4(old[q].x + v.x, old[q].y + v.y, old[q].z + v.z, old[q].w + v.w);
        }
      }
    } else {
      for (int i = lane; i < 512; i += 32) {
        const int r = i / 16, j = i % 16;
        if (r < n && col + j < p.columns)
          C[(size_t)(r0 + r) * p.columns + col + j] += *reinterpret_cast<const float*>(stage + tiles::piece_at(r, j / 4) + j % 4 * 4);
      }
    }
  }

  __device__ __forceinline__ void store(const float (&f)[32], const Unit& x, int col) {
    if (!VOCAB || p.part != nullptr) {
      put(f, x, col, true);
      put(f, x, col + 16, false);
      return;
    }
    using T = std::conditional_t<FP32, float, __nv_bfloat16>;
    const long long r0 = x.row0 + rank * tiles::kBM + quad * 32;
    tiles::store32<T>(stage, lane, f, static_cast<T*>(p.out), p.columns, r0, min(32, x.end - (int)r0), col, p.columns, p.wide);
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
  const long long units = row_tiles * p.ctiles * p.splits;
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
