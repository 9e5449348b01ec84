// The gated feed-forward part of a block over ragged groups of rows:
//
//   forward   y = Wy x, u = Wu x, h = y act(u)          W [groups, Wy over Wu: 2 out, in]
//   backward  dy = dh act(u), du = dh y act'(u), dx = Wy^T dy + Wu^T du, dW = [dy | du]^T x
//
// Forward: one product of both projections.  A tile holds 128 columns of y and
// the same 128 of u side by side (a pair of blocks: one block copies Wy's rows,
// the other Wu's), so the epilogue has both in registers and only h is written.
// Backward: the same product again, y and u meet dh in the epilogue and leave as
// dt = [dy | du] in the rows' type; then the grouped products of mt_linear*.cu make
// dx and dW from it.  Nothing but x is kept between the two: y and u would be 4 n out
// bytes written and read against 4 n in out operations.
//
// Bound: by the tensor cores where rows are long (40,009 rows on 32 uneven experts, 1024 -> 2048, backward's product 250 us:
// 1.34 PFLOP/s; forward of 122,880 x 1024 -> 512 1.78), else by the epilogue (122,880 x 256 -> 512 59 us: 1.09 PFLOP/s and 48%
// of the copy bandwidth; half of the rest is the stores, 3 to 8 us the gate).
//
// dt is rounded to bf16 (with bf16 rows) because the tensor cores take it so: each
// dx and dW is then about as far from the exact value as its own rounding puts it.
#include <algorithm>

#include "mt_linear.cuh"
#include "mt_parts.cuh"
#include "mt_tiles.cuh"

namespace mt {
namespace {

using tiles::Acc;
using tiles::Unit;

// The gate's factor and its derivative.  bf16 rows: by the hardware's exponential and reciprocal (2^-22 off).
template <typename T>
__device__ __forceinline__ float sigmoid_of(float u) {
  if constexpr (sizeof(T) == 4) {
    return 1.0f / (1.0f + expf(-u));
  } else {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(u * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
  }
}
constexpr float kGelu = 1.5957691216057308f, kCube = 0.044715f;  // 2 sqrt(2 / pi)

template <typename T, int GATE>
__device__ __forceinline__ float gate_of(float u) {
  if constexpr (GATE == MT_GATE_LINEAR) return u;
  if constexpr (GATE == MT_GATE_SIGMOID) return sigmoid_of<T>(u);
  if constexpr (GATE == MT_GATE_SILU) return u * sigmoid_of<T>(u);
  return u * sigmoid_of<T>(kGelu * fmaf(kCube * u * u, u, u));
}
// The factors of two bf16 columns (one column at a time: forward of 122,880 x 512 -> 512 85 us, two 82.5).
template <int GATE>
__device__ __forceinline__ f32x2 gate_of2(f32x2 u) {
  if constexpr (GATE == MT_GATE_LINEAR) return u;
  constexpr float kLog2e = 1.4426950408889634f;
  f32x2 t;
  if constexpr (GATE == MT_GATE_GELU) t = mul2(u, fma2(mul2(u, u), both(-kLog2e * kGelu * kCube), both(-kLog2e * kGelu)));
  else t = mul2(u, both(-kLog2e));
  float2 e = upk(t), r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(e.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(e.y));
  e = upk(add2(pk(e.x, e.y), both(1.0f)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(e.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(e.y));
  if constexpr (GATE == MT_GATE_SIGMOID) return pk(r.x, r.y);
  return mul2(u, pk(r.x, r.y));
}
template <typename T, int GATE>
__device__ __forceinline__ float2 gate_grad(float u) {
  if constexpr (GATE == MT_GATE_LINEAR) return make_float2(u, 1.0f);
  if constexpr (GATE == MT_GATE_SIGMOID) {
    const float p = sigmoid_of<T>(u);
    return make_float2(p, p * (1.0f - p));
  }
  if constexpr (GATE == MT_GATE_SILU) {
    const float p = sigmoid_of<T>(u), a = u * p;
    return make_float2(a, fmaf(a, 1.0f - p, p));
  }
  // (p is 0 or 1 long before the limit on u u, which keeps 0 from meeting infinity)
  const float uu = fminf(u * u, 1e30f), p = sigmoid_of<T>(kGelu * fmaf(kCube * uu, u, u)), a = u * p;
  return make_float2(a, fmaf(a * (1.0f - p), kGelu * fmaf(3.0f * kCube, uu, 1.0f), p));
}
template <int GATE>
struct GateIs {
  static constexpr int value = GATE;
};
// f(GateIs<gate>): the gate is known where the columns are gone through.
template <typename F>
__host__ __device__ __forceinline__ void by_gate(int gate, F&& f) {
  if (gate == MT_GATE_SILU) f(GateIs<MT_GATE_SILU>{});
  else if (gate == MT_GATE_GELU) f(GateIs<MT_GATE_GELU>{});
  else if (gate == MT_GATE_SIGMOID) f(GateIs<MT_GATE_SIGMOID>{});
  else f(GateIs<MT_GATE_LINEAR>{});
}

struct GatedParams {
  long long n;
  const long long* offsets;
  int32_t* status;
  const void* dh;
  void* out;  // h, or dt
  long long lddh, ldo;
  int groups, out_dim, jtiles;
  int u_col;  // dt: the column of du's first
  int gate;
  int steps;  // of the contraction, per pass
  int passes, a_part, b_part, b_second, promote;
  int reach, reach_dh;  // of out's rows and dh's
};

// T: the rows' type.  BACKWARD: dt instead of h.
template <typename T, bool BACKWARD>
struct Gated {
  using Params = GatedParams;
  static constexpr int kBN = 256;
  static constexpr bool kAMN = false, kBMN = false, kTwoB = true, kTeams = false, kKeep = false, kSingle = true, kTri = false;
  static constexpr int kStageOut = 2048;  // 32 rows x 64 bytes
  static constexpr bool kSplit = !BACKWARD || sizeof(T) == 2;
  static constexpr bool kAhead = BACKWARD && sizeof(T) == 2;  // dh of a tile's first columns is on its way before the tile
  const Params& p;
  const long long* off;
  const int* cum;
  int rank, rows_per_tile, quad, team, lane, group = 0;
  uint8_t* stage;
  uint4 dh[4];

  __device__ Gated(const Params& params, uint8_t* mem, int r) : p(params), rank(r) {
    long long* s_off = reinterpret_cast<long long*>(mem);
    int* s_cum = reinterpret_cast<int*>(s_off + p.groups + 1);
    load_offsets(p.offsets, p.groups, p.n, s_off, p.status);
    rows_per_tile = tiles::kBM * cluster();
    count_tiles(s_off, p.groups, rows_per_tile, s_cum);
    off = s_off;
    cum = s_cum;
  }
  static __device__ __forceinline__ int cluster() {
    int c;
    asm("mov.u32 %0, %cluster_nctaid.x;" : "=r"(c));
    return c;
  }
  __device__ long long units() const { return (long long)cum[p.groups] * p.jtiles; }
  // Units come in ascending order: the group is looked for from the last one's on.  Columns fastest: a row tile's products
  // read the same rows of x.
  __device__ Unit unit(long long u) {
    const unsigned rt = u <= 0xFFFFFFFFll ? (unsigned)u / (unsigned)p.jtiles : (unsigned)(u / p.jtiles);
    const int c = (int)(u - (long long)rt * p.jtiles);
    while (cum[group + 1] <= (int)rt) ++group;
    Unit x;
    x.g = group;
    x.row0 = (int)off[x.g] + ((int)rt - cum[x.g]) * rows_per_tile;
    x.end = (int)off[x.g + 1];
    x.ct0 = c;
    x.ct1 = c + 1;
    x.k0 = 0;
    x.k1 = p.steps;
    x.slot = 0;
    return x;
  }
  __device__ void warp(uint8_t* s, int q, int h, int l) {
    stage = s;
    quad = q;
    team = h;
    lane = l;
    const int J = BACKWARD ? 2 * p.u_col : p.out_dim;
    zero_outside<T>(off, p.groups, p.n, static_cast<T*>(p.out), p.ldo, J, tiles::kEpiWarps * 32, (h * 4 + q) * 32 + l);
  }
  __device__ void begin(const Unit&) {}
  __device__ void finish() {}
  __device__ void end(const Unit&) {}

  // 32 columns of dh as they lie, where they lie on 16 bytes
  __device__ __forceinline__ void fetch(const Unit& x, int col) {
    const long long r0 = x.row0 + rank * tiles::kBM + quad * 32;
    const T* from = static_cast<const T*>(p.dh) + (size_t)(r0 + lane) * p.lddh + col;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      dh[c] = make_uint4(0u, 0u, 0u, 0u);
      if (r0 + lane < x.end && col + c * 8 < p.out_dim) dh[c] = reinterpret_cast<const uint4*>(from)[c];
    }
  }
  __device__ __forceinline__ void ahead(const Unit& x, int ct) {
    if (p.reach_dh != tiles::kElements) fetch(x, ct * 128 + team * 64);
  }

  template <int CG>
  __device__ __forceinline__ void tile(const Unit& x, int ct, const Acc& acc, bool, bool) {
    by_gate(p.gate, [&](auto gate) { columns<CG, decltype(gate)::value>(x, ct, acc); });
  }
  template <int CG, int GATE>
  __device__ __forceinline__ void columns(const Unit& x, int ct, const Acc& acc) {
    const long long r0 = x.row0 + rank * tiles::kBM + quad * 32;
    const int rows = min(32, x.end - (int)r0);  // <= 0: none of this warp's rows is in the group
    T* out = static_cast<T*>(p.out);
    // Of the team's 64 columns the forward loads all at once: the accumulator is free for the next products before the
    // arithmetic begins.  (The backward has registers for 32.)  Teams in turns took as long in bf16, and fp32's product of 5003
    // rows, 100 to 333, 60 us instead of 39; four teams of 32 columns took 74 us for 122,880 x 256 -> 512 instead of 60.
    constexpr int kOnce = BACKWARD ? 1 : 2;
    uint32_t ys[kOnce][32], us[kOnce][32];
#pragma unroll(kOnce)
    for (int i = 0; i < 2; ++i) {
      const int col = ct * 128 + team * 64 + i * 32;
      uint32_t (&y)[32] = ys[BACKWARD ? 0 : i];
      uint32_t (&u)[32] = us[BACKWARD ? 0 : i];
      if (BACKWARD || i == 0) {
#pragma unroll
        for (int k = 0; k < kOnce; ++k) {
          acc.load(team * 64 + (i + k) * 32, ys[k]);
          acc.load(128 + team * 64 + (i + k) * 32, us[k]);
        }
      }
      uint32_t d[BACKWARD ? 32 : 1];  // dh: bf16 pairs as they lie in the first 16, or fp32
      if constexpr (BACKWARD) {
        if constexpr (sizeof(T) == 2) {
          if (p.reach_dh != tiles::kElements) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              d[4 * j] = dh[j].x;
              d[4 * j + 1] = dh[j].y;
              d[4 * j + 2] = dh[j].z;
              d[4 * j + 3] = dh[j].w;
            }
            if (i == 0) fetch(x, col + 32);
          }
        }
        if (sizeof(T) == 4 || p.reach_dh == tiles::kElements) {
          float f[32];
          tiles::load_rows<T>(stage, lane, f, static_cast<const T*>(p.dh), p.lddh, r0, col < p.out_dim ? rows : 0, col, p.out_dim, p.reach_dh);
          if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int j = 0; j < 16; ++j) d[j] = bf16x2_of(f[2 * j], f[2 * j + 1]);  // (bf16 already)
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) d[j] = __float_as_uint(f[j]);
          }
        }
      }
      if (BACKWARD || i == 0) {
        tc::tmem_load_wait();
#pragma unroll
        for (int k = 0; k < kOnce; ++k) {
          tc::tmem_loaded(ys[k]);
          tc::tmem_loaded(us[k]);
        }
        if (!BACKWARD || i == 1) acc.release<CG>(lane);
      }
      // y becomes h, or dy; u du.  bf16: two columns to a word
      constexpr int kWords = sizeof(T) == 2 ? 16 : 32;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if constexpr (!BACKWARD && sizeof(T) == 2) {
          const float2 h = upk(mul2(pk(__uint_as_float(y[2 * j]), __uint_as_float(y[2 * j + 1])),
                                    gate_of2<GATE>(pk(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1])))));
          y[j] = bf16x2_of(h.x, h.y);
          continue;
        }
        float a[2], b[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float yy = __uint_as_float(y[2 * j + e]), uu = __uint_as_float(u[2 * j + e]);
          if constexpr (BACKWARD) {
            float g;
            if constexpr (sizeof(T) == 2) g = __uint_as_float(e == 0 ? d[j] << 16 : d[j] & 0xFFFF0000u);
            else g = __uint_as_float(d[2 * j + e]);
            const float2 t = gate_grad<T, GATE>(uu);
            a[e] = g * t.x;
            b[e] = g * yy * t.y;
          } else {
            a[e] = yy * gate_of<T, GATE>(uu);
          }
        }
        if constexpr (sizeof(T) == 2) {
          y[j] = bf16x2_of(a[0], a[1]);
          if constexpr (BACKWARD) u[j] = bf16x2_of(b[0], b[1]);
        } else {
          y[2 * j] = __float_as_uint(a[0]);
          y[2 * j + 1] = __float_as_uint(a[1]);
          if constexpr (BACKWARD) {
            u[2 * j] = __float_as_uint(b[0]);
            u[2 * j + 1] = __float_as_uint(b[1]);
          }
        }
      }
#pragma unroll
      for (int h = 0; h < kWords / 16; ++h) {
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j] = y[h * 16 + j];
        tiles::store_rows<T>(stage, lane, w, out, p.ldo, r0, rows, col + h * 16, p.out_dim, p.reach);
        if constexpr (BACKWARD) {
#pragma unroll
          for (int j = 0; j < 16; ++j) w[j] = u[h * 16 + j];
          tiles::store_rows<T>(stage, lane, w, out + p.u_col, p.ldo, r0, rows, col + h * 16, p.out_dim, p.reach);
        }
      }
    }
  }
};

// ---- forward of a few rows --------------------------------------------------------------
//
// A few tokens being served: the weights' bytes and the latency of one load are all there is.  A warp takes two
// neighbouring rows of Wy and the same two of Wu (32 lanes by eight columns a step, the loads in flight together) against
// two rows of x; lanes then join by shuffles and h is made in registers.  A group's further rows are tasks of their own, so
// a batch costs the same whichever groups its rows are in.
constexpr int kFewRows = 2, kFewOuts = 2, kFewBlocks = 3;

struct FewParams {
  long long n;
  const long long* offsets;
  int32_t* status;
  const void* x;
  long long ldx;
  const void* w;
  void* h;
  long long ldh;
  int groups, in_dim, out_dim, gate;
};

template <typename T>
__global__ void __launch_bounds__(256, kFewBlocks) k_gated_few(const FewParams p) {
  extern __shared__ long long s_off[];
  int* s_cum = reinterpret_cast<int*>(s_off + p.groups + 1);
  load_offsets(p.offsets, p.groups, p.n, s_off, p.status);
  count_tiles(s_off, p.groups, kFewRows, s_cum);
  const int lane = threadIdx.x & 31;
  T* H = static_cast<T*>(p.h);
  zero_outside<T>(s_off, p.groups, p.n, H, p.ldh, p.out_dim, blockDim.x, threadIdx.x);
  const int per_tile = (p.out_dim + kFewOuts - 1) / kFewOuts;
  const int warps = (gridDim.x * blockDim.x) >> 5;
  for (int t = (blockIdx.x * blockDim.x + threadIdx.x) >> 5; t < s_cum[p.groups] * per_tile; t += warps) {
    const int q = t / per_tile, j0 = (t - q * per_tile) * kFewOuts, g = tile_group(s_cum, p.groups, q);
    const int outs = min(kFewOuts, p.out_dim - j0);
    const int r0 = (int)s_off[g] + (q - s_cum[g]) * kFewRows, rows = min(kFewRows, (int)s_off[g + 1] - r0);
    const T* W = static_cast<const T*>(p.w) + ((size_t)g * 2 * p.out_dim + j0) * p.in_dim;
    f32x2 acc[kFewRows][2 * kFewOuts] = {};
#pragma unroll 2
    for (int i = lane * 8; i < p.in_dim; i += 256) {
      Raw8<T> w[2 * kFewOuts], x[kFewRows];  // every load of the step issued before the first is used
#pragma unroll
      for (int o = 0; o < 2 * kFewOuts; ++o) {  // the rows of Wy, then those of Wu
        const int row = (o % kFewOuts < outs ? o % kFewOuts : 0) + (o < kFewOuts ? 0 : p.out_dim);
        w[o] = load8<T, true>(Rows{const_cast<T*>(W), (int64_t)p.in_dim, nullptr, nullptr}, row, i >> 3, p.in_dim);
      }
#pragma unroll
      for (int r = 0; r < kFewRows; ++r)
        if (r < rows) x[r] = load8<T, true>(Rows{const_cast<void*>(p.x), p.ldx, nullptr, nullptr}, r0 + r, i >> 3, p.in_dim);
#pragma unroll
      for (int r = 0; r < kFewRows; ++r) {
        if (r >= rows) break;
        f32x2 v[4];
        widen8<T>(x[r], false, v);
#pragma unroll
        for (int o = 0; o < 2 * kFewOuts; ++o) {
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
      float s[2 * kFewOuts];
#pragma unroll
      for (int o = 0; o < 2 * kFewOuts; ++o) {
        s[o] = pair_sum(acc[r][o]);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s[o] += __shfl_xor_sync(kFull, s[o], d);
      }
#pragma unroll
      for (int o = 0; o < kFewOuts; ++o)
        if (lane == o && o < outs)
          by_gate(p.gate, [&](auto gate) { H[row_offset(r0 + r, p.ldh) + j0 + o] = from_f<T>(s[o] * gate_of<T, decltype(gate)::value>(s[kFewOuts + o])); });
    }
  }
}

// ---- host --------------------------------------------------------------------------------------

// The forward of few rows goes to k_gated_few: up to kFewTc rows per group on average (bf16) or kFewParts (fp32, whose weights
// would be copied first), as long as each warp that the SMs hold has no more than kFewTasks tasks.  Measured
// against the tiles: bf16, 512 -> 1024, 8 tokens on 8 experts 6.4 and 8.6 us, 16 on 8 7.6 and 8.5, 24 on 8 10.7 and 8.5, 64 on 32
// (more tasks) 19.8 and 16.6; 1 token, 1024 -> 4096, 5.8 and 9.8; 16 on 8, 2048 -> 2048, 31.8 and 30.3.  fp32: 64 on 8, 512 ->
// 1024, 25.3 and 39.0, 128 on 8 46.3 and 39.1 (each further pair of a group's rows reads its weights again: 64 rows on 8 experts
// 134 MB, from L2 at 5 TB/s, where the weights once are 5 us of HBM).
constexpr int kFewTc = 2, kFewParts = 8, kFewTasks = 6;
bool few(const mt_gated_linear& c) {
  const long long tiles = (c.n + std::min<long long>(c.n, c.groups) * (kFewRows - 1)) / kFewRows;  // at most
  const long long tasks = tiles * ((c.out_dim + kFewOuts - 1) / kFewOuts), held = (long long)sm_count() * kFewBlocks * 8;
  return c.n <= (long long)(c.dtype == MT_BF16 ? kFewTc : kFewParts) * c.groups && tasks <= kFewTasks * held && c.in_dim % 8 == 0 &&
         (c.n <= 1 || c.ldx * elem_bytes(c.dtype) % 16 == 0) && is_aligned(c.x, 16) && is_aligned(c.w, 16);
}

// How a call's operands reach the tensor cores.
struct Layout {
  bool copies;     // x and W are copied first: fp32 in three parts, bf16 padded to multiples of 8
  int parts;
  int64_t k, m;    // in_dim of a part and out_dim, padded
  size_t x, w, dt, dx, dw, partial, total;  // where the workspace has them
};

bool fits(const mt_gated_linear& c) {
  return c.in_dim % 8 == 0 && c.out_dim % 8 == 0 && (c.n <= 1 || c.ldx % 8 == 0) && is_aligned(c.x, 16) && is_aligned(c.w, 16);
}

Layout layout_of(const mt_gated_linear& c, bool backward) {
  Layout l{};
  l.parts = c.dtype == MT_F32 ? 3 : 1;
  if (!backward && few(c)) return l;
  l.copies = c.dtype == MT_F32 || !fits(c);
  l.k = part_columns(c.in_dim, l.parts);
  l.m = c.dtype == MT_F32 ? c.out_dim : (c.out_dim + 7) / 8 * 8;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align_up(bytes, 256);
    return here;
  };
  const size_t e = elem_bytes(c.dtype);
  if (l.copies) {
    l.x = take((size_t)c.n * l.parts * l.k * 2);
    l.w = take((size_t)c.groups * 2 * l.m * l.parts * l.k * 2);
  }
  if (backward) {
    l.dt = take((size_t)c.n * 2 * l.m * e);
    const bool padded = l.copies && c.dtype == MT_BF16;
    if (padded) {
      l.dx = take((size_t)c.n * l.k * 2);
      l.dw = take((size_t)c.groups * 2 * l.m * l.k * 2);
    }
    l.partial = take(partial_bytes(c.n, c.groups, padded ? (int32_t)l.k : c.in_dim, (int32_t)(2 * l.m)));
  }
  l.total = at;
  return l;
}

int check(const mt_gated_linear* c) {
  if (c == nullptr || (c->dtype != MT_F32 && c->dtype != MT_BF16)) return MT_EINVAL;
  if (c->gate < MT_GATE_LINEAR || c->gate > MT_GATE_GELU) return MT_EINVAL;
  if (c->n < 0 || c->n > MT_MAX_BLOCK_ROWS || c->groups < 1 || c->groups > MT_MAX_GROUPS) return MT_EINVAL;
  if (c->in_dim < 1 || c->in_dim > MT_MAX_BLOCK_DIM || c->out_dim < 1 || c->out_dim > MT_MAX_BLOCK_DIM) return MT_EINVAL;
  if (c->offsets == nullptr || !is_aligned(c->offsets, 8) || !is_aligned(c->status, 4)) return MT_EINVAL;
  if (c->w == nullptr || !is_aligned(c->w, elem_bytes(c->dtype))) return MT_EINVAL;
  if (c->n > 0 && !rows_ok(c->x, c->ldx, c->in_dim, c->dtype)) return MT_EINVAL;
  return MT_OK;
}

template <typename T, bool BACKWARD>
cudaError_t launch_product(const mt_gated_linear& c, const Layout& l, GatedParams p, char* ws, cudaStream_t s) {
  const void* x = l.copies ? ws + l.x : c.x;
  const void* w = l.copies ? ws + l.w : c.w;
  if (l.copies) {
    cudaError_t e = launch_parts(c.x, c.ldx, 1, c.n, c.n, c.in_dim, c.dtype, reinterpret_cast<__nv_bfloat16*>(ws + l.x), s);
    if (e == cudaSuccess)
      e = launch_parts(c.w, c.in_dim, (int64_t)c.groups * 2, c.out_dim, l.m, c.in_dim, c.dtype, reinterpret_cast<__nv_bfloat16*>(ws + l.w), s);
    if (e != cudaSuccess) return e;
  }
  p.n = c.n;
  p.offsets = reinterpret_cast<const long long*>(c.offsets);
  p.status = c.status;
  p.groups = c.groups;
  p.out_dim = c.out_dim;
  p.jtiles = (c.out_dim + 127) / 128;
  p.gate = c.gate;
  p.steps = (int)((l.k + tiles::kBK - 1) / tiles::kBK);
  p.passes = l.parts == 3 ? 6 : 1;
  p.a_part = p.b_part = (int)l.k;
  p.b_second = (int)l.m;
  p.promote = 1 << 30;
  const bool pair = sizeof(T) == 2 && l.k > 2 * tiles::kBK && c.n / c.groups >= 256 && c.n / 256 * p.jtiles >= sm_count() / 2;
  CUtensorMap a, b;
  const uint64_t width = (uint64_t)l.parts * l.k;
  if (!tc::encode_bf16(&a, 2, x, width, c.n, l.copies ? width : (c.n <= 1 ? width : c.ldx), 1, 0, tiles::kBK, tiles::kBM)) return cudaErrorInvalidValue;
  if (!tc::encode_bf16(&b, 3, w, width, 2 * l.m, width, c.groups, width * 2 * l.m, tiles::kBK, 128)) return cudaErrorInvalidValue;
  const size_t extra = rows_smem(c.groups), most = rows_smem(MT_MAX_GROUPS);
  const char* name = BACKWARD ? "k_gated_backward" : "k_gated_forward";
  const long long units1 = (c.n / 128 + c.groups) * p.jtiles, units2 = (c.n / 256 + c.groups) * p.jtiles;  // at most
  if constexpr (sizeof(T) == 2) {
    if (pair) return tiles::launch<Gated<T, BACKWARD>, 2>(name, a, b, p, units2, extra, most, s);
  }
  return tiles::launch<Gated<T, BACKWARD>, 1>(name, a, b, p, units1, extra, most, s);
}

}  // namespace
}  // namespace mt

extern "C" {

size_t mt_gated_linear_workspace_bytes(const mt_gated_linear* c, int backward) {
  using namespace mt;
  if (check(c) != MT_OK) return 0;
  return layout_of(*c, backward != 0).total;
}

int mt_gated_linear_forward(const mt_gated_linear* c, void* h, int64_t ldh, void* ws, size_t ws_bytes, mt_stream stream) {
  using namespace mt;
  const int rc = check(c);
  if (rc != MT_OK) return rc;
  if (c->n == 0) return MT_OK;
  if (!rows_ok(h, ldh, c->out_dim, c->dtype)) return MT_EINVAL;
  const Layout l = layout_of(*c, false);
  if (l.total > 0 && (ws == nullptr || !is_aligned(ws, 256) || ws_bytes < l.total)) return MT_ENOSPACE;
  Regions all;
  all.in(Rows{const_cast<void*>(c->x), c->ldx, nullptr, nullptr}, c->n, c->in_dim, c->dtype);
  all.in(whole_region(c->w, (size_t)c->groups * 2 * c->out_dim * c->in_dim * elem_bytes(c->dtype)));
  all.in(whole_region(c->offsets, (size_t)(c->groups + 1) * 8));
  all.out(Rows{h, ldh, nullptr, nullptr}, c->n, c->out_dim, c->dtype);
  if (l.total > 0) all.out(whole_region(ws, l.total));
  if (all.clash()) return MT_EINVAL;
  if (few(*c)) {
    const FewParams f{c->n, reinterpret_cast<const long long*>(c->offsets), c->status, c->x, c->n <= 1 ? c->in_dim : c->ldx, c->w, h, ldh,
                      c->groups, c->in_dim, c->out_dim, c->gate};
    const long long tasks = (c->n + std::min<long long>(c->n, c->groups) * (kFewRows - 1)) / kFewRows * ((c->out_dim + kFewOuts - 1) / kFewOuts);
    const int grid = grid_for(tasks * 32, 256, kFewBlocks);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    MT_LAUNCH("k_gated_few", s);
    if (c->dtype == MT_F32) k_gated_few<float><<<grid, 256, rows_smem(c->groups), s>>>(f);
    else k_gated_few<__nv_bfloat16><<<grid, 256, rows_smem(c->groups), s>>>(f);
    return cudaGetLastError() == cudaSuccess ? MT_OK : MT_ECUDA;
  }
  GatedParams p{};
  p.out = h;
  p.ldo = ldh;
  p.reach = tiles::reach_of(h, ldh, c->out_dim, elem_bytes(c->dtype));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* w = static_cast<char*>(ws);
  const cudaError_t e = c->dtype == MT_F32 ? launch_product<float, false>(*c, l, p, w, s) : launch_product<__nv_bfloat16, false>(*c, l, p, w, s);
  return e == cudaSuccess ? MT_OK : MT_ECUDA;
}

int mt_gated_linear_backward(const mt_gated_linear* c, const void* dh, int64_t lddh, void* dx, int64_t lddx, void* dw, void* ws,
                             size_t ws_bytes, mt_stream stream) {
  using namespace mt;
  const int rc = check(c);
  if (rc != MT_OK) return rc;
  if (dx == nullptr && dw == nullptr) return MT_EINVAL;
  if (c->n > 0 && !rows_ok(dh, lddh, c->out_dim, c->dtype)) return MT_EINVAL;
  if (c->n > 0 && dx != nullptr && !rows_ok(dx, lddx, c->in_dim, c->dtype)) return MT_EINVAL;
  if (!is_aligned(dw, elem_bytes(c->dtype))) return MT_EINVAL;
  const Layout l = layout_of(*c, true);
  if (ws == nullptr || !is_aligned(ws, 256) || ws_bytes < l.total) return MT_ENOSPACE;
  const size_t e = elem_bytes(c->dtype), weights = (size_t)c->groups * 2 * c->out_dim * c->in_dim * e;
  Regions all;
  if (c->n > 0) {
    all.in(Rows{const_cast<void*>(dh), lddh, nullptr, nullptr}, c->n, c->out_dim, c->dtype);
    all.in(Rows{const_cast<void*>(c->x), c->ldx, nullptr, nullptr}, c->n, c->in_dim, c->dtype);
    if (dx != nullptr) all.out(Rows{dx, lddx, nullptr, nullptr}, c->n, c->in_dim, c->dtype);
  }
  all.in(whole_region(c->w, weights));
  all.in(whole_region(c->offsets, (size_t)(c->groups + 1) * 8));
  if (dw != nullptr) all.out(whole_region(dw, weights));
  all.out(whole_region(ws, l.total));
  if (all.clash()) return MT_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (c->n == 0) {
    if (dw == nullptr) return MT_OK;
    return cudaMemsetAsync(dw, 0, weights, s) == cudaSuccess ? MT_OK : MT_ECUDA;
  }
  char* base = static_cast<char*>(ws);
  const bool padded = l.copies && c->dtype == MT_BF16;
  GatedParams p{};
  p.dh = dh;
  p.lddh = lddh;
  p.out = base + l.dt;
  p.ldo = 2 * l.m;
  p.u_col = (int)l.m;
  p.reach = tiles::reach_of(p.out, l.m, l.m, e);  // (dt's own rows: no column behind the last is the user's)
  p.reach_dh = tiles::reach_of(dh, c->n <= 1 ? c->out_dim : lddh, c->out_dim, e);
  cudaError_t err = cudaSuccess;
  err = c->dtype == MT_F32 ? launch_product<float, true>(*c, l, p, base, s) : launch_product<__nv_bfloat16, true>(*c, l, p, base, s);
  const int32_t k = padded ? (int32_t)l.k : c->in_dim, m2 = (int32_t)(2 * l.m);
  if (dx != nullptr && err == cudaSuccess) {
    LinearRows r{};
    r.n = c->n;
    r.groups = c->groups;
    r.offsets = reinterpret_cast<const long long*>(c->offsets);
    r.a = base + l.dt;
    r.lda = 2 * l.m;
    r.w = padded ? base + l.w : c->w;
    r.wg = (size_t)k * m2;
    r.wi = k;
    r.wj = 1;
    r.c = padded ? static_cast<void*>(base + l.dx) : dx;
    r.ldc = padded ? l.k : lddx;
    r.I = m2;
    r.J = k;
    r.status = c->status;
    r.any_c = c->dtype == MT_BF16;  // (the other operands fit: dx of 40,009 rows on 32 experts, 1024 -> 2048, on one element 479 us of 461, by the fp32 pipes 10,500)
    err = launch_linear_rows(r, c->dtype, s);
    if (padded && err == cudaSuccess)
      err = launch_unpad(reinterpret_cast<__nv_bfloat16*>(base + l.dx), l.k, 1, c->n, c->n, c->in_dim, static_cast<__nv_bfloat16*>(dx), lddx, s);
  }
  if (dw != nullptr && err == cudaSuccess) {
    LinearWeights q{};
    q.n = c->n;
    q.groups = c->groups;
    q.offsets = reinterpret_cast<const long long*>(c->offsets);
    q.status = c->status;
    q.dy = base + l.dt;
    q.lddy = 2 * l.m;
    q.x = padded ? Rows{base + l.x, l.k, nullptr, nullptr} : Rows{const_cast<void*>(c->x), c->n <= 1 ? c->in_dim : c->ldx, nullptr, nullptr};
    q.K = k;
    q.M = m2;
    q.chosen = reinterpret_cast<int*>(base + l.partial);
    q.part = reinterpret_cast<float*>(base + l.partial) + 64;
    if (c->dtype == MT_F32) q.dw = static_cast<float*>(dw);
    else q.dw16 = padded ? reinterpret_cast<__nv_bfloat16*>(base + l.dw) : static_cast<__nv_bfloat16*>(dw);
    err = launch_linear_weights(q, c->dtype, s);
    if (err == cudaSuccess) err = launch_linear_sums(q, s);
    if (padded && err == cudaSuccess)
      err = launch_unpad(reinterpret_cast<__nv_bfloat16*>(base + l.dw), l.k, (int64_t)c->groups * 2, c->out_dim, l.m, c->in_dim,
                         static_cast<__nv_bfloat16*>(dw), c->in_dim, s);
  }
  return err == cudaSuccess ? MT_OK : MT_ECUDA;
}

}  // extern "C"
