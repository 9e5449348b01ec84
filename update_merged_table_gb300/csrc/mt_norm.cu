// The norm after a block, its gate and its residual scale, the residual sum and
// the next block's norm, in one pass over the rows; and their backward.
//
//   yh = norm(y)   t = wp * yh + bp   a = act(u)   z = x + s * t * a
//   zh = norm(z)   h = wq * zh + bq
//
// with one set of parameters (wp, bp, s, wq, bq) per group of rows.  A row is
// held in registers by a team of lanes (16 columns per lane) from its first
// load to its last store, so every tensor is read once and written once and
// HBM bandwidth is the bound.  The backward keeps no statistics: means and
// deviations come again from y and z, which it has in registers anyway, so
// checkpoints in 8 bits need nothing stored beside them.
//
// Kernels:
//  k_norm_fwd    teams stride over the rows.
//  k_norm_bwd    a block per chunk of rows of one group: the parameter
//                gradients of the chunk stay in registers and leave as one
//                partial sum per chunk (no atomics, so the sums have one order).
//  k_norm_sums   the chunks' partial sums of each group, in fp64.
#include <algorithm>

#include "mt_block.cuh"

namespace mt {
namespace {

constexpr int kNV = 2;         // vectors of eight columns per lane
constexpr int kNormThreads = 256;
constexpr int kSums = 5;       // partial sums: dwp, dbp, ds, dwq, dbq

struct NormParams {
  long long n;
  int d, groups, kind, gate;
  float eps;
  const long long* offsets;
  int32_t* status;
  const float *wp, *bp, *sc, *wq, *bq;
  Rows x, y, u, z, h;            // forward
  Rows dz, dh, dx, dy, du;       // backward (with y, u, z)
  float* part;                   // [chunks][kSums][d]
  float *dwp, *dbp, *dsc, *dwq, *dbq;
  int log_team;                  // log2 lanes per row
  int chunk_rows, chunks;        // chunks: upper bound (the launch's grid)
  int wide;                      // parameters reached with 16-byte loads
};

// Sums a and b over a team: shuffles inside a warp, shared memory across a team's warps.  A team of more than one
// warp owns the named barrier 1 + team; `slot` alternates so that one barrier per call is enough.
__device__ __forceinline__ void team_sum2(float& a, float& b, int team_lanes, float2* s_red, int& slot) {
  const int in_warp = team_lanes < 32 ? team_lanes : 32;
  for (int o = in_warp >> 1; o > 0; o >>= 1) {
    a += __shfl_xor_sync(kFull, a, o);
    b += __shfl_xor_sync(kFull, b, o);
  }
  if (team_lanes <= 32) return;
  const int warp = threadIdx.x >> 5, warps = team_lanes >> 5, first = warp / warps * warps;
  float2* buf = s_red + slot * 16;
  if ((threadIdx.x & 31) == 0) buf[warp] = make_float2(a, b);
  asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / warps), "r"(team_lanes) : "memory");
  a = b = 0.0f;
  for (int k = 0; k < warps; ++k) {
    const float2 v = buf[first + k];
    a += v.x;
    b += v.y;
  }
  slot ^= 1;
}

// Eight parameters of a group's row, `none` for an absent parameter and zero past d.
__device__ __forceinline__ void param8(const float* p, int g, int vec, int d, int wide, float none, float f[8]) {
  const int c0 = vec * 8;
  if (p == nullptr || c0 >= d) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = none;
    return;
  }
  p += (size_t)g * d + c0;
  if (wide) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = c0 + j < d ? __ldg(p + j) : 0.0f;
  }
}

// The gate's factor a = act(u) and its derivative.  fp32 rows take the accurate exponential and division; for bf16
// rows the fast ones (a few units of 2^-22) are far below the rounding of the result.
template <typename T>
__device__ __forceinline__ float gate_value(int gate, float u, float& da) {
  if (gate == MT_GATE_LINEAR) {
    da = 1.0f;
    return u;
  }
  float p;
  if constexpr (sizeof(T) == 4) p = 1.0f / (1.0f + expf(-u));
  else p = __frcp_rn(1.0f + __expf(-u));
  if (gate == MT_GATE_SIGMOID) {
    da = p * (1.0f - p);
    return p;
  }
  da = p * (1.0f + u * (1.0f - p));
  // silu(-inf) = -inf * 0 is NaN by the formula; u * p keeps that
  return u * p;
}

// Mean (layer norm; 0 for rms) and inverse deviation of the row held in v; columns past d are zero and stay out.
__device__ __forceinline__ void row_stats(const float (&v)[kNV][8], const NormParams& p, int team, int lt, float2* s_red,
                                          int& slot, float& mean, float& r) {
  float a = 0.0f, b = 0.0f;
  mean = 0.0f;
  const float inv_d = 1.0f / (float)p.d;
  if (p.kind == MT_NORM_LAYER) {
#pragma unroll
    for (int k = 0; k < kNV; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) a += v[k][j];
    team_sum2(a, b, team, s_red, slot);
    mean = a * inv_d;
    a = 0.0f;
  }
#pragma unroll
  for (int k = 0; k < kNV; ++k) {
    const int left = p.d - (k * team + lt) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float c = j < left ? v[k][j] - mean : 0.0f;
      a += c * c;
    }
  }
  b = 0.0f;
  team_sum2(a, b, team, s_red, slot);
  r = rsqrtf(a * inv_d + p.eps);
}

template <typename T, bool AL, int THREADS>
__global__ void __launch_bounds__(THREADS) k_norm_fwd(const NormParams p) {
  extern __shared__ long long s_off[];
  __shared__ float2 s_red[32];
  load_offsets(p.offsets, p.groups, p.n, s_off, p.status);
  const int team = 1 << p.log_team;
  const int lt = threadIdx.x & (team - 1);
  const int sub = threadIdx.x >> p.log_team;
  const int teams = blockDim.x >> p.log_team;  // teams per block
  const bool has_y = p.y.data != nullptr, has_u = p.u.data != nullptr, has_h = p.wq != nullptr;
  const bool put_z = p.z.data != nullptr || p.z.codes != nullptr;
  int slot = 0;
  // every team of a block runs the same number of rounds, so the shuffles and barriers meet
  for (long long base = (long long)blockIdx.x * teams; base < p.n; base += (long long)gridDim.x * teams) {
    const long long row = base + sub;
    const int g = row < p.n ? row_group(s_off, p.groups, row) : -1;
    const bool in = row < p.n, live = g >= 0;
    Raw8<T> rx[kNV], ry[kNV], ru[kNV];
#pragma unroll
    for (int k = 0; k < kNV; ++k) {
      const int vec = k * team + lt, dd = live ? p.d : 0;
      const long long rr = live ? row : 0;
      rx[k] = load8<T, AL>(p.x, rr, vec, dd);
      if (has_y) ry[k] = load8<T, AL>(p.y, rr, vec, dd);
      if (has_u) ru[k] = load8<T, AL>(p.u, rr, vec, dd);
    }
    float z[kNV][8], mean, r;
#pragma unroll
    for (int k = 0; k < kNV; ++k) widen8<T>(rx[k], false, z[k]);
    if (has_y) {
      float y[kNV][8];
#pragma unroll
      for (int k = 0; k < kNV; ++k) {
        widen8<T>(ry[k], false, y[k]);
        if (p.y.codes != nullptr) store_packed8<AL>(p.y, row, k * team + lt, p.d, y[k], in);
      }
      row_stats(y, p, team, lt, s_red, slot, mean, r);
#pragma unroll
      for (int k = 0; k < kNV; ++k) {
        const int vec = k * team + lt;
        float w[8], b[8], s[8], u[8];
        param8(p.wp, live ? g : 0, vec, p.d, p.wide, 1.0f, w);
        param8(p.bp, live ? g : 0, vec, p.d, p.wide, 0.0f, b);
        param8(p.sc, live ? g : 0, vec, p.d, p.wide, 1.0f, s);
        if (has_u) {
          widen8<T>(ru[k], false, u);
          if (p.u.codes != nullptr) store_packed8<AL>(p.u, row, vec, p.d, u, in);
        }
        const int left = p.d - vec * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float t = (w[j] * ((y[k][j] - mean) * r) + b[j]) * s[j], da;
          if (has_u) t *= gate_value<T>(p.gate, u[j], da);
          if (live && j < left) z[k][j] += t;
        }
      }
    }
    if (has_h) row_stats(z, p, team, lt, s_red, slot, mean, r);
#pragma unroll
    for (int k = 0; k < kNV; ++k) {
      const int vec = k * team + lt;
      if (has_h) {
        float w[8], b[8], h[8];
        param8(p.wq, live ? g : 0, vec, p.d, p.wide, 1.0f, w);
        param8(p.bq, live ? g : 0, vec, p.d, p.wide, 0.0f, b);
        const int left = p.d - vec * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = live && j < left ? w[j] * ((z[k][j] - mean) * r) + b[j] : 0.0f;
        if (in) store8<T, AL>(p.h.data, p.h.ld, row, vec, p.d, h);
        if (p.h.codes != nullptr) store_packed8<AL>(p.h, row, vec, p.d, h, in);
      }
      if (put_z) {
        if (p.z.data != nullptr && in) store8<T, AL>(p.z.data, p.z.ld, row, vec, p.d, z[k]);
        if (p.z.codes != nullptr) store_packed8<AL>(p.z, row, vec, p.d, z[k], in);
      }
    }
  }
}

// dv = r * (dvh - [mean dvh] - vh * mean(dvh * vh)), the gradient through a norm, in place of dvh.
__device__ __forceinline__ void norm_grad(float (&dvh)[kNV][8], const float (&vh)[kNV][8], float r, const NormParams& p,
                                          int team, int lt, float2* s_red, int& slot) {
  float a = 0.0f, b = 0.0f;
#pragma unroll
  for (int k = 0; k < kNV; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      a += dvh[k][j] * vh[k][j];
      b += dvh[k][j];
    }
  team_sum2(a, b, team, s_red, slot);
  const float inv_d = 1.0f / (float)p.d;
  const float ma = a * inv_d, mb = p.kind == MT_NORM_LAYER ? b * inv_d : 0.0f;
#pragma unroll
  for (int k = 0; k < kNV; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) dvh[k][j] = r * (dvh[k][j] - mb - vh[k][j] * ma);
}

template <typename T, bool AL, int THREADS>
__global__ void __launch_bounds__(THREADS) k_norm_bwd(const NormParams p) {
  extern __shared__ long long s_off[];  // [groups + 1], then int [groups + 1] chunks before each group
  __shared__ float2 s_red[32];
  __shared__ float s_sum[8192];         // one parameter's sums of the block's teams: teams * d <= 8192
  int* s_cum = reinterpret_cast<int*>(s_off + p.groups + 1);
  load_offsets(p.offsets, p.groups, p.n, s_off, p.status);
  count_tiles(s_off, p.groups, p.chunk_rows, s_cum);
  const int team = 1 << p.log_team;
  const int lt = threadIdx.x & (team - 1);
  const int sub = threadIdx.x >> p.log_team;
  const int teams = blockDim.x >> p.log_team;
  const bool has_y = p.y.data != nullptr || p.y.codes != nullptr, has_u = p.u.data != nullptr || p.u.codes != nullptr;
  const bool has_h = p.wq != nullptr, has_dz = p.dz.data != nullptr;
  const bool y8 = p.y.data == nullptr, u8 = p.u.data == nullptr, z8 = p.z.data == nullptr;
  const int total = s_cum[p.groups];
  int slot = 0;

  // rows in no group: their gradients are zero
  const long long outside = s_off[0] + (p.n - s_off[p.groups]);
  for (long long q = (long long)blockIdx.x * teams + sub; q < outside; q += (long long)gridDim.x * teams) {
    const long long row = q < s_off[0] ? q : q - s_off[0] + s_off[p.groups];
    float zero[8] = {};
#pragma unroll
    for (int k = 0; k < kNV; ++k) {
      const int vec = k * team + lt;
      store8<T, AL>(p.dx.data, p.dx.ld, row, vec, p.d, zero);
      if (has_y) store8<T, AL>(p.dy.data, p.dy.ld, row, vec, p.d, zero);
      if (has_u) store8<T, AL>(p.du.data, p.du.ld, row, vec, p.d, zero);
    }
  }

  for (int c = blockIdx.x; c < total; c += gridDim.x) {
    const int g = tile_group(s_cum, p.groups, c);
    const long long first = s_off[g] + (long long)(c - s_cum[g]) * p.chunk_rows;
    const long long last = min(first + p.chunk_rows, s_off[g + 1]);
    float acc[kSums][kNV][8];
#pragma unroll
    for (int q = 0; q < kSums; ++q)
#pragma unroll
      for (int k = 0; k < kNV; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[q][k][j] = 0.0f;
    for (long long base = first; base < last; base += teams) {
      const long long row = base + sub;
      const bool live = row < last;
      const int dd = live ? p.d : 0;
      const long long rr = live ? row : first;
      Raw8<T> ry[kNV], ru[kNV], rz[kNV], rdz[kNV], rdh[kNV];
#pragma unroll
      for (int k = 0; k < kNV; ++k) {
        const int vec = k * team + lt;
        if (has_h) {
          rz[k] = load8<T, AL>(p.z, rr, vec, dd);
          rdh[k] = load8<T, AL>(p.dh, rr, vec, dd);
        }
        if (has_dz) rdz[k] = load8<T, AL>(p.dz, rr, vec, dd);
        if (has_y) ry[k] = load8<T, AL>(p.y, rr, vec, dd);
        if (has_u) ru[k] = load8<T, AL>(p.u, rr, vec, dd);
      }
      float D[kNV][8], mean, r;
#pragma unroll
      for (int k = 0; k < kNV; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) D[k][j] = 0.0f;
      if (has_h) {  // through the next block's norm
        float zh[kNV][8];
#pragma unroll
        for (int k = 0; k < kNV; ++k) widen8<T>(rz[k], z8, zh[k]);
        row_stats(zh, p, team, lt, s_red, slot, mean, r);
#pragma unroll
        for (int k = 0; k < kNV; ++k) {
          const int vec = k * team + lt, left = p.d - vec * 8;
          float dh[8], w[8];
          widen8<T>(rdh[k], false, dh);
          param8(p.wq, g, vec, p.d, p.wide, 1.0f, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            zh[k][j] = live && j < left ? (zh[k][j] - mean) * r : 0.0f;
            acc[3][k][j] += dh[j] * zh[k][j];
            acc[4][k][j] += dh[j];
            D[k][j] = j < left ? dh[j] * w[j] : 0.0f;
          }
        }
        norm_grad(D, zh, r, p, team, lt, s_red, slot);
      }
      if (has_dz) {
#pragma unroll
        for (int k = 0; k < kNV; ++k) {
          float dz[8];
          widen8<T>(rdz[k], false, dz);
#pragma unroll
          for (int j = 0; j < 8; ++j) D[k][j] += dz[j];
        }
      }
      if (has_y) {
        float yh[kNV][8], dyh[kNV][8];
#pragma unroll
        for (int k = 0; k < kNV; ++k) widen8<T>(ry[k], y8, yh[k]);
        row_stats(yh, p, team, lt, s_red, slot, mean, r);
#pragma unroll
        for (int k = 0; k < kNV; ++k) {
          const int vec = k * team + lt, left = p.d - vec * 8;
          float w[8], b[8], s[8], u[8], du[8];
          param8(p.wp, g, vec, p.d, p.wide, 1.0f, w);
          param8(p.bp, g, vec, p.d, p.wide, 0.0f, b);
          param8(p.sc, g, vec, p.d, p.wide, 1.0f, s);
          if (has_u) widen8<T>(ru[k], u8, u);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const bool on = live && j < left;
            yh[k][j] = on ? (yh[k][j] - mean) * r : 0.0f;
            float a = 1.0f, da = 0.0f;
            if (has_u) a = gate_value<T>(p.gate, u[j], da);
            const float t = w[j] * yh[k][j] + b[j];
            const float dst = D[k][j] * s[j];
            const float dt = on ? dst * a : 0.0f;
            du[j] = dst * t * da;
            acc[0][k][j] += dt * yh[k][j];
            acc[1][k][j] += dt;
            acc[2][k][j] += on ? D[k][j] * t * a : 0.0f;
            dyh[k][j] = on ? dt * w[j] : 0.0f;
          }
          if (has_u && live) store8<T, AL>(p.du.data, p.du.ld, row, vec, p.d, du);
        }
        norm_grad(dyh, yh, r, p, team, lt, s_red, slot);
        if (live) {
#pragma unroll
          for (int k = 0; k < kNV; ++k) store8<T, AL>(p.dy.data, p.dy.ld, row, k * team + lt, p.d, dyh[k]);
        }
      }
      if (live) {
#pragma unroll
        for (int k = 0; k < kNV; ++k) store8<T, AL>(p.dx.data, p.dx.ld, row, k * team + lt, p.d, D[k]);
      }
    }
    // the chunk's sums: the teams' registers meet in shared memory, one parameter at a time, in the teams' order
#pragma unroll
    for (int q = 0; q < kSums; ++q) {
      if (q < 3 ? !has_y : !has_h) continue;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kNV; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int col = (k * team + lt) * 8 + j;
          if (col < p.d) s_sum[sub * p.d + col] = acc[q][k][j];
        }
      __syncthreads();
      float* out = p.part + ((size_t)c * kSums + q) * p.d;
      for (int col = threadIdx.x; col < p.d; col += blockDim.x) {
        float s = 0.0f;
        for (int m = 0; m < teams; ++m) s += s_sum[m * p.d + col];
        out[col] = s;
      }
    }
  }
}

// The sums of each group over its chunks: 32 columns by 8 slices of chunks per block, in fp64, joined in the slices'
// order.
__global__ void __launch_bounds__(256) k_norm_sums(const NormParams p) {
  extern __shared__ long long s_off[];
  __shared__ double s_part[8][33];
  int* s_cum = reinterpret_cast<int*>(s_off + p.groups + 1);
  load_offsets(p.offsets, p.groups, p.n, s_off, p.status);
  count_tiles(s_off, p.groups, p.chunk_rows, s_cum);
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane, q = blockIdx.y;
  float* const outs[kSums] = {p.dwp, p.dbp, p.dsc, p.dwq, p.dbq};
  float* out = nullptr;
#pragma unroll
  for (int i = 0; i < kSums; ++i)
    if (i == q) out = outs[i];
  if (out == nullptr) return;  // uniform over the block
  for (int g = blockIdx.z; g < p.groups; g += gridDim.z) {
    double s = 0.0;
    if (col < p.d) {
      for (int c = s_cum[g] + slice; c < s_cum[g + 1]; c += 8) s += (double)__ldg(&p.part[((size_t)c * kSums + q) * p.d + col]);
    }
    s_part[slice][lane] = s;
    __syncthreads();
    if (slice == 0 && col < p.d) {
      for (int k = 1; k < 8; ++k) s += s_part[k][lane];
      out[(size_t)g * p.d + col] = (float)s;
    }
    __syncthreads();
  }
}

// ---- host ---------------------------------------------------------------------------

int log_team_of(int d) {  // 16 columns per lane; at least the four lanes of an 8-bit block
  int l = 2;
  while ((16 << l) < d) ++l;
  return l;
}
int threads_of(int log_team) { return log_team > 8 ? 1 << log_team : kNormThreads; }

// Rows per chunk: two chunks per SM when the rows are many (each leaves kSums sums of d columns), at least four
// rows per team.
int chunk_rows_of(long long n, int d) {
  const int teams = threads_of(log_team_of(d)) >> log_team_of(d);
  const long long want = (n + 2LL * sm_count() - 1) / (2LL * sm_count());
  const long long least = 4LL * teams;
  return (int)std::max<long long>(least, (want + teams - 1) / teams * teams);
}

size_t norm_smem(int groups) { return (size_t)(groups + 1) * (8 + 4); }

int norm_params(const mt_gated_norm* c, NormParams& p) {
  if (c == nullptr) return MT_EINVAL;
  if (c->n < 0 || c->n > 0x7FFFFFFF || c->dim < 1 || c->dim > MT_MAX_BLOCK_DIM) return MT_EINVAL;
  if (c->groups < 1 || c->groups > MT_MAX_GROUPS || (c->offsets == nullptr && c->groups != 1)) return MT_EINVAL;
  if (c->dtype != MT_F32 && c->dtype != MT_BF16) return MT_EINVAL;
  if (c->kind != MT_NORM_RMS && c->kind != MT_NORM_LAYER) return MT_EINVAL;
  if (c->gate < MT_GATE_NONE || c->gate > MT_GATE_SILU) return MT_EINVAL;
  if (!(c->eps > 0.0f) || c->eps > 1e30f) return MT_EINVAL;
  if (!is_aligned(c->offsets, 8) || !is_aligned(c->status, 4)) return MT_EINVAL;
  const float* ps[] = {c->post_weight, c->post_bias, c->scale, c->pre_weight, c->pre_bias};
  p.wide = c->dim % 8 == 0;
  for (const float* f : ps) {
    if (!is_aligned(f, 4)) return MT_EINVAL;
    p.wide = p.wide && is_aligned(f, 16);
  }
  p.n = c->n;
  p.d = c->dim;
  p.groups = c->groups;
  p.kind = c->kind;
  p.gate = c->gate;
  p.eps = c->eps;
  p.offsets = reinterpret_cast<const long long*>(c->offsets);
  p.status = c->status;
  p.wp = c->post_weight;
  p.bp = c->post_bias;
  p.sc = c->scale;
  p.wq = c->pre_weight;
  p.bq = c->pre_bias;
  p.log_team = log_team_of(p.d);
  return MT_OK;
}

template <typename T, bool AL>
void norm_launch_fwd_as(const NormParams& p, int grid, int threads, size_t smem, cudaStream_t s) {
  if (threads > kNormThreads) k_norm_fwd<T, AL, 2 * kNormThreads><<<grid, threads, smem, s>>>(p);
  else k_norm_fwd<T, AL, kNormThreads><<<grid, threads, smem, s>>>(p);
}
void norm_launch_fwd(const NormParams& p, int dtype, bool wide, int grid, int threads, size_t smem, cudaStream_t s) {
  if (dtype == MT_F32) {
    if (wide) norm_launch_fwd_as<float, true>(p, grid, threads, smem, s);
    else norm_launch_fwd_as<float, false>(p, grid, threads, smem, s);
  } else {
    if (wide) norm_launch_fwd_as<__nv_bfloat16, true>(p, grid, threads, smem, s);
    else norm_launch_fwd_as<__nv_bfloat16, false>(p, grid, threads, smem, s);
  }
}

template <typename T, bool AL>
void norm_launch_bwd_as(const NormParams& p, int grid, int threads, size_t smem, cudaStream_t s) {
  if (threads > kNormThreads) k_norm_bwd<T, AL, 2 * kNormThreads><<<grid, threads, smem, s>>>(p);
  else k_norm_bwd<T, AL, kNormThreads><<<grid, threads, smem, s>>>(p);
}
void norm_launch_bwd(const NormParams& p, int dtype, bool wide, int grid, int threads, size_t smem, cudaStream_t s) {
  if (dtype == MT_F32) {
    if (wide) norm_launch_bwd_as<float, true>(p, grid, threads, smem, s);
    else norm_launch_bwd_as<float, false>(p, grid, threads, smem, s);
  } else {
    if (wide) norm_launch_bwd_as<__nv_bfloat16, true>(p, grid, threads, smem, s);
    else norm_launch_bwd_as<__nv_bfloat16, false>(p, grid, threads, smem, s);
  }
}

bool packed_rows(const Rows& r) { return r.codes != nullptr && r.exps != nullptr; }
bool half_packed(const Rows& r) { return (r.codes == nullptr) != (r.exps == nullptr); }
bool absent(const Rows& r) { return r.data == nullptr && r.codes == nullptr && r.exps == nullptr; }
Rows rows_of(const mt_rows* r) { return r != nullptr ? *r : Rows{nullptr, 0, nullptr, nullptr}; }

}  // namespace
}  // namespace mt

extern "C" {

int mt_gated_norm_forward(const mt_gated_norm* cfg, const mt_rows* x, const mt_rows* y, const mt_rows* gate,
                          const mt_rows* z, const mt_rows* h, mt_stream stream) {
  using namespace mt;
  NormParams p{};
  const int rc = norm_params(cfg, p);
  if (rc != MT_OK) return rc;
  p.x = rows_of(x);
  p.y = rows_of(y);
  p.u = rows_of(gate);
  p.z = rows_of(z);
  p.h = rows_of(h);
  if (p.n == 0) return MT_OK;
  const bool has_y = !absent(p.y), has_u = !absent(p.u);
  if (half_packed(p.y) || half_packed(p.u) || half_packed(p.z) || half_packed(p.h) || p.x.codes != nullptr) return MT_EINVAL;
  if (has_y != (p.wp != nullptr) || has_u != (p.gate != MT_GATE_NONE) || (has_u && !has_y)) return MT_EINVAL;
  if (!has_y && (p.bp != nullptr || p.sc != nullptr)) return MT_EINVAL;
  if (p.wq == nullptr && (p.bq != nullptr || !absent(p.h))) return MT_EINVAL;
  if (!rows_ok(p.x.data, p.x.ld, p.d, cfg->dtype)) return MT_EINVAL;
  if (has_y && !rows_ok(p.y.data, p.y.ld, p.d, cfg->dtype)) return MT_EINVAL;
  if (has_u && !rows_ok(p.u.data, p.u.ld, p.d, cfg->dtype)) return MT_EINVAL;
  if (has_y ? !rows_ok(p.z.data, p.z.ld, p.d, cfg->dtype) : p.z.data != nullptr) return MT_EINVAL;
  if (p.wq != nullptr && !rows_ok(p.h.data, p.h.ld, p.d, cfg->dtype)) return MT_EINVAL;
  bool wide = true;
  for (const Rows* r : {&p.x, &p.y, &p.u, &p.z, &p.h}) wide = wide && rows_wide(*r, p.d, cfg->dtype);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int threads = threads_of(p.log_team), teams = threads >> p.log_team;
  const int grid = grid_for((p.n + teams - 1) / teams * threads, threads, 2048 / threads);
  const size_t smem = norm_smem(p.groups);
  {
    MT_LAUNCH("k_norm_fwd", s);
    norm_launch_fwd(p, cfg->dtype, wide, grid, threads, smem, s);
  }
  return cudaGetLastError() == cudaSuccess ? MT_OK : MT_ECUDA;
}

size_t mt_gated_norm_workspace_bytes(int64_t n, int32_t dim, int32_t groups) {
  using namespace mt;
  if (n < 0 || n > 0x7FFFFFFF || dim < 1 || dim > MT_MAX_BLOCK_DIM || groups < 1 || groups > MT_MAX_GROUPS) return 0;
  const long long chunks = n / chunk_rows_of(n, dim) + groups;
  return align_up((size_t)chunks * kSums * dim * 4, 256);
}

int mt_gated_norm_backward(const mt_gated_norm* cfg, const mt_rows* dz, const mt_rows* dh, const mt_rows* y,
                           const mt_rows* gate, const mt_rows* z, const mt_rows* dx, const mt_rows* dy,
                           const mt_rows* dgate, float* dpost_weight, float* dpost_bias, float* dscale,
                           float* dpre_weight, float* dpre_bias, void* ws, size_t ws_bytes, mt_stream stream) {
  using namespace mt;
  NormParams p{};
  const int rc = norm_params(cfg, p);
  if (rc != MT_OK) return rc;
  p.dz = rows_of(dz);
  p.dh = rows_of(dh);
  p.y = rows_of(y);
  p.u = rows_of(gate);
  p.z = rows_of(z);
  p.dx = rows_of(dx);
  p.dy = rows_of(dy);
  p.du = rows_of(dgate);
  p.dwp = dpost_weight;
  p.dbp = dpost_bias;
  p.dsc = dscale;
  p.dwq = dpre_weight;
  p.dbq = dpre_bias;
  // an empty batch has no rows to point at: its parts are the parameters'
  const bool has_y = p.n > 0 ? !absent(p.y) : p.wp != nullptr;
  const bool has_u = p.n > 0 ? !absent(p.u) : p.gate != MT_GATE_NONE;
  const bool has_h = p.wq != nullptr;
  if (half_packed(p.y) || half_packed(p.u) || half_packed(p.z)) return MT_EINVAL;
  for (const Rows* r : {&p.dz, &p.dh, &p.dx, &p.dy, &p.du})
    if (r->codes != nullptr || r->exps != nullptr) return MT_EINVAL;
  if (has_y != (p.wp != nullptr) || has_u != (p.gate != MT_GATE_NONE) || (has_u && !has_y)) return MT_EINVAL;
  if (!has_y && (p.bp != nullptr || p.sc != nullptr)) return MT_EINVAL;
  if (!has_h && p.bq != nullptr) return MT_EINVAL;
  if (!has_y && !has_h) return MT_EINVAL;
  // a gradient for every parameter that is there, none for the others
  if ((p.wp != nullptr) != (p.dwp != nullptr) || (p.bp != nullptr) != (p.dbp != nullptr) ||
      (p.sc != nullptr) != (p.dsc != nullptr) || (p.wq != nullptr) != (p.dwq != nullptr) ||
      (p.bq != nullptr) != (p.dbq != nullptr))
    return MT_EINVAL;
  for (float* f : {p.dwp, p.dbp, p.dsc, p.dwq, p.dbq})
    if (!is_aligned(f, 4)) return MT_EINVAL;
  if (p.n > 0) {
    const int dt = cfg->dtype;
    if (!rows_ok(p.dx.data, p.dx.ld, p.d, dt)) return MT_EINVAL;
    if (p.dz.data != nullptr && !rows_ok(p.dz.data, p.dz.ld, p.d, dt)) return MT_EINVAL;
    if (has_h && !rows_ok(p.dh.data, p.dh.ld, p.d, dt)) return MT_EINVAL;
    if (has_h && !(packed_rows(p.z) && p.z.data == nullptr) && !rows_ok(p.z.data, p.z.ld, p.d, dt)) return MT_EINVAL;
    if (has_y && !(packed_rows(p.y) && p.y.data == nullptr) && !rows_ok(p.y.data, p.y.ld, p.d, dt)) return MT_EINVAL;
    if (has_u && !(packed_rows(p.u) && p.u.data == nullptr) && !rows_ok(p.u.data, p.u.ld, p.d, dt)) return MT_EINVAL;
    if (has_y && !rows_ok(p.dy.data, p.dy.ld, p.d, dt)) return MT_EINVAL;
    if (has_u && !rows_ok(p.du.data, p.du.ld, p.d, dt)) return MT_EINVAL;
  }
  if (ws == nullptr || !is_aligned(ws, 256) || ws_bytes < mt_gated_norm_workspace_bytes(p.n, p.d, p.groups))
    return MT_ENOSPACE;
  p.part = static_cast<float*>(ws);
  p.chunk_rows = chunk_rows_of(p.n, p.d);
  p.chunks = (int)(p.n / p.chunk_rows) + p.groups;
  bool wide = true;
  for (const Rows* r : {&p.dz, &p.dh, &p.y, &p.u, &p.z, &p.dx, &p.dy, &p.du})
    wide = wide && rows_wide(*r, p.d, cfg->dtype);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int threads = threads_of(p.log_team);
  const size_t smem = norm_smem(p.groups);
  if (p.n > 0) {
    MT_LAUNCH("k_norm_bwd", s);
    const int grid = p.chunks;
    norm_launch_bwd(p, cfg->dtype, wide, grid, threads, smem, s);
  }
  {
    MT_LAUNCH("k_norm_sums", s);
    const dim3 grid((p.d + 31) / 32, kSums, p.groups);
    k_norm_sums<<<grid, 256, smem, s>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? MT_OK : MT_ECUDA;
}

}  // extern "C"
