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
//  k_norm_fwd    each block takes an even run of the rows in the groups; teams
//                stride over it.
//  k_norm_bwd    the same split; the parameter gradients of a run stay in
//                registers and leave as one partial sum per block and group (no
//                atomics, so the sums have one order).  With S1 = sum D a yh and
//                S2 = sum D a, dwp = s S1, dbp = s S2 and ds = wp S1 + bp S2: two
//                sums for three gradients, and one when there is no bp.
//  k_norm_sums   the runs' partial sums of each group (8 to 12 us, latency).
//
// Measured, all parts, with the sums, of the copy bandwidth.  bf16, 490,011 x 512
// rms: forward 405 us (91%), with h in 8 bits as well 467 (87%), with all four
// checkpoints of y and u side by side 680 (77%); backward 639 (93%), from 8 bits 698
// (69%: issue at 57%, three rows widened and their exponent bytes loaded one by one
// between dependent steps).  200,003 x 1024 layer norm with biases: forward 555 (54%;
// 24 warps an SM, issue at 57% and shared memory's pipe at 60%, most stalls on
// loads: five rows of fp32 parameters come through L1 for every row, and each
// statistic waits for two reductions in a row) and backward 850 (57%; 12 warps an SM,
// bound by issue and by the latency between dependent steps); the same as rms without
// biases 379 (80%) and 594 (81%).  fp32, 245,003 x 512 rms: 461 (80%) and 666 (89%).
// Widths that are no multiple of 8 go an element at a time: 200,003 x 777 rms 1.1 ms
// forward (21%) and 2.0 backward (19%).
#include <algorithm>

#include "mt_block.cuh"

namespace mt {
namespace {

constexpr int kNV = 2;   // vectors of eight columns per lane
constexpr int kSums = 4; // partial sums: S1 = sum D a yh, S2 = sum D a, T1 = sum dh zh, T2 = sum dh

struct NormParams {
  long long n;
  int d, groups, kind, gate;
  float eps;
  const long long* offsets;
  int32_t* status;
  const float *wp, *bp, *sc, *wq, *bq;
  Rows x, y, u, z, h;            // forward
  Rows dz, dh, dx, dy, du;       // backward (with y, u, z)
  float* part;                   // [blocks + groups - 1][kSums][d]: block b's sums over group g at b + g
  float *dwp, *dbp, *dsc, *dwq, *dbq;
  int log_team;                  // log2 lanes per row
  int blocks;                    // blocks of k_norm_bwd
  int wide;                      // parameters reached with 16-byte loads
};

// Runs that m rows are cut into for `blocks` blocks: no more than there are rows, so that no run is empty (a group's partial
// sums are those of all runs from its first row's to its last row's).
__device__ __forceinline__ int runs_of(long long m, int blocks) { return m < blocks ? (m > 0 ? (int)m : 1) : blocks; }
// The rows of run b of B: an even share of the rows [off0, off0 + m) that lie in groups.
__device__ __forceinline__ long long run_start(long long off0, long long m, int b, int B) { return off0 + m * b / B; }
// The run that holds the row off0 + r (0 <= r < m).
__device__ __forceinline__ int run_of(long long r, long long m, int B) { return (int)(((r + 1) * B - 1) / m); }

// Sums a (and b, where TWO) over a team: shuffles inside a warp, shared memory across a team's warps.  A team of more than one
// warp owns a named barrier (a block has at most two such teams; the barriers' numbers are constants, as a number from
// a register would reserve all sixteen and leave an SM four blocks); `slot` alternates so that one barrier per call is
// enough.
template <bool TWO>
__device__ __forceinline__ void team_sum(float& a, float& b, int team_lanes, float2* s_red, int& slot) {
  const int in_warp = team_lanes < 32 ? team_lanes : 32;
  for (int o = in_warp >> 1; o > 0; o >>= 1) {
    a += __shfl_xor_sync(kFull, a, o);
    if (TWO) b += __shfl_xor_sync(kFull, b, o);
  }
  if (team_lanes <= 32) return;
  const int warp = threadIdx.x >> 5, warps = team_lanes >> 5, first = warp / warps * warps;
  float2* buf = s_red + slot * 16;
  if ((threadIdx.x & 31) == 0) buf[warp] = make_float2(a, b);
  if (first == 0) asm volatile("bar.sync 1, %0;" ::"r"(team_lanes) : "memory");
  else asm volatile("bar.sync 2, %0;" ::"r"(team_lanes) : "memory");
  a = b = 0.0f;
  for (int k = 0; k < warps; ++k) {
    const float2 v = buf[first + k];
    a += v.x;
    if (TWO) b += v.y;
  }
  slot ^= 1;
}

// How the rows lie: any strides and widths; 16-byte vectors; 16-byte vectors that fill their team exactly (no lane
// holds columns past d, so nothing is masked).
constexpr int kAny = 0, kVectors = 1, kWhole = 2;

// Which parts there are: asked at run time; all of them (y, a gate, a scale, the next norm, dz; every parameter on 16
// bytes), saved rows plain; the same with saved rows in 8 bits.  The last two leave out the checks.
constexpr int kParts = 0, kAllPlain = 1, kAllPacked = 2;

// Zeros where a vector's columns lie past d.
template <int MODE>
__device__ __forceinline__ void mask8(f32x2 (&v)[4], int left) {
  if constexpr (MODE == kVectors) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = left > 0 ? v[j] : 0ull;
  } else if constexpr (MODE == kAny) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = upk(v[j]);
      v[j] = pk(2 * j < left ? f.x : 0.0f, 2 * j + 1 < left ? f.y : 0.0f);
    }
  }
}

// Eight parameters of a group's row, `none` for an absent parameter and for a vector past d; zeros past d inside one.
// SURE: it is there, on 16 bytes, and the vector lies below d.
template <bool SURE>
__device__ __forceinline__ void param8(const float* p, int g, int vec, int d, int wide, float none, f32x2 (&f)[4]) {
  const int c0 = vec * 8;
  if (!SURE && (p == nullptr || c0 >= d)) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = both(none);
    return;
  }
  p += (uint32_t)(g * d + c0);  // groups * d <= 2^23
  if (SURE || wide) {
    const ulonglong2 a = __ldg(reinterpret_cast<const ulonglong2*>(p)), b = __ldg(reinterpret_cast<const ulonglong2*>(p) + 1);
    f[0] = a.x;
    f[1] = a.y;
    f[2] = b.x;
    f[3] = b.y;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      f[j] = pk(c0 + 2 * j < d ? __ldg(p + 2 * j) : 0.0f, c0 + 2 * j + 1 < d ? __ldg(p + 2 * j + 1) : 0.0f);
  }
}

// 1 / (1 + exp(-u)).  fp32 rows take the accurate exponential and division; for bf16 rows the hardware's own (2^-22 off)
// are far below the rounding of the result.
template <typename T>
__device__ __forceinline__ float sigmoid(float u) {
  if constexpr (sizeof(T) == 4) return 1.0f / (1.0f + expf(-u));
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(u * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}

// The gate's factors a = act(u) of eight columns and their derivatives (where DA).  The choice of the gate is made once
// for the eight, so that their chains overlap.
template <typename T, bool DA>
__device__ __forceinline__ void gate8(int gate, const f32x2 (&u)[4], f32x2 (&a)[4], f32x2 (&da)[4]) {
  const f32x2 one = both(1.0f);
  if (gate == MT_GATE_LINEAR) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[j] = u[j];
      if constexpr (DA) da[j] = one;
    }
    return;
  }
  f32x2 p[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = upk(u[j]);
    p[j] = pk(sigmoid<T>(f.x), sigmoid<T>(f.y));
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const f32x2 q = sub2(one, p[j]);
    a[j] = gate == MT_GATE_SIGMOID ? p[j] : mul2(u[j], p[j]);
    if constexpr (DA) da[j] = gate == MT_GATE_SIGMOID ? mul2(p[j], q) : fma2(a[j], q, p[j]);
  }
}

// A row v normalised is v * r + c: r its inverse deviation, c = -mean * r (0 for rms).  TWO rows v and w at once, or v
// alone.  Columns past d hold zeros and stay out of the deviation.
struct Stats {
  float r, c;
};
template <int MODE, bool TWO>
__device__ __forceinline__ void row_stats(const f32x2 (&v)[kNV][4], const f32x2 (&w)[kNV][4], const NormParams& p, int team,
                                          int lt, float2* s_red, int& slot, Stats& sv, Stats& sw) {
  f32x2 a = 0ull, b = 0ull;
  const float inv_d = 1.0f / (float)p.d;
  float x, y = 0.0f, mv = 0.0f, mw = 0.0f;
  if (p.kind == MT_NORM_LAYER) {
#pragma unroll
    for (int k = 0; k < kNV; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a = add2(a, v[k][j]);
        if (TWO) b = add2(b, w[k][j]);
      }
    x = pair_sum(a);
    if (TWO) y = pair_sum(b);
    team_sum<TWO>(x, y, team, s_red, slot);
    mv = x * inv_d;
    mw = y * inv_d;
    a = b = 0ull;
    const f32x2 nv = both(-mv), nw = both(-mw);
#pragma unroll
    for (int k = 0; k < kNV; ++k) {
      const int left = p.d - (k * team + lt) * 8;
      f32x2 c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] = add2(v[k][j], nv);
      mask8<MODE>(c, left);
#pragma unroll
      for (int j = 0; j < 4; ++j) a = fma2(c[j], c[j], a);
      if (TWO) {
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = add2(w[k][j], nw);
        mask8<MODE>(c, left);
#pragma unroll
        for (int j = 0; j < 4; ++j) b = fma2(c[j], c[j], b);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < kNV; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a = fma2(v[k][j], v[k][j], a);
        if (TWO) b = fma2(w[k][j], w[k][j], b);
      }
  }
  x = pair_sum(a);
  if (TWO) y = pair_sum(b);
  team_sum<TWO>(x, y, team, s_red, slot);
  sv.r = rsqrtf(x * inv_d + p.eps);
  sv.c = -mv * sv.r;
  if (TWO) {
    sw.r = rsqrtf(y * inv_d + p.eps);
    sw.c = -mw * sw.r;
  }
}

// ---- rows on their way -------------------------------------------------------------
//
// The next rows of a team are copied to shared memory while it works on the
// present ones.  A lane copies exactly what it will read, so waiting for its
// own copies is all the synchronisation there is, and the rows in flight cost no
// registers.  Rows that cannot be reached with 16-byte accesses, and the
// widest rows in fp32 (whose stages would not fit), are loaded when they are used.

template <typename T, int MODE, int THREADS>
constexpr bool kStaged = MODE != kAny && (THREADS == 128 || sizeof(T) == 2);
constexpr uint32_t kNoExp = 0xFFFFFFFFu;  // plain rows have no exponent byte
template <typename T>
constexpr int kVecBytes = 8 * (int)sizeof(T);

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(on ? 8 : 0) : "memory");
}
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// NROWS row tensors, two stages; the lane's vector k of tensor i in stage s.
template <typename T, int THREADS, int NROWS>
struct Stages {
  static constexpr int kBytes = 2 * NROWS * kNV * THREADS * kVecBytes<T>;
  uint32_t base;
  __device__ __forceinline__ uint32_t at(int s, int i, int k) const {
    return base + (uint32_t)((((s * NROWS + i) * kNV + k) * THREADS + threadIdx.x) * kVecBytes<T>);
  }
};

// Starts the copy of eight columns (zeros where they lie past d or the row is not there); e: a packed block's exponent
// byte, which comes by an ordinary load.
template <typename T, bool SURE>
__device__ __forceinline__ void fetch8(uint32_t dst, const Rows& r, int row, int vec, int d, bool live, bool packed,
                                       uint32_t& e) {
  const int c0 = vec * 8;
  const bool on = live && (SURE || c0 < d);
  if (packed) {
    const int nb = (d + kPackBlock - 1) / kPackBlock;
    copy8(dst, r.codes + row_offset(row, d) + (SURE || on ? c0 : 0), on);
    e = on ? (uint32_t)__ldg(r.exps + row_offset(row, nb) + c0 / kPackBlock) : 127u;
  } else {
    const T* p = static_cast<const T*>(r.data) + row_offset(row, r.ld) + (SURE || on ? c0 : 0);
    copy16(dst, p, on);
    if constexpr (sizeof(T) == 4) copy16(dst + 16, p + 4, on);
  }
}
template <typename T>
__device__ __forceinline__ Raw8<T> staged8(uint32_t at, uint32_t e) {
  Raw8<T> v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.a.x), "=r"(v.a.y), "=r"(v.a.z), "=r"(v.a.w) : "r"(at));
  if constexpr (sizeof(T) == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.b.x), "=r"(v.b.y), "=r"(v.b.z), "=r"(v.b.w) : "r"(at + 16));
  if (e != kNoExp) v.a.z = e;
  return v;
}

// Blocks of 128 threads that share an SM's registers and stages (wider rows: one block of 512).
constexpr int fwd_blocks_per_sm(int elem) { return elem == 4 ? 4 : 6; }
constexpr int bwd_blocks_per_sm(int elem, bool bias) { return elem == 4 ? 2 : bias ? 3 : 4; }

template <typename T, int MODE, int THREADS, int FORM>
__global__ void __launch_bounds__(THREADS, THREADS == 128 ? fwd_blocks_per_sm(sizeof(T)) : 1)
k_norm_fwd(const NormParams p) {
  constexpr bool AL = MODE != kAny, STAGED = kStaged<T, MODE, THREADS>;
  using St = Stages<T, THREADS, 3>;
  extern __shared__ __align__(16) uint8_t s_raw[];  // the stages, then the offsets
  __shared__ float2 s_red[32];
  const St st{(uint32_t)__cvta_generic_to_shared(s_raw)};
  long long* s_off = reinterpret_cast<long long*>(s_raw + (STAGED ? St::kBytes : 0));
  load_offsets(p.offsets, p.groups, p.n, s_off, p.status);
  const int team = 1 << p.log_team;
  const int lt = threadIdx.x & (team - 1);
  const int sub = threadIdx.x >> p.log_team;
  const int teams = THREADS >> p.log_team;  // teams per block
  constexpr bool ALL = FORM != kParts, SURE = ALL && MODE == kWhole;
  const bool has_y = ALL || p.y.data != nullptr, has_u = ALL || p.u.data != nullptr, has_h = ALL || p.wq != nullptr;
  const long long off0 = s_off[0], m = s_off[p.groups] - off0;
  int slot = 0;

  // rows in no group: zeros, and their checkpoints zeros
  for (long long q0 = (long long)blockIdx.x * teams; q0 < p.n - m; q0 += (long long)gridDim.x * teams) {
    const long long q = q0 + sub, row = q < off0 ? q : q + m;
    const bool in = q < p.n - m;
    const Raw8<T> zero{};
#pragma unroll
    for (int k = 0; k < kNV; ++k) {
      const int vec = k * team + lt;
      if (in && p.z.data != nullptr) put8<T, AL>(p.z, row, vec, p.d, zero);
      if (in && has_h) put8<T, AL>(p.h, row, vec, p.d, zero);
      if (p.y.codes != nullptr) put_packed8<T, AL>(p.y, row, vec, p.d, zero, in);
      if (p.u.codes != nullptr) put_packed8<T, AL>(p.u, row, vec, p.d, zero, in);
      if (p.z.codes != nullptr) put_packed8<T, AL>(p.z, row, vec, p.d, zero, in);
      if (p.h.codes != nullptr) put_packed8<T, AL>(p.h, row, vec, p.d, zero, in);
    }
  }

  const long long end = run_start(off0, m, blockIdx.x + 1, gridDim.x);
  long long first = run_start(off0, m, blockIdx.x, gridDim.x);
  for (int g = first < end ? row_group(s_off, p.groups, first) : 0; first < end; ++g) {
    const int last = (int)min(end, s_off[g + 1]);
    // a row's vectors start on their way, or are loaded where they are used
    auto fetch = [&](int base, int s) {
      const bool live = base + sub < last;
      const int row = live ? base + sub : base;
      uint32_t none;
#pragma unroll
      for (int k = 0; k < kNV; ++k) {
        const int vec = k * team + lt;
        if (has_y) fetch8<T, SURE>(st.at(s, 0, k), p.y, row, vec, p.d, live, false, none);
        if (has_u) fetch8<T, SURE>(st.at(s, 1, k), p.u, row, vec, p.d, live, false, none);
        fetch8<T, SURE>(st.at(s, 2, k), p.x, row, vec, p.d, live, false, none);
      }
    };
    int cur = 0;
    if constexpr (STAGED) {
      if (first < last) fetch((int)first, 0);
      copies_close();
    }
    // every team of the block runs the same number of rounds, so the shuffles and barriers meet
    for (int base = (int)first; base < last; base += teams, cur ^= 1) {
      const bool live = base + sub < last;
      const int row = live ? base + sub : base, dd = live ? p.d : 0;  // a team without a row computes on zeros
      if constexpr (STAGED) {
        if (base + teams < last) fetch(base + teams, cur ^ 1);
        copies_close();
        copies_wait<1>();
      }
      auto get = [&](int i, const Rows& r, int k) {
        if constexpr (STAGED) return staged8<T>(st.at(cur, i, k), kNoExp);
        else return load8<T, AL>(r, row, k * team + lt, dd);
      };
      f32x2 z[kNV][4];
      if (has_y) {
        f32x2 y[kNV][4];
#pragma unroll
        for (int k = 0; k < kNV; ++k) {
          const Raw8<T> raw = get(0, p.y, k);
          widen8<T>(raw, false, y[k]);
          if (p.y.codes != nullptr) put_packed8<T, AL>(p.y, row, k * team + lt, p.d, raw, live);
        }
        Stats sy;
        row_stats<MODE, false>(y, y, p, team, lt, s_red, slot, sy, sy);
        const f32x2 r2 = both(sy.r), c2 = both(sy.c);
#pragma unroll
        for (int k = 0; k < kNV; ++k) {
          const int vec = k * team + lt;
          f32x2 f[4];
          param8<SURE>(p.wp, g, vec, p.d, p.wide, 1.0f, f);
#pragma unroll
          for (int j = 0; j < 4; ++j) y[k][j] = mul2(f[j], fma2(y[k][j], r2, c2));
          if (MODE != kWhole) mask8<MODE>(y[k], p.d - vec * 8);
          if (p.bp != nullptr) {
            param8<false>(p.bp, g, vec, p.d, p.wide, 0.0f, f);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[k][j] = add2(y[k][j], f[j]);
          }
          if (ALL || p.sc != nullptr) {
            param8<SURE>(p.sc, g, vec, p.d, p.wide, 1.0f, f);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[k][j] = mul2(y[k][j], f[j]);
          }
          widen8<T>(get(2, p.x, k), false, z[k]);
          if (has_u) {
            f32x2 u[4], da[4];
            const Raw8<T> raw = get(1, p.u, k);
            widen8<T>(raw, false, u);
            if (p.u.codes != nullptr) put_packed8<T, AL>(p.u, row, vec, p.d, raw, live);
            gate8<T, false>(p.gate, u, f, da);
#pragma unroll
            for (int j = 0; j < 4; ++j) z[k][j] = fma2(y[k][j], f[j], z[k][j]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) z[k][j] = add2(z[k][j], y[k][j]);
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < kNV; ++k) widen8<T>(get(2, p.x, k), false, z[k]);
      }
      if (ALL || p.z.data != nullptr || p.z.codes != nullptr) {
#pragma unroll
        for (int k = 0; k < kNV; ++k) {
          const Raw8<T> raw = narrow8<T>(z[k]);
          if ((ALL || p.z.data != nullptr) && live) put8<T, AL>(p.z, row, k * team + lt, p.d, raw);
          if (p.z.codes != nullptr) put_packed8<T, AL>(p.z, row, k * team + lt, p.d, raw, live);
        }
      }
      if (has_h) {
        Stats sz;
        row_stats<MODE, false>(z, z, p, team, lt, s_red, slot, sz, sz);
        const f32x2 r2 = both(sz.r), c2 = both(sz.c);
#pragma unroll
        for (int k = 0; k < kNV; ++k) {
          const int vec = k * team + lt;
          f32x2 f[4];
          param8<SURE>(p.wq, g, vec, p.d, p.wide, 1.0f, f);
#pragma unroll
          for (int j = 0; j < 4; ++j) z[k][j] = mul2(f[j], fma2(z[k][j], r2, c2));
          if (MODE != kWhole) mask8<MODE>(z[k], p.d - vec * 8);
          if (p.bq != nullptr) {
            param8<false>(p.bq, g, vec, p.d, p.wide, 0.0f, f);
#pragma unroll
            for (int j = 0; j < 4; ++j) z[k][j] = add2(z[k][j], f[j]);
          }
          const Raw8<T> raw = narrow8<T>(z[k]);
          if (live) put8<T, AL>(p.h, row, vec, p.d, raw);
          if (p.h.codes != nullptr) put_packed8<T, AL>(p.h, row, vec, p.d, raw, live);
        }
      }
    }
    first = last;
  }
}

// dv = r * (dvh - [mean dvh] - vh * mean(dvh * vh)), the gradient through a norm, in place of dvh.
template <int MODE>
__device__ __forceinline__ void norm_grad(f32x2 (&dvh)[kNV][4], const f32x2 (&vh)[kNV][4], float r, const NormParams& p,
                                          int team, int lt, float2* s_red, int& slot) {
  const bool layer = p.kind == MT_NORM_LAYER;
  f32x2 a = 0ull, b = 0ull;
#pragma unroll
  for (int k = 0; k < kNV; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) a = fma2(dvh[k][j], vh[k][j], a);
  if (layer) {
#pragma unroll
    for (int k = 0; k < kNV; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) b = add2(b, dvh[k][j]);
  }
  float x = pair_sum(a), y = pair_sum(b);
  if (layer) team_sum<true>(x, y, team, s_red, slot);
  else team_sum<false>(x, y, team, s_red, slot);
  const float inv_d = 1.0f / (float)p.d;
  const f32x2 r2 = both(r), ma = both(-r * x * inv_d), mb = both(-r * y * inv_d);
#pragma unroll
  for (int k = 0; k < kNV; ++k) {
#pragma unroll
    for (int j = 0; j < 4; ++j) dvh[k][j] = fma2(vh[k][j], ma, fma2(dvh[k][j], r2, mb));
    if (MODE != kWhole && layer) mask8<MODE>(dvh[k], p.d - (k * team + lt) * 8);
  }
}

// BIAS: the norms have biases (their sums S2 and T2 are kept too).
template <typename T, int MODE, int THREADS, bool BIAS, int FORM>
__global__ void __launch_bounds__(THREADS, THREADS == 128 ? bwd_blocks_per_sm(sizeof(T), BIAS) : 1)
k_norm_bwd(const NormParams p) {
  constexpr bool AL = MODE != kAny, STAGED = kStaged<T, MODE, THREADS>;
  constexpr int kAcc = BIAS ? 4 : 2;       // S1, T1, S2, T2
  using St = Stages<T, THREADS, 5>;
  extern __shared__ __align__(16) uint8_t s_raw[];  // the stages (later the sums of the block's teams), the offsets
  __shared__ float2 s_red[32];
  const St st{(uint32_t)__cvta_generic_to_shared(s_raw)};
  float* s_sum = reinterpret_cast<float*>(s_raw);   // teams * d <= 16 * THREADS floats
  static_assert(St::kBytes >= 16 * THREADS * 4, "the sums fit the stages");
  long long* s_off = reinterpret_cast<long long*>(s_raw + (STAGED ? St::kBytes : 16 * THREADS * 4));
  load_offsets(p.offsets, p.groups, p.n, s_off, p.status);
  const int team = 1 << p.log_team;
  const int lt = threadIdx.x & (team - 1);
  const int sub = threadIdx.x >> p.log_team;
  const int teams = THREADS >> p.log_team;
  constexpr bool ALL = FORM != kParts, SURE = ALL && MODE == kWhole, P8 = FORM == kAllPacked;
  const bool has_y = ALL || p.y.data != nullptr || p.y.codes != nullptr;
  const bool has_u = ALL || p.u.data != nullptr || p.u.codes != nullptr;
  const bool has_h = ALL || p.wq != nullptr, has_dz = ALL || p.dz.data != nullptr;
  const bool y8 = ALL ? P8 : p.y.data == nullptr, u8 = ALL ? P8 : p.u.data == nullptr, z8 = ALL ? P8 : p.z.data == nullptr;
  const long long off0 = s_off[0], m = s_off[p.groups] - off0;
  int slot = 0;

  // rows in no group: their gradients are zero
  for (long long q = (long long)blockIdx.x * teams + sub; q < p.n - m; q += (long long)gridDim.x * teams) {
    const long long row = q < off0 ? q : q + m;
    const Raw8<T> zero{};
#pragma unroll
    for (int k = 0; k < kNV; ++k) {
      const int vec = k * team + lt;
      put8<T, AL>(p.dx, row, vec, p.d, zero);
      if (has_y) put8<T, AL>(p.dy, row, vec, p.d, zero);
      if (has_u) put8<T, AL>(p.du, row, vec, p.d, zero);
    }
  }

  const int runs = runs_of(m, gridDim.x), run = min((int)blockIdx.x, runs);  // blocks past the runs: an empty one
  const long long end = run_start(off0, m, min(run + 1, runs), runs);
  long long first = run_start(off0, m, run, runs);
  for (int g = first < end ? row_group(s_off, p.groups, first) : 0; first < end; ++g) {
    const int last = (int)min(end, s_off[g + 1]);
    if (last <= first) continue;  // an empty group
    f32x2 acc[kAcc][kNV][4] = {};
    uint32_t next_e[3][kNV];  // exponent bytes of the rows on their way: z, y, u
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
      for (int k = 0; k < kNV; ++k) next_e[i][k] = kNoExp;
    auto fetch = [&](int base, int s) {
      const bool live = base + sub < last;
      const int row = live ? base + sub : base;
#pragma unroll
      for (int k = 0; k < kNV; ++k) {
        const int vec = k * team + lt;
        uint32_t none;
        if (has_h) fetch8<T, SURE>(st.at(s, 0, k), p.z, row, vec, p.d, live, z8, next_e[0][k]);
        if (has_y) fetch8<T, SURE>(st.at(s, 1, k), p.y, row, vec, p.d, live, y8, next_e[1][k]);
        if (has_h) fetch8<T, SURE>(st.at(s, 2, k), p.dh, row, vec, p.d, live, false, none);
        if (has_dz) fetch8<T, SURE>(st.at(s, 3, k), p.dz, row, vec, p.d, live, false, none);
        if (has_u) fetch8<T, SURE>(st.at(s, 4, k), p.u, row, vec, p.d, live, u8, next_e[2][k]);
      }
    };
    int cur = 0;
    if constexpr (STAGED) {
      fetch((int)first, 0);
      copies_close();
    }
    for (int base = (int)first; base < last; base += teams, cur ^= 1) {
      const bool live = base + sub < last;
      const int row = live ? base + sub : base, dd = live ? p.d : 0;  // a team without a row computes on zeros
      uint32_t e[3][kNV];
      if constexpr (STAGED) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
#pragma unroll
          for (int k = 0; k < kNV; ++k) e[i][k] = next_e[i][k];
        if (base + teams < last) fetch(base + teams, cur ^ 1);
        copies_close();
        copies_wait<1>();
      }
      // a row's vector, from its stage or from where it lies
      auto get = [&](int i, const Rows& r, int k, uint32_t ex) {
        if constexpr (STAGED) return staged8<T>(st.at(cur, i, k), ex);
        else return load8<T, AL>(r, row, k * team + lt, dd);
      };
      Stats sy, sz;
      f32x2 yh[kNV][4] = {}, D[kNV][4] = {};
      {
        f32x2 zh[kNV][4] = {};
#pragma unroll
        for (int k = 0; k < kNV; ++k) {
          if (has_h) widen8<T>(get(0, p.z, k, e[0][k]), z8, zh[k]);
          if (has_y) widen8<T>(get(1, p.y, k, e[1][k]), y8, yh[k]);
        }
        row_stats<MODE, true>(yh, zh, p, team, lt, s_red, slot, sy, sz);
        if (has_h) {  // through the next block's norm
          const f32x2 r2 = both(sz.r), c2 = both(sz.c);
#pragma unroll
          for (int k = 0; k < kNV; ++k) {
            const int vec = k * team + lt;
            f32x2 dh[4], w[4];
            widen8<T>(get(2, p.dh, k, kNoExp), false, dh);
            param8<SURE>(p.wq, g, vec, p.d, p.wide, 1.0f, w);
#pragma unroll
            for (int j = 0; j < 4; ++j) zh[k][j] = fma2(zh[k][j], r2, c2);
            mask8<MODE>(zh[k], p.d - vec * 8);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              acc[1][k][j] = fma2(dh[j], zh[k][j], acc[1][k][j]);
              if constexpr (BIAS) acc[3][k][j] = add2(acc[3][k][j], dh[j]);
              D[k][j] = mul2(dh[j], w[j]);  // dh is zero past d
            }
          }
          norm_grad<MODE>(D, zh, sz.r, p, team, lt, s_red, slot);
        }
      }
      if (has_dz) {
#pragma unroll
        for (int k = 0; k < kNV; ++k) {
          f32x2 dz[4];
          widen8<T>(get(3, p.dz, k, kNoExp), false, dz);
#pragma unroll
          for (int j = 0; j < 4; ++j) D[k][j] = add2(D[k][j], dz[j]);
        }
      }
      if (live) {
#pragma unroll
        for (int k = 0; k < kNV; ++k) put8<T, AL>(p.dx, row, k * team + lt, p.d, narrow8<T>(D[k]));
      }
      if (has_y) {
        const f32x2 r2 = both(sy.r), c2 = both(sy.c);
#pragma unroll
        for (int k = 0; k < kNV; ++k) {
          const int vec = k * team + lt;
          f32x2 w[4], s[4];
          param8<SURE>(p.wp, g, vec, p.d, p.wide, 1.0f, w);
          param8<SURE>(p.sc, g, vec, p.d, p.wide, 1.0f, s);
#pragma unroll
          for (int j = 0; j < 4; ++j) yh[k][j] = fma2(yh[k][j], r2, c2);
          mask8<MODE>(yh[k], p.d - vec * 8);
          if (has_u) {
            f32x2 u[4], a[4], da[4];
            widen8<T>(get(4, p.u, k, e[2][k]), u8, u);
            gate8<T, true>(p.gate, u, a, da);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              u[j] = mul2(w[j], yh[k][j]);
              da[j] = mul2(da[j], mul2(D[k][j], s[j]));
              D[k][j] = mul2(D[k][j], a[j]);
            }
            if constexpr (BIAS) {
              if (p.bp != nullptr) {
                param8<false>(p.bp, g, vec, p.d, p.wide, 0.0f, a);
#pragma unroll
                for (int j = 0; j < 4; ++j) u[j] = add2(u[j], a[j]);
              }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) da[j] = mul2(da[j], u[j]);
            if (live) put8<T, AL>(p.du, row, vec, p.d, narrow8<T>(da));
          }
          // D now holds D a
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[0][k][j] = fma2(D[k][j], yh[k][j], acc[0][k][j]);
            if constexpr (BIAS) acc[2][k][j] = add2(acc[2][k][j], D[k][j]);
            D[k][j] = mul2(mul2(D[k][j], s[j]), w[j]);
          }
        }
        norm_grad<MODE>(D, yh, sy.r, p, team, lt, s_red, slot);
        if (live) {
#pragma unroll
          for (int k = 0; k < kNV; ++k) put8<T, AL>(p.dy, row, k * team + lt, p.d, narrow8<T>(D[k]));
        }
      }
    }
    if constexpr (STAGED) copies_wait<0>();
    // the run's sums: the teams' registers meet in shared memory, one sum at a time, in the teams' order
#pragma unroll
    for (int q = 0; q < kAcc; ++q) {
      if (q % 2 == 0 ? !has_y : !has_h) continue;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kNV; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int col = (k * team + lt) * 8 + 2 * j;
          const float2 f = upk(acc[q][k][j]);
          if (col < p.d) s_sum[sub * p.d + col] = f.x;
          if (col + 1 < p.d) s_sum[sub * p.d + col + 1] = f.y;
        }
      __syncthreads();
      float* out = p.part + ((size_t)(blockIdx.x + g) * kSums + (q == 0 ? 0 : q == 1 ? 2 : q == 2 ? 1 : 3)) * p.d;
      for (int col = threadIdx.x; col < p.d; col += THREADS) {
        float s = 0.0f;
        for (int t = 0; t < teams; ++t) s += s_sum[t * p.d + col];
        out[col] = s;
      }
    }
    __syncthreads();  // the next group's rows may come
    first = last;
  }
}

// The parameter gradients of each group from its runs' partial sums (a few hundred, each already a sum of many rows):
// 32 columns by 16 slices of runs per block, the slices joined in their order.
constexpr int kSlices = 16;
__global__ void __launch_bounds__(32 * kSlices) k_norm_sums(const NormParams p) {
  extern __shared__ long long s_off[];
  __shared__ float2 s_part[2][kSlices][33];
  int buffer = 0;
  load_offsets(p.offsets, p.groups, p.n, s_off, p.status);
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  const bool post = blockIdx.y == 0;  // the block's two sums: S1, S2 or T1, T2
  if (post ? p.dwp == nullptr : p.dwq == nullptr) return;
  const bool second = post ? p.bp != nullptr : p.bq != nullptr;
  const long long off0 = s_off[0], m = s_off[p.groups] - off0;
  const int runs = runs_of(m, p.blocks);
  // the slices take turns at a group's last step, and two buffers, so that nobody waits for it
  for (int g = blockIdx.z, turn = 0; g < p.groups; g += gridDim.z, turn = turn + 1 == kSlices ? 0 : turn + 1) {
    float a = 0.0f, b = 0.0f;
    if (s_off[g] < s_off[g + 1]) {
      if (col < p.d) {
        const int b0 = run_of(s_off[g] - off0, m, runs), b1 = run_of(s_off[g + 1] - 1 - off0, m, runs);
        const float* base = p.part + (size_t)(post ? 0 : 2) * p.d + col;
#pragma unroll 8
        for (int k = b0 + slice; k <= b1; k += kSlices) {
          const float* at = base + (size_t)(k + g) * kSums * p.d;
          a += __ldg(at);
          if (second) b += __ldg(at + p.d);
        }
      }
      auto& part = s_part[buffer];
      buffer ^= 1;
      part[slice][lane] = make_float2(a, b);
      __syncthreads();
      if (slice != turn) continue;
      a = part[0][lane].x;
      b = part[0][lane].y;
      for (int k = 1; k < kSlices; ++k) {
        const float2 v = part[k][lane];
        a += v.x;
        b += v.y;
      }
    }
    if (slice != turn || col >= p.d) continue;
    const size_t at = (size_t)g * p.d + col;
    if (s_off[g] == s_off[g + 1]) {  // no rows: zeros, whatever the parameters are
      for (float* f : {post ? p.dwp : p.dwq, post ? p.dbp : p.dbq, post ? p.dsc : nullptr})
        if (f != nullptr) f[at] = 0.0f;
    } else if (post) {
      const float s = p.sc != nullptr ? p.sc[at] : 1.0f;
      p.dwp[at] = s * a;
      if (p.dbp != nullptr) p.dbp[at] = s * b;
      if (p.dsc != nullptr) p.dsc[at] = p.wp[at] * a + (p.bp != nullptr ? p.bp[at] * b : 0.0f);
    } else {
      p.dwq[at] = a;
      if (p.dbq != nullptr) p.dbq[at] = b;
    }
  }
}

// ---- host ---------------------------------------------------------------------------

int log_team_of(int d) {  // 16 columns per lane; at least the four lanes of an 8-bit block
  int l = 2;
  while ((16 << l) < d) ++l;
  return l;
}
int threads_of(int log_team) { return log_team > 7 ? 512 : 128; }

// Blocks of a backward over n rows: what the SMs hold at once, and at least two rows per team.
int bwd_blocks(long long n, int d, int elem, bool bias) {
  const int lt = log_team_of(d), threads = threads_of(lt), teams = threads >> lt;
  const long long most = (long long)sm_count() * (threads == 128 ? bwd_blocks_per_sm(elem, bias) : 1);
  return (int)std::max<long long>(1, std::min<long long>(most, (n + 2 * teams - 1) / (2 * teams)));
}

int norm_params(const mt_gated_norm* c, NormParams& p) {
  if (c == nullptr) return MT_EINVAL;
  if (c->n < 0 || c->n > MT_MAX_BLOCK_ROWS || c->dim < 1 || c->dim > MT_MAX_BLOCK_DIM) return MT_EINVAL;
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

bool absent(const Rows& r) { return r.data == nullptr && r.codes == nullptr && r.exps == nullptr; }

size_t offsets_smem(int groups) { return (size_t)(groups + 1) * 8; }

template <typename T, int MODE, int THREADS, int FORM>
cudaError_t norm_fwd_as(const NormParams& p, cudaStream_t s) {
  const int teams = THREADS >> p.log_team;
  const int grid = grid_for((p.n + teams - 1) / teams * THREADS, THREADS, THREADS == 128 ? fwd_blocks_per_sm(sizeof(T)) : 1);
  constexpr size_t stages = kStaged<T, MODE, THREADS> ? Stages<T, THREADS, 3>::kBytes : 0;
  static SmemLimit limit;
  const cudaError_t e = limit.allow(k_norm_fwd<T, MODE, THREADS, FORM>, stages + offsets_smem(MT_MAX_GROUPS));
  if (e != cudaSuccess) return e;
  k_norm_fwd<T, MODE, THREADS, FORM><<<grid, THREADS, stages + offsets_smem(p.groups), s>>>(p);
  return cudaGetLastError();
}
template <typename T, int MODE, int THREADS, bool BIAS, int FORM>
cudaError_t norm_bwd_as(const NormParams& p, cudaStream_t s) {
  constexpr size_t stages = kStaged<T, MODE, THREADS> ? Stages<T, THREADS, 5>::kBytes : 16 * THREADS * 4;
  static SmemLimit limit;
  const cudaError_t e = limit.allow(k_norm_bwd<T, MODE, THREADS, BIAS, FORM>, stages + offsets_smem(MT_MAX_GROUPS));
  if (e != cudaSuccess) return e;
  k_norm_bwd<T, MODE, THREADS, BIAS, FORM><<<p.blocks, THREADS, stages + offsets_smem(p.groups), s>>>(p);
  return cudaGetLastError();
}
template <typename T, int MODE>
cudaError_t norm_fwd(const NormParams& p, cudaStream_t s) {
  if (p.log_team > 7) return norm_fwd_as<T, MODE, 512, kParts>(p, s);
  if constexpr (MODE == kWhole) {
    if (p.y.data != nullptr && p.u.data != nullptr && p.wq != nullptr && p.sc != nullptr && p.wide)
      return norm_fwd_as<T, MODE, 128, kAllPlain>(p, s);
  }
  return norm_fwd_as<T, MODE, 128, kParts>(p, s);
}
template <typename T, int MODE, bool BIAS>
cudaError_t norm_bwd(const NormParams& p, cudaStream_t s) {
  if (p.log_team > 7) return norm_bwd_as<T, MODE, 512, BIAS, kParts>(p, s);
  if constexpr (MODE == kWhole) {
    if (!absent(p.y) && !absent(p.u) && p.wq != nullptr && p.sc != nullptr && p.dz.data != nullptr && p.wide) {
      if (p.y.data != nullptr && p.u.data != nullptr && p.z.data != nullptr) return norm_bwd_as<T, MODE, 128, BIAS, kAllPlain>(p, s);
      if (p.y.data == nullptr && p.u.data == nullptr && p.z.data == nullptr) return norm_bwd_as<T, MODE, 128, BIAS, kAllPacked>(p, s);
    }
  }
  return norm_bwd_as<T, MODE, 128, BIAS, kParts>(p, s);
}
template <typename T, int MODE>
cudaError_t norm_bwd(const NormParams& p, cudaStream_t s) {
  return p.bp != nullptr || p.bq != nullptr ? norm_bwd<T, MODE, true>(p, s) : norm_bwd<T, MODE, false>(p, s);
}

int mode_of(const NormParams& p, bool wide) { return !wide ? kAny : (16 << p.log_team) == p.d ? kWhole : kVectors; }

bool packed_rows(const Rows& r) { return r.codes != nullptr && r.exps != nullptr; }
bool half_packed(const Rows& r) { return (r.codes == nullptr) != (r.exps == nullptr); }
Rows rows_of(const mt_rows* r) { return r != nullptr ? *r : Rows{nullptr, 0, nullptr, nullptr}; }

// What both directions read beside rows.
void common_inputs(Regions& all, const NormParams& p) {
  const size_t bytes = (size_t)p.groups * p.d * 4;
  for (const float* f : {p.wp, p.bp, p.sc, p.wq, p.bq}) all.in(whole_region(f, bytes));
  all.in(whole_region(p.offsets, (size_t)(p.groups + 1) * 8));
}

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
  Regions all;
  common_inputs(all, p);
  for (const Rows* r : {&p.x, &p.y, &p.u}) {
    all.in(Regions::plain(*r, p.n, p.d, cfg->dtype));
    all.out_packed(*r, p.n, p.d);
  }
  for (const Rows* r : {&p.z, &p.h}) all.out(*r, p.n, p.d, cfg->dtype);
  if (all.clash()) return MT_EINVAL;
  bool wide = true;
  for (const Rows* r : {&p.x, &p.y, &p.u, &p.z, &p.h}) wide = wide && rows_wide(*r, p.d, cfg->dtype);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  {
    MT_LAUNCH("k_norm_fwd", s);
    const int mode = mode_of(p, wide);
    if (cfg->dtype == MT_F32)
      e = mode == kWhole ? norm_fwd<float, kWhole>(p, s) : mode == kVectors ? norm_fwd<float, kVectors>(p, s) : norm_fwd<float, kAny>(p, s);
    else
      e = mode == kWhole     ? norm_fwd<__nv_bfloat16, kWhole>(p, s)
          : mode == kVectors ? norm_fwd<__nv_bfloat16, kVectors>(p, s)
                             : norm_fwd<__nv_bfloat16, kAny>(p, s);
  }
  return e == cudaSuccess ? MT_OK : MT_ECUDA;
}

size_t mt_gated_norm_workspace_bytes(int64_t n, int32_t dim, int32_t groups) {
  using namespace mt;
  if (n < 0 || n > MT_MAX_BLOCK_ROWS || dim < 1 || dim > MT_MAX_BLOCK_DIM || groups < 1 || groups > MT_MAX_GROUPS) return 0;
  return align_up(((size_t)bwd_blocks(n, dim, 2, false) + groups) * kSums * dim * 4, 256);
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
  Regions all;
  common_inputs(all, p);
  for (const Rows* r : {&p.dz, &p.dh, &p.y, &p.u, &p.z})
    all.in(r->data != nullptr ? Rows{r->data, r->ld, nullptr, nullptr} : *r, p.n, p.d, cfg->dtype);
  for (const Rows* r : {&p.dx, &p.dy, &p.du}) all.out(*r, p.n, p.d, cfg->dtype);
  for (const float* f : {p.dwp, p.dbp, p.dsc, p.dwq, p.dbq}) all.out(whole_region(f, (size_t)p.groups * p.d * 4));
  all.out(whole_region(ws, mt_gated_norm_workspace_bytes(p.n, p.d, p.groups)));
  if (all.clash()) return MT_EINVAL;
  p.part = static_cast<float*>(ws);
  p.blocks = bwd_blocks(p.n, p.d, (int)elem_bytes(cfg->dtype), p.bp != nullptr || p.bq != nullptr);
  bool wide = true;
  for (const Rows* r : {&p.dz, &p.dh, &p.y, &p.u, &p.z, &p.dx, &p.dy, &p.du})
    wide = wide && rows_wide(*r, p.d, cfg->dtype);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.n > 0) {
    MT_LAUNCH("k_norm_bwd", s);
    cudaError_t e;
    const int mode = mode_of(p, wide);
    if (cfg->dtype == MT_F32)
      e = mode == kWhole ? norm_bwd<float, kWhole>(p, s) : mode == kVectors ? norm_bwd<float, kVectors>(p, s) : norm_bwd<float, kAny>(p, s);
    else
      e = mode == kWhole     ? norm_bwd<__nv_bfloat16, kWhole>(p, s)
          : mode == kVectors ? norm_bwd<__nv_bfloat16, kVectors>(p, s)
                             : norm_bwd<__nv_bfloat16, kAny>(p, s);
    if (e != cudaSuccess) return MT_ECUDA;
  }
  {
    MT_LAUNCH("k_norm_sums", s);
    // as many groups at a time as the SMs hold blocks for; each block reads the offsets once (1024 groups x 2048 columns, one
    // row: the whole backward 104 us, with a block per group and 32 columns 1677)
    const int across = (p.d + 31) / 32 * 2, held = sm_count() * (64 / kSlices);
    const dim3 grid((p.d + 31) / 32, 2, std::max(1, std::min(p.groups, held / across)));
    k_norm_sums<<<grid, 32 * kSlices, offsets_smem(p.groups), s>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? MT_OK : MT_ECUDA;
}

}  // extern "C"
