// The losses over a vocabulary for narrow rows (up to 128 columns of bf16): their
// statistics, and gradients for which the gradient of the logits never leaves the
// chip.
//
// With few columns a logit is a few products and one exponential, and writing its
// gradient out (2 bytes) and reading it back twice costs more than making it
// again.  So there are two passes over the tiles of 128 rows by 128 entries, each
// with its own sum:
//
//   dx  a block keeps 128 rows of x and goes over entries of W
//   dW  a block keeps 128 entries of W and goes over rows of x
//
//   S = x W^T into tensor memory; dz from S by teams of four warps, rounded to bf16;
//   then dx += dz W, dz in tensor memory in the place of S (its rows are the
//   operand's), or dW += dz^T x, dz in shared memory (64 entries of a row are one
//   128-byte swizzled row) and read across; with the same tile of W or x that made
//   S, read across.
//
// One warp issues the products of S, as far ahead as there is room, another those
// of the sums as their dz comes, so neither waits for what the other waits for; teams of four warps take the
// tiles in turn, so that one's loads and waits overlap the others' arithmetic.
//
// Bound: by the latency from S to dz to the sum, three tiles of it under way, which tensor memory and shared memory have room
// for (16,384 rows x 98,001 x 64: statistics 295 us, dx 410, dW 425, about 1200 clocks a tile against 512 of exponentials and
// 690 of products).
#include "mt_tiles.cuh"
#include "mt_vocab.cuh"
#include "mt_vocab_rows.cuh"

namespace mt {
namespace {

constexpr int kT = 128;                  // rows and entries of a tile
constexpr int kSlab = kT * 128;          // 128 rows of 64 columns
constexpr int kDz = 2 * kSlab;           // a tile of dz
constexpr int kAccAt = 3 * kT;           // tensor memory: S, then the sum

struct FusedBarriers {
  uint64_t full[8], empty[8];        // a streamed tile has landed; its products are done
  uint64_t s_full[4], s_empty[4];    // S is finished; it has been read
  uint64_t dz_full[3];               // a team's dz is in its place
  uint64_t dz_empty[3];              // the products of a team's last tile of dz are done
  uint64_t kept_full, kept_empty;    // the kept tile has landed; its products are done
  uint64_t acc_full, acc_empty;      // a unit's sum is finished; it has been read
  uint64_t s_done, done;             // every product issued is done
  uint32_t tmem;
};

// What a launch computes: dx, dW, or the rows' statistics (with smoothing: the sums of their logits too).
enum Fused { kDx, kDw, kStats, kStatsSmooth };

// KS: slabs of 64 columns.  Teams of four warps, streamed tiles, S under way, and (dW) a tile of dz for each team.
template <int KS, int WHAT>
struct FusedRing {
  static constexpr int kTile = KS * kSlab;
  static constexpr int kTeams = WHAT >= kStats ? kNarrowTeams : KS == 1 ? 3 : 2, kThreads = (4 + kTeams * 4) * 32;
  static constexpr int kStages = KS == 1 ? 6 : WHAT == kDx ? 5 : 4;
  static constexpr int kS = WHAT >= kStats ? 4 : 3;  // S under way
  static constexpr int kDzAt = (1 + kStages) * kTile;
  // behind the tiles: dz (dW), or where the sum's rows are turned (dx)
  static constexpr int kBytes = kDzAt + (WHAT == kDw ? kTeams * kDz : WHAT == kDx ? 8 * 2048 : 0);
};

// A unit: a kept tile and streamed tiles [t0, t1).
struct FusedUnit {
  int kept, t0, t1, slot;
};
// The kept tiles that make whole rounds of the blocks go over all streamed tiles (if they are no more than kLongest terms); the
// rest are cut into `chunks` runs, so that the last round is a full one too (766 kept tiles on 152 blocks: five rounds and a
// 25th, not six).
struct FusedWork {
  int live, kept_tiles, streamed, whole, chunks;
  __device__ __forceinline__ int units() const { return whole + (kept_tiles - whole) * chunks; }
  __device__ __forceinline__ FusedUnit unit(int u) const {  // kept tiles fastest: blocks at work together read the same streamed tiles
    if (u < whole) return {u, 0, streamed, 0};
    const int rest = kept_tiles - whole, c = (u - whole) / rest;
    return {whole + (u - whole) - c * rest, (int)((long long)c * streamed / chunks), (int)((long long)(c + 1) * streamed / chunks), c};
  }
};

template <int KS, int WHAT>
__global__ void __launch_bounds__(FusedRing<KS, WHAT>::kThreads, 1)
k_vocab_fused(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w, const __grid_constant__ FusedParams p) {
  constexpr bool VOCAB = WHAT == kDw, STATS = WHAT >= kStats;
  using R = FusedRing<KS, WHAT>;
  constexpr int kS = R::kS;
  // a team's next tile waits for the products of its last: dW, whose dz has one place for each team; dx where there are more S
  // than teams (else the team's next S waits for them)
  constexpr bool kWaits = VOCAB || (WHAT == kDx && R::kTeams < kS);
  extern __shared__ uint8_t s_raw[];
  __shared__ FusedBarriers bar;
  uint8_t* base = reinterpret_cast<uint8_t*>(((uintptr_t)s_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* s_kept = base;
  uint8_t* s_ring = base + R::kTile;
  uint8_t* s_dz = base + R::kDzAt;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < R::kStages; ++i) {
      tc::mbar_init(&bar.full[i], 1);
      tc::mbar_init(&bar.empty[i], 1);
    }
    for (int i = 0; i < kS; ++i) {
      tc::mbar_init(&bar.s_full[i], 1);
      tc::mbar_init(&bar.s_empty[i], WHAT == kDx ? 1 : 4);
    }
    for (int i = 0; i < 3; ++i) {
      tc::mbar_init(&bar.dz_full[i], 4);
      tc::mbar_init(&bar.dz_empty[i], 1);
    }
    tc::mbar_init(&bar.kept_full, 1);
    tc::mbar_init(&bar.kept_empty, 1);
    tc::mbar_init(&bar.acc_full, 1);
    tc::mbar_init(&bar.acc_empty, 8);
    tc::mbar_init(&bar.s_done, 1);
    tc::mbar_init(&bar.done, 1);
    tc::mbar_init_fence();
  }
  __syncwarp();
  if (warp == 1) tc::tmem_alloc<1>(&bar.tmem, 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = bar.tmem;
  lead();
  follow();
  FusedWork work;
  work.live = *p.rows.count;
  {
    const int rt = (work.live + kT - 1) / kT, vt = (p.vocab + kT - 1) / kT;
    work.kept_tiles = VOCAB ? vt : rt;
    work.streamed = VOCAB ? rt : vt;
    const int least = STATS ? 1 : max(1, (work.streamed + kLongest / kT - 1) / (kLongest / kT));
    work.whole = VOCAB ? p.whole : STATS || least > 1 ? 0 : work.kept_tiles / (int)gridDim.x * (int)gridDim.x;
    work.chunks = choose_chunks(work.kept_tiles - work.whole, work.streamed, p.max_chunks, gridDim.x, 4, least);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      p.cut[0] = STATS ? work.chunks : work.whole * kT;
      p.cut[1] = work.chunks;
    }
  }
  const int units = work.units();

  if (warp == 0) {
    const bool one = tc::elect_one();
    tc::Slot s;
    long long issued = 0;
    uint32_t kept_phase = 0;
    bool ok = true, any = false;
    const CUtensorMap* kept_map = VOCAB ? &map_w : &map_x;
    const CUtensorMap* ring_map = VOCAB ? &map_x : &map_w;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const FusedUnit x = work.unit(u);
      if (x.t0 == x.t1) continue;
      ok = tc::warp_wait(&bar.kept_empty, kept_phase ^ 1);
      if (!ok) break;
      kept_phase ^= 1;
      any = true;
      if (one) {
        tc::mbar_expect(&bar.kept_full, R::kTile);
#pragma unroll
        for (int k = 0; k < KS; ++k) tc::tma_load_2d(s_kept + k * kSlab, kept_map, &bar.kept_full, k * 64, x.kept * kT);
      }
      __syncwarp();
      for (int t = x.t0; t < x.t1; ++t) {
        ok = tc::warp_wait(&bar.empty[s.stage], s.phase ^ 1);
        if (!ok) break;
        if (one) {
          uint8_t* st = s_ring + s.stage * R::kTile;
          tc::mbar_expect(&bar.full[s.stage], R::kTile);
#pragma unroll
          for (int k = 0; k < KS; ++k) tc::tma_load_2d(st + k * kSlab, ring_map, &bar.full[s.stage], k * 64, t * kT);
        }
        __syncwarp();
        ++issued;
        s.next<R::kStages>();
      }
    }
    ok = ok && tc::all_released<R::kStages>(bar, s, issued);
    if (!ok) {
      if (one) tc::latch_status(p.status, MT_ECUDA);
      tc::drain<R::kStages>(bar, s, issued);
      if (any) tc::mbar_wait(&bar.kept_full, kept_phase ^ 1);
    }
  } else if (warp == 1) {
    // S: as far ahead as there is room
    constexpr uint32_t instr = tc::instr_bf16(kT, kT, false, false);
    const bool one = tc::elect_one();
    const uint32_t kept = tc::desc_low(tc::smem_addr(s_kept), 16), ring = tc::desc_low(tc::smem_addr(s_ring), 16);
    tc::Slot s;
    uint32_t b = 0, phase = 0, kept_phase = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const FusedUnit x = work.unit(u);
      if (x.t0 == x.t1) continue;
      ok = tc::warp_wait(&bar.kept_full, kept_phase);
      kept_phase ^= 1;
      for (int t = x.t0; t < x.t1 && ok; ++t) {
        ok = tc::warp_wait(&bar.s_empty[b], phase ^ 1) && tc::warp_wait(&bar.full[s.stage], s.phase);
        if (!ok) break;
        tc::fence_after();
        const uint32_t at = ring + s.stage * (R::kTile >> 4);
        const uint32_t ax = VOCAB ? at : kept, aw = VOCAB ? kept : at;
        if (one) {
#pragma unroll
          for (int i = 0; i < KS * 4; ++i) {
            const uint32_t o = ((i >> 2) * kSlab + (i & 3) * 32) >> 4;
            tc::mma_bf16<1>(tmem + b * kT, ax + o, aw + o, instr, i > 0);
          }
          if (STATS) tc::mma_commit<1>(&bar.empty[s.stage]);
          tc::mma_commit<1>(&bar.s_full[b]);
          if (STATS && t + 1 == x.t1) tc::mma_commit<1>(&bar.kept_empty);
        }
        __syncwarp();
        if (++b == kS) {
          b = 0;
          phase ^= 1;
        }
        s.next<R::kStages>();
      }
    }
    if (one) tc::mma_commit<1>(&bar.s_done);  // tensor memory is freed only when no product writes it, also after a wait ran out
    __syncwarp();
    ok = tc::mbar_wait(&bar.s_done, 0) && ok;
    if (!ok && one) tc::latch_status(p.status, MT_ECUDA);
  } else if (!STATS && warp == 2) {
    // the sums.  A tile's S is done before its dz is, so what this warp signals of a sum holds for its S too.
    constexpr uint32_t instr = tc::instr_bf16(kT, KS * 64, VOCAB, true);
    const bool one = tc::elect_one();
    const uint32_t ring = tc::desc_low(tc::smem_addr(s_ring), kSlab), dz = tc::desc_low(tc::smem_addr(s_dz), kSlab);
    tc::Slot s;
    uint32_t n = 0, acc_phase = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const FusedUnit x = work.unit(u);
      if (x.t0 == x.t1) continue;
      ok = tc::warp_wait(&bar.acc_empty, acc_phase ^ 1);
      acc_phase ^= 1;
      for (int t = x.t0; t < x.t1 && ok; ++t) {
        const uint32_t b = n % R::kTeams;
        ok = tc::warp_wait(&bar.dz_full[b], n / R::kTeams & 1);
        if (!ok) break;
        tc::fence_after();
        const uint32_t from = dz + b * (kDz >> 4), with = ring + s.stage * (R::kTile >> 4);
        if (one) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (VOCAB) tc::mma_bf16<1>(tmem + kAccAt, from + (i * 2048 >> 4), with + (i * 2048 >> 4), instr, t > x.t0 || i > 0);
            else tc::mma_bf16_tmem(tmem + kAccAt, tmem + n % kS * kT + i * 8, with + (i * 2048 >> 4), instr, t > x.t0 || i > 0);
          }
          tc::mma_commit<1>(&bar.empty[s.stage]);
          if (!VOCAB) tc::mma_commit<1>(&bar.s_empty[n % kS]);
          if (kWaits) tc::mma_commit<1>(&bar.dz_empty[b]);
        }
        __syncwarp();
        ++n;
        s.next<R::kStages>();
      }
      if (!ok) break;
      if (one) {
        tc::mma_commit<1>(&bar.kept_empty);
        tc::mma_commit<1>(&bar.acc_full);
      }
      __syncwarp();
    }
    if (one) tc::mma_commit<1>(&bar.done);
    __syncwarp();
    ok = tc::mbar_wait(&bar.done, 0) && ok;
    if (!ok && one) tc::latch_status(p.status, MT_ECUDA);
  } else if (STATS && warp >= 4) {
    const int quad = warp & 3, team = (warp - 4) >> 2;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    uint32_t n = 0;  // tiles so far
    bool ok = true;
    RowTargets to;
    RowStats<WHAT == kStatsSmooth> stats;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const FusedUnit x = work.unit(u);
      const int row = x.kept * kT + quad * 32 + lane;
      to.start(p.rows, row, work.live, x.t0 * kT);
      stats.clear();
      for (int t = x.t0 + (team + R::kTeams - (int)(n % R::kTeams)) % R::kTeams; t < x.t1; t += R::kTeams) {
        // (a team sees every third S or so of a buffer: the S before are done before its own is)
        const uint32_t of = n + (t - x.t0), b = of % kS, from = tmem + b * kT + lanes;
        const int v0 = t * kT, left = p.vocab - v0;
        const bool some = left < kT || __any_sync(kFull, to.next < v0 + kT);
        ok = tc::warp_wait(&bar.s_full[b], of / kS & 1);
        if (!ok) break;
        tc::fence_after();
#pragma unroll
        for (int c = 0; c < kT; c += 64) {
          uint32_t v[2][32];
          tc::tmem_load32(from + c, v[0]);
          tc::tmem_load32(from + c + 32, v[1]);
          tc::tmem_load_wait(v[0]);
          tc::tmem_loaded(v[1]);
          if (c + 64 == kT) {
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bar.s_empty[b]);
          }
          if (some) {
            to.pick(p.rows, v0 + c, v[0], p.picked);
            to.pick(p.rows, v0 + c + 32, v[1], p.picked);
          }
          stats.add(v, p.scale2, some ? left - c : 64);
        }
      }
      if (!ok) break;
      n += x.t1 - x.t0;
      if (row < work.live) {
        const size_t at = (size_t)(x.slot * R::kTeams + team) * p.stride + row;
        p.stats[at] = make_float2(stats.top, stats.sum);
        if (WHAT == kStatsSmooth) p.sum_z[at] = stats.total;
      }
    }
    if (!ok) tc::latch_status(p.status, MT_ECUDA);
  } else if (!STATS && warp >= 4) {
    const int quad = warp & 3, team = (warp - 4) >> 2;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    // dW: the warp's rows of dz, through which the sum goes out too; the thread's row: two halves of 64 entries
    uint8_t* const stage = VOCAB ? s_dz + team * kDz + quad * 4096 : s_dz + (team & 1) * 8192 + quad * 2048;
    uint8_t* const dz = stage + lane * 128;
    const f32x2 s2 = both(p.scale2);
    uint32_t n = 0, acc_phase = 0;  // tiles so far
    bool ok = true;
    RowTargets to;
    float4 k = make_float4(0.0f, 0.0f, 0.0f, 0.0f), k_next = k;
    int id_next = 0x7FFFFFFF;  // a row's only target
    // dz of 32 entries from their logits: four 16-byte pieces of a swizzled 128-byte row (dW), or 16 columns of tensor memory in
    // the place of S, whose columns up to there have been read (dx)
    auto columns = [&](const uint32_t (&v)[32], uint32_t from, int c, int row, int v0, bool some) {
      float f[32];
      const f32x2 x2 = both(-k.x), y2 = both(k.y), z2 = both(-k.z);
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        const float2 e = upk(fma2(pk(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), s2, x2));
        const float2 g = upk(fma2(pk(exp2_of(e.x), exp2_of(e.y)), y2, z2));
        f[j] = g.x;
        f[j + 1] = g.y;
      }
      if (some) {  // targets, or entries or rows that are not there
        to.take(p.rows, v0 + c, k.w, f);
        const uint32_t there = row < work.live ? below(p.vocab - v0 - c) : 0u;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (!(there >> j & 1)) f[j] = 0.0f;
      }
      if constexpr (!VOCAB) {
        uint32_t w[16];
        tiles::narrow32(f, w);
        tc::tmem_store16(from + (c >> 1), w);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint4*>(dz + (c >> 6) * kSlab + (((((c >> 5) & 1) * 4 + q) ^ (lane & 7)) << 4)) =
              make_uint4(bf16x2_of(f[q * 8], f[q * 8 + 1]), bf16x2_of(f[q * 8 + 2], f[q * 8 + 3]), bf16x2_of(f[q * 8 + 4], f[q * 8 + 5]),
                         bf16x2_of(f[q * 8 + 6], f[q * 8 + 7]));
      }
    };
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const FusedUnit x = work.unit(u);
      if (x.t0 < x.t1) {
        auto row_at = [&](int tile) { return tile * kT + quad * 32 + lane; };
        auto id_at = [&](int row) { return p.rows.top == 1 && row < work.live ? p.rows.ids[row] : 0x7FFFFFFF; };
        auto coef_at = [&](int row) { return row < work.live ? p.coef[row] : make_float4(0.0f, 0.0f, 0.0f, 0.0f); };
        const int first = x.t0 + (team + R::kTeams - (int)(n % R::kTeams)) % R::kTeams;  // this team's first tile
        if (VOCAB) {
          k_next = coef_at(row_at(first));
          id_next = id_at(row_at(first));
        } else {
          k = coef_at(row_at(x.kept));
          to.start(p.rows, row_at(x.kept), work.live, x.t0 * kT);
        }
        for (int t = first; t < x.t1; t += R::kTeams) {
          // (a team sees every third S or so of a buffer: its tiles' S come in order, so that one of an earlier turn is done)
          const uint32_t of = n + (t - x.t0), b = of % kS, from = tmem + b * kT + lanes;
          const int row = row_at(VOCAB ? t : x.kept), v0 = (VOCAB ? x.kept : t) * kT;
          if (VOCAB) {
            k = k_next;
            if (p.rows.top == 1) {
              to.row = row;
              to.pos = 0;
              to.next = id_next >= v0 ? id_next : 0x7FFFFFFF;
            } else {
              to.start(p.rows, row, work.live, v0);
            }
            if (t + R::kTeams < x.t1) {
              k_next = coef_at(row_at(t + R::kTeams));
              id_next = id_at(row_at(t + R::kTeams));
            }
          }
          const bool some = __any_sync(kFull, to.next < v0 + kT || row >= work.live) || v0 + kT > p.vocab;
          ok = __all_sync(kFull, tc::mbar_wait(&bar.s_full[b], of / kS & 1) && (!kWaits || tc::mbar_wait(&bar.dz_empty[team], (of / R::kTeams & 1) ^ 1)));
          if (!ok) break;
          tc::fence_after();
#pragma unroll
          for (int c = 0; c < kT; c += 64) {
            uint32_t v[2][32];
            tc::tmem_load32(from + c, v[0]);
            tc::tmem_load32(from + c + 32, v[1]);
            tc::tmem_load_wait(v[0]);
            tc::tmem_loaded(v[1]);
            if (VOCAB && c + 64 == kT) {
              tc::fence_before();
              __syncwarp();
              if (lane == 0) tc::mbar_arrive(&bar.s_empty[b]);
            }
            columns(v[0], from, c, row, v0, some);
            columns(v[1], from, c + 32, row, v0, some);
          }
          if (VOCAB) {
            tc::fence_async_proxy();
          } else {
            tc::tmem_store_wait();
            tc::fence_before();
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&bar.dz_full[team]);
        }
        if (!ok) break;
        n += x.t1 - x.t0;
      }
      // The unit's sum, by the first two teams: 32 columns at a time.  A third neither reads it nor waits for it: it has no tile
      // in some units of one or two, acc_empty does not count it, so sums could be two phases ahead of a wait here, which a
      // parity cannot tell from none.  Its next dz waits for what it needs: dx for S (free again once the sum has had the dz
      // there), dW for dz_empty.
      if (team >= 2) continue;
      if (x.t0 < x.t1) {
        ok = __all_sync(kFull, tc::mbar_wait(&bar.acc_full, acc_phase));
        if (!ok) break;
        acc_phase ^= 1;
        tc::fence_after();
      }
      const int c0 = team * KS * 32;  // half of the columns each team
      const int rows = min(32, (VOCAB ? p.vocab : work.live) - (x.kept * kT + quad * 32));
      const long long r0 = x.kept * kT + quad * 32;
#pragma unroll
      for (int c = 0; c < KS; ++c) {
        uint32_t v[32];
        if (x.t0 < x.t1) {
          tc::tmem_load32(tmem + kAccAt + c0 + c * 32 + lanes, v);
          tc::tmem_load_wait(v);
          if (c + 1 == KS) {
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bar.acc_empty);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0u;
        }
        float f[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(v[j]);
        if (VOCAB && x.kept < work.whole)
          tiles::store32<__nv_bfloat16>(stage, lane, f, p.out, p.columns, r0, rows, c0 + c * 32, p.columns, p.reach);
        else
          tiles::store32<float>(stage, lane, f, p.part + (size_t)x.slot * p.stride * p.columns, p.columns, VOCAB ? r0 - work.whole * kT : r0,
                                rows, c0 + c * 32, p.columns, p.reach_part);
      }
    }
    if (!ok) tc::latch_status(p.status, MT_ECUDA);
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 1) tc::tmem_free<1>(tmem, 512);
}

template <int KS, int WHAT>
cudaError_t launch(const char* name, const CUtensorMap& x, const CUtensorMap& w, const FusedParams& p, long long units, cudaStream_t s) {
  using R = FusedRing<KS, WHAT>;
  constexpr size_t bytes = 1024 + R::kBytes;
  static SmemLimit limit;
  const cudaError_t e = limit.allow(k_vocab_fused<KS, WHAT>, bytes);
  if (e != cudaSuccess) return e;
  const int blocks = sm_count();
  MT_LAUNCH(name, s);
  return launch_following(k_vocab_fused<KS, WHAT>, (int)(units < blocks ? (units > 0 ? units : 1) : blocks), R::kThreads, bytes, s, x, w, p);
}

template <int WHAT>
cudaError_t launch_of(const char* name, const CUtensorMap& x, const CUtensorMap& w, const FusedParams& p, long long units, cudaStream_t s) {
  return p.columns <= 64 ? launch<1, WHAT>(name, x, w, p, units, s) : launch<2, WHAT>(name, x, w, p, units, s);
}

}  // namespace

cudaError_t launch_fused(bool vocab, const FusedParams& p, const CUtensorMap& x, const CUtensorMap& w, long long units, cudaStream_t s) {
  return vocab ? launch_of<kDw>("k_vocab_fused_dw", x, w, p, units, s) : launch_of<kDx>("k_vocab_fused_dx", x, w, p, units, s);
}
cudaError_t launch_narrow_stats(const FusedParams& p, const CUtensorMap& x, const CUtensorMap& w, long long units, cudaStream_t s) {
  return p.sum_z != nullptr ? launch_of<kStatsSmooth>("k_vocab_fused_stats", x, w, p, units, s) : launch_of<kStats>("k_vocab_fused_stats", x, w, p, units, s);
}

}  // namespace mt
