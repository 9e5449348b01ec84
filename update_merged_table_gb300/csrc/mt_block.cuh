// Shared device code of the dense block's operators (mt_linear*.cu, mt_norm.cu,
// mt_pack.cu): ragged groups of rows, loads and stores of eight columns, and the
// 8-bit form of a block of 32 columns.
#pragma once

#include <atomic>

#include "mt_kernels.cuh"

namespace mt {

// Row tensors as the kernels see them (mt_rows with its data typed away).
using Rows = mt_rows;

// ---- ragged groups -------------------------------------------------------------
//
// Group g holds the rows [off[g], off[g+1]).  The offsets are device data, so
// they are made safe where they are read: clamped to [0, n] and replaced by
// their running maximum.  Offsets that needed either latch MT_EINVAL; whatever
// they were, the groups are then disjoint, in order and inside [0, n], so no
// access leaves a buffer and no row belongs to two groups.

__device__ __forceinline__ long long warp_max_scan(long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long w = __shfl_up_sync(kFull, v, o);
    if (lane >= o) v = w > v ? w : v;
  }
  return v;
}

__device__ __forceinline__ int warp_sum_scan(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int w = __shfl_up_sync(kFull, v, o);
    if (lane >= o) v += w;
  }
  return v;
}

// Fills s_off[0 .. G] (shared) with the safe offsets; every thread of the block calls it.
// offsets = NULL: one group of all rows.
__device__ __forceinline__ void load_offsets(const long long* offsets, int G, long long n, long long* s_off,
                                             int32_t* status) {
  if (offsets == nullptr) {
    if (threadIdx.x == 0) {
      s_off[0] = 0;
      s_off[1] = n;
    }
    __syncthreads();
    return;
  }
  for (int i = threadIdx.x; i <= G; i += blockDim.x) s_off[i] = offsets[i];
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    long long carry = 0;
    bool bad = false;
    for (int i0 = 0; i0 <= G; i0 += 32) {
      const int i = i0 + lane;
      const long long raw = i <= G ? s_off[i] : 0;
      long long v = raw < 0 ? 0 : (raw > n ? n : raw);
      v = warp_max_scan(v, lane);
      v = v < carry ? carry : v;
      if (i <= G) {
        bad |= v != raw;
        s_off[i] = v;
      }
      carry = __shfl_sync(kFull, v, 31);
    }
    if (bad && status != nullptr && blockIdx.x == 0 && blockIdx.y == 0) atomicCAS(status, 0, MT_EINVAL);
  }
  __syncthreads();
}

// s_cum[0 .. G] (shared): tiles of R rows in the groups before each one; after load_offsets, by every thread.
__device__ __forceinline__ void count_tiles(const long long* s_off, int G, int R, int* s_cum) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int carry = 0;
    for (int i0 = 0; i0 < G; i0 += 32) {
      const int i = i0 + lane;
      const int t = i < G ? (int)((s_off[i + 1] - s_off[i] + R - 1) / R) : 0;
      const int inc = warp_sum_scan(t, lane);
      if (i < G) s_cum[i] = carry + inc - t;
      carry += __shfl_sync(kFull, inc, 31);
    }
    if (lane == 0) s_cum[G] = carry;
  }
  __syncthreads();
}

// The last i in [0, G) with s_cum[i] <= t (so the group of tile t when t < s_cum[G]; empty groups are passed over).
__device__ __forceinline__ int tile_group(const int* s_cum, int G, int t) {
  int lo = 0, hi = G;  // s_cum[lo] <= t < s_cum[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s_cum[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The group of a row, -1 when the row is in none.
__device__ __forceinline__ int row_group(const long long* s_off, int G, long long row) {
  if (row < s_off[0] || row >= s_off[G]) return -1;
  int lo = 0, hi = G;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s_off[mid] <= row) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ---- 8-bit blocks ----------------------------------------------------------------
//
// 32 columns share the exponent e: the least with max|x| <= 127 * 2^e, held in
// [-120, 121] so that every value and both powers of two stay normal fp32
// numbers.  A column is q * 2^e with q = rint(x * 2^-e) in [-127, 127]: seven
// bits and a sign times a power of two, exact in bf16, so a product that reads
// it rounds nothing.  A block that holds an infinity or a NaN is stored with
// exponent byte 255 and stands for NaN.

constexpr int kPackBlock = MT_PACK_BLOCK;
constexpr uint32_t kPackNan = 255;

// Exponent byte (e + 127) of a block from the largest |x| as fp32 bits.
__device__ __forceinline__ uint32_t pack_exp_byte(uint32_t top) {
  if (top >= 0x7F800000u) return kPackNan;
  int e = (int)(top >> 23) - 127 - 6 + ((top & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);  // 127 = 1.984375 * 2^6
  e = e < -120 ? -120 : (e > 121 ? 121 : e);
  return (uint32_t)(e + 127);
}
__device__ __forceinline__ float pack_inv(uint32_t byte) {  // 2^-e; 0 for a block that is not finite
  return byte == kPackNan ? 0.0f : __uint_as_float((254u - byte) << 23);
}
__device__ __forceinline__ float pack_scale(uint32_t byte) {  // 2^e, or NaN
  return byte == kPackNan ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte << 23);
}
// The codes of four columns as bytes, v[j] = x[j] * 2^-e with |v[j]| <= 127.  Adding 1.5 * 2^23 rounds a product to
// the nearest integer (ties to even) in the last bits of the sum, whose low byte is then the code; the product itself
// is exact, so a fused multiply-add rounds once.
__device__ __forceinline__ uint32_t pack_codes4(float x0, float x1, float x2, float x3, float inv) {
  constexpr float kMagic = 12582912.0f;
  const uint32_t a = __float_as_uint(fmaf(x0, inv, kMagic)), b = __float_as_uint(fmaf(x1, inv, kMagic));
  const uint32_t c = __float_as_uint(fmaf(x2, inv, kMagic)), d = __float_as_uint(fmaf(x3, inv, kMagic));
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
// The same where the codes have to be clamped to [-127, 127] (the exponent is at its upper end), or the block is not
// finite (codes 0).
__device__ __forceinline__ uint32_t pack_codes4_edge(float x0, float x1, float x2, float x3, float inv) {
  if (inv == 0.0f) return 0u;
  auto cut = [&](float x) { return fminf(fmaxf(x * inv, -127.0f), 127.0f); };
  return pack_codes4(cut(x0), cut(x1), cut(x2), cut(x3), 1.0f);
}
constexpr uint32_t kPackEdge = 248;  // exponent bytes from here on take the edge form

// ---- eight columns of a row --------------------------------------------------------

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  uint32_t w;
  memcpy(&w, &v, 4);
  return w;
}

// Eight columns as they were loaded: bf16 in a, fp32 in a and b, 8-bit codes in a.x and a.y with the exponent
// byte in a.z.  Kept raw so that a row's loads are all issued before the first is used.
template <typename T>
struct Raw8 {
  uint4 a;
};
template <>
struct Raw8<float> {
  uint4 a, b;
};

// Element offset of a row: rows and strides fit 32 bits (checked on the host), so one wide multiplication.
__device__ __forceinline__ size_t row_offset(long long row, int64_t ld) { return (size_t)(uint32_t)row * (uint32_t)ld; }

// Columns [8 vec, 8 vec + 8) of `row`, or zeros where they lie past d.  AL: every row starts on 16 bytes (codes: 8)
// and d is a multiple of 8.
template <typename T, bool AL>
__device__ __forceinline__ Raw8<T> load8(const Rows& r, long long row, int vec, int d) {
  Raw8<T> v;
  v.a = make_uint4(0u, 0u, 0u, 0u);
  if constexpr (sizeof(T) == 4) v.b = v.a;
  const int c0 = vec * 8;
  if (c0 >= d) return v;
  if (r.data != nullptr) {
    const T* p = static_cast<const T*>(r.data) + row_offset(row, r.ld) + c0;
    if constexpr (AL) {
      v.a = __ldg(reinterpret_cast<const uint4*>(p));
      if constexpr (sizeof(T) == 4) v.b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    } else {
      const int k = min(8, d - c0);
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = j < k ? to_f<T>(p[j]) : 0.0f;
      if constexpr (sizeof(T) == 4) {
        v.a = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        v.b = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
      } else {
        v.a = make_uint4(bf16x2_of(f[0], f[1]), bf16x2_of(f[2], f[3]), bf16x2_of(f[4], f[5]), bf16x2_of(f[6], f[7]));
      }
    }
  } else {
    const int nb = (d + kPackBlock - 1) / kPackBlock;
    const int8_t* p = r.codes + row_offset(row, d) + c0;
    if constexpr (AL) {
      const uint2 c = __ldg(reinterpret_cast<const uint2*>(p));
      v.a.x = c.x;
      v.a.y = c.y;
    } else {
      const int k = min(8, d - c0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t q = j < k ? (uint32_t)(uint8_t)p[j] : 0u;
        if (j < 4) v.a.x |= q << (8 * j);
        else v.a.y |= q << (8 * (j - 4));
      }
    }
    v.a.z = __ldg(r.exps + row_offset(row, nb) + c0 / kPackBlock);
  }
  return v;
}

// The signed bytes of w times s: with the sign bit flipped a byte is q + 128, which stands in the last bits of
// 2^23 + 128 + q; taking 2^23 + 128 off leaves q exactly.
__device__ __forceinline__ void codes_f(uint32_t w, float s, float* f) {
  const uint32_t x = w ^ 0x80808080u;
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = (__uint_as_float(__byte_perm(x, 0x4B000000u, 0x7540 + j)) - 8388736.0f) * s;
}

template <typename T>
__device__ __forceinline__ void widen8(const Raw8<T>& v, bool packed, float f[8]) {
  if (packed) {
    const float s = pack_scale(v.a.z);
    codes_f(v.a.x, s, f);
    codes_f(v.a.y, s, f + 4);
  } else if constexpr (sizeof(T) == 4) {
    const uint32_t w[8] = {v.a.x, v.a.y, v.a.z, v.a.w, v.b.x, v.b.y, v.b.z, v.b.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(w[j]);
  } else {
    const uint32_t w[4] = {v.a.x, v.a.y, v.a.z, v.a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(w[j] << 16);
      f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
}

// ---- eight columns as four pairs ----------------------------------------------------
//
// The norms are bound by the instructions they issue as soon as their loads
// keep up, so their arithmetic works on pairs of columns (one instruction for
// two fp32 operations, each rounded as the single one is).

__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 both(float x) { return pk(x, x); }
__device__ __forceinline__ float pair_sum(f32x2 a) {
  const float2 f = upk(a);
  return f.x + f.y;
}

template <typename T>
__device__ __forceinline__ void widen8(const Raw8<T>& v, bool packed, f32x2 (&f)[4]) {
  if (packed) {
    // as codes_f does it, two columns an instruction
    const f32x2 s = both(pack_scale(v.a.z)), off = both(-8388736.0f);
    const uint32_t w[2] = {v.a.x ^ 0x80808080u, v.a.y ^ 0x80808080u};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t x = w[j >> 1];
      const int b = (j & 1) * 2;
      f[j] = mul2(add2(pk(__uint_as_float(__byte_perm(x, 0x4B000000u, 0x7540 + b)),
                          __uint_as_float(__byte_perm(x, 0x4B000000u, 0x7541 + b))),
                       off),
                  s);
    }
  } else if constexpr (sizeof(T) == 4) {
    const uint32_t w[8] = {v.a.x, v.a.y, v.a.z, v.a.w, v.b.x, v.b.y, v.b.z, v.b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = pk(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
  } else {
    const uint32_t w[4] = {v.a.x, v.a.y, v.a.z, v.a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = bf16x2_to_f32x2(w[j]);
  }
}

// Rounds eight columns to T.
template <typename T>
__device__ __forceinline__ Raw8<T> narrow8(const f32x2 (&f)[4]) {
  Raw8<T> v;
  float2 g[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) g[j] = upk(f[j]);
  if constexpr (sizeof(T) == 4) {
    v.a = make_uint4(__float_as_uint(g[0].x), __float_as_uint(g[0].y), __float_as_uint(g[1].x), __float_as_uint(g[1].y));
    v.b = make_uint4(__float_as_uint(g[2].x), __float_as_uint(g[2].y), __float_as_uint(g[3].x), __float_as_uint(g[3].y));
  } else {
    v.a = make_uint4(bf16x2_of(g[0].x, g[0].y), bf16x2_of(g[1].x, g[1].y), bf16x2_of(g[2].x, g[2].y),
                     bf16x2_of(g[3].x, g[3].y));
  }
  return v;
}

// Stores the columns of a vector that lie below d.
template <typename T, bool AL>
__device__ __forceinline__ void put8(const Rows& r, long long row, int vec, int d, const Raw8<T>& v) {
  const int c0 = vec * 8;
  if (c0 >= d) return;
  T* p = static_cast<T*>(r.data) + row_offset(row, r.ld) + c0;
  if constexpr (AL) {
    *reinterpret_cast<uint4*>(p) = v.a;
    if constexpr (sizeof(T) == 4) reinterpret_cast<uint4*>(p)[1] = v.b;
  } else {
    float f[8];
    widen8<T>(v, false, f);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c0 + j < d) p[j] = from_f<T>(f[j]);
  }
}

// The 8-bit form of a vector as it was stored or loaded (zeros past d): four neighbouring lanes hold a block's 32
// columns and call this together.
template <typename T, bool AL>
__device__ __forceinline__ void put_packed8(const Rows& r, long long row, int vec, int d, const Raw8<T>& v, bool live) {
  float f[8];
  widen8<T>(v, false, f);
  uint32_t top = 0;  // the largest magnitude as fp32 bits
  if constexpr (sizeof(T) == 2) {  // magnitudes of bf16 order as their 15 bits do, two to a word
    constexpr uint32_t k = 0x7FFF7FFFu;
    top = __vmaxu2(__vmaxu2(v.a.x & k, v.a.y & k), __vmaxu2(v.a.z & k, v.a.w & k));
    top = __vmaxu2(top, __shfl_xor_sync(kFull, top, 1));
    top = __vmaxu2(top, __shfl_xor_sync(kFull, top, 2));
    top = max(top << 16, top & 0xFFFF0000u);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(f[j]) & 0x7FFFFFFFu);
    top = max(top, __shfl_xor_sync(kFull, top, 1));
    top = max(top, __shfl_xor_sync(kFull, top, 2));
  }
  const int c0 = vec * 8;
  if (!live || c0 >= d) return;
  const uint32_t byte = pack_exp_byte(top);
  const float inv = pack_inv(byte);
  uint32_t w[2];
  if (byte < kPackEdge) {
    w[0] = pack_codes4(f[0], f[1], f[2], f[3], inv);
    w[1] = pack_codes4(f[4], f[5], f[6], f[7], inv);
  } else {
    w[0] = pack_codes4_edge(f[0], f[1], f[2], f[3], inv);
    w[1] = pack_codes4_edge(f[4], f[5], f[6], f[7], inv);
  }
  int8_t* p = r.codes + row_offset(row, d) + c0;
  if constexpr (AL) {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c0 + j < d) p[j] = (int8_t)(w[j >> 2] >> (8 * (j & 3)));
  }
  if ((vec & 3) == 0) r.exps[row_offset(row, (d + kPackBlock - 1) / kPackBlock) + vec / 4] = (uint8_t)byte;
}

// ---- host-side checks ------------------------------------------------------------------

inline bool is_aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Lets a kernel have `most` bytes of dynamic shared memory, what its largest launch needs.  The limit belongs to the kernel
// and the device, not to a launch: it is set once, to a constant, so that calls from several threads do not lower it for
// one another.  registers: a kernel that the compiler gave fewer is refused (asked for once, too).
class SmemLimit {
 public:
  template <typename Kernel>
  cudaError_t allow(Kernel kernel, size_t most, int registers = 0) {
    const int dev = current_device();
    if (dev < 0) return cudaErrorInvalidDevice;
    if (set_[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    const cudaError_t e =
        cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess) return e;
    if (registers > 0) {
      cudaFuncAttributes f;
      const cudaError_t fe = cudaFuncGetAttributes(&f, reinterpret_cast<const void*>(kernel));
      if (fe != cudaSuccess) return fe;
      if (f.numRegs < registers) return cudaErrorInvalidValue;
    }
    set_[dev].store(true, std::memory_order_relaxed);
    return cudaSuccess;
  }

 private:
  std::atomic<bool> set_[kMaxDevices] = {};
};

// A kernel that starts while the one before it on the stream ends: its blocks set themselves up and then wait (follow()) until
// that one is done and its writes are seen.  Every block calls follow() before it touches global memory, and lead() once it
// runs, which lets the next kernel's blocks in.  It is resident while the one before it (the caller's, or another call's) still
// writes, so it reads by ordinary loads: the read-only path is for memory that nothing writes during a kernel's whole life.
// (k_vocab_rows may read its caller's rows so: k_vocab_mark before it waited for everything in front of the call.)
__device__ __forceinline__ void follow() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void lead() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_following(void (*kernel)(P...), int grid, int threads, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

inline size_t elem_bytes(int dtype) { return dtype == MT_F32 ? 4 : 2; }

// A plain row tensor: pointer, element alignment, row stride of at least d and below 2^31.
inline bool rows_ok(const void* data, int64_t ld, int64_t d, int dtype) {
  return data != nullptr && is_aligned(data, elem_bytes(dtype)) && ld >= d && ld <= 0x7FFFFFFF;
}

// Whether eight-column vectors of a row tensor may be reached with 16-byte (codes: 8-byte) accesses.
inline bool rows_wide(const Rows& r, int64_t d, int dtype) {
  if (d % 8 != 0) return false;
  if (r.data != nullptr && (!is_aligned(r.data, 16) || (r.ld * elem_bytes(dtype)) % 16 != 0)) return false;
  return r.codes == nullptr || is_aligned(r.codes, 8);
}

// Where a call reads or writes: n runs of `width` bytes, `step` bytes apart.
struct Region {
  uintptr_t at = 0;
  long long n = 0, width = 0, step = 0;
};
inline Region whole_region(const void* p, size_t bytes) {
  return p == nullptr ? Region{} : Region{(uintptr_t)p, bytes > 0, (long long)bytes, (long long)bytes};
}

// Whether two regions share a byte.  Runs equally far apart (column slices of one tensor, alternate rows): exactly, from the
// runs of one that can reach a run of the other.  Otherwise: whether their address ranges meet.
inline bool regions_meet(const Region& a, const Region& b) {
  if (a.n == 0 || b.n == 0) return false;
  const long long d = (long long)(b.at - a.at);
  if (d >= (a.n - 1) * a.step + a.width || -d >= (b.n - 1) * b.step + b.width) return false;
  if (a.n == 1 && b.n == 1) return true;
  const long long step = a.n == 1 ? b.step : a.step;
  if ((b.n > 1 && b.step != step) || a.width > step || b.width > step) return true;
  long long k = d / step;  // b's first run starts k steps and r bytes (0 <= r < step) after a's
  if (k * step > d) --k;
  const long long r = d - k * step;
  auto same = [&](long long i) { return i <= a.n - 1 && -i <= b.n - 1; };  // some run of b lies i steps after one of a
  return (r < a.width && same(k)) || (r + b.width > step && same(k + 1));
}

// The inputs and outputs of a call, and whether an output shares a byte with an input or with another output.
class Regions {
 public:
  void in(const Region& r) {
    if (r.n > 0) in_[ins_++] = r;
  }
  void out(const Region& r) {
    if (r.n > 0) out_[outs_++] = r;
  }
  // A row tensor of n rows: its plain rows and its checkpoint.
  void in(const Rows& r, int64_t n, int64_t d, int dtype) {
    in(plain(r, n, d, dtype));
    in(whole_region(r.codes, (size_t)n * d));
    in(whole_region(r.exps, (size_t)n * ((d + kPackBlock - 1) / kPackBlock)));
  }
  void out(const Rows& r, int64_t n, int64_t d, int dtype) {
    out(plain(r, n, d, dtype));
    out_packed(r, n, d);
  }
  void out_packed(const Rows& r, int64_t n, int64_t d) {
    out(whole_region(r.codes, (size_t)n * d));
    out(whole_region(r.exps, (size_t)n * ((d + kPackBlock - 1) / kPackBlock)));
  }
  static Region plain(const Rows& r, int64_t n, int64_t d, int dtype) {
    const long long e = (long long)elem_bytes(dtype);
    return r.data == nullptr ? Region{} : Region{(uintptr_t)r.data, n, d * e, r.ld * e};
  }
  bool clash() const {
    for (int i = 0; i < outs_; ++i) {
      for (int j = 0; j < ins_; ++j)
        if (regions_meet(out_[i], in_[j])) return true;
      for (int j = 0; j < i; ++j)
        if (regions_meet(out_[i], out_[j])) return true;
    }
    return false;
  }

 private:
  Region in_[24], out_[16];  // the norms' backward has the most: 21 and 9
  int ins_ = 0, outs_ = 0;
};

}  // namespace mt
