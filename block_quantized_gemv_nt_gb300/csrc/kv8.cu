// kv8.cu — the 8-bit KV cache: rows quantised as they are written and read
// back, attention over the cache, and attention over the blocks that a bound on
// their scores selects for each query.  It stands beside the F16 cache
// ("Ntransformer", en.unwiki.net, roadmap) and the attention over it (ops.cu).
//
// Cache: bytes [n_kvh][kv_stride][HD]; one scale per 64 positions (a block) and
// head, for K and for V.  A scale is a power of two, so dividing by it is exact:
// what is stored depends only on the values, not on how the division rounds,
// and a block whose scale has to grow while it fills (a later token is larger)
// loses nothing but the low bits that the larger scale cannot hold.
#include <cuda_fp16.h>
#include <algorithm>
#include <type_traits>

#include "kv8_choose.cuh"
#include "nt_internal.cuh"
#include "ops.cuh"

namespace nt {
namespace {

constexpr int kB = kKv8Block;

// ---- scales and 8-bit values ---------------------------------------------------

// the least power of two t >= 2^-100 with a <= QMAX t (a >= 0, finite).  QMAX =
// 1.m * 2^E: t = 2^(e - E) when the mantissa of a (exponent e) is at most m, else
// one more.
template <int E, uint32_t MANT>
__device__ __forceinline__ float pow2_scale(float a) {
  const uint32_t u = __float_as_uint(a);
  int e = int(u >> 23) - 127 - E + ((u & 0x7FFFFFu) > MANT ? 1 : 0);
  e = e < -100 ? -100 : e;
  return __uint_as_float(uint32_t(e + 127) << 23);
}
template <int FMT>
__device__ __forceinline__ float kv8_scale(float a) {
  if (FMT == NT_KV8_I8) return pow2_scale<6, 0x7E0000u>(a);  // QMAX 127 = 1.984375 * 2^6
  return pow2_scale<8, 0x600000u>(a);                        // QMAX 448 = 1.75 * 2^8
}
// the least power of two >= t (positive and normal)
__device__ __forceinline__ float pow2_ceil(float t) {
  return __uint_as_float((__float_as_uint(t) + 0x7FFFFFu) & 0xFF800000u);
}
__device__ __forceinline__ float pow2_inv(float t) { return __uint_as_float((254u << 23) - __float_as_uint(t)); }

// four finite values times inv (1 / scale) -> four bytes, nearest, ties to even.  I8:
// one fused step adds 1.5 * 2^23, which leaves the rounded number in the low byte.
template <int FMT>
__device__ __forceinline__ uint32_t pack8(const float v[4], float inv) {
  if (FMT == NT_KV8_I8) {
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = fmaf(v[i], inv, 12582912.f);
    const uint32_t lo = __byte_perm(__float_as_uint(q[0]), __float_as_uint(q[1]), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(q[2]), __float_as_uint(q[3]), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
  }
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v[1] * inv), "f"(v[0] * inv));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v[3] * inv), "f"(v[2] * inv));
  return uint32_t(lo) | (uint32_t(hi) << 16);
}

// (x & m) ^ b as one three-input operation
__device__ __forceinline__ uint32_t and_xor(uint32_t x, uint32_t m, uint32_t b) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(r) : "r"(x), "r"(m), "r"(b));
  return r;
}

// Four bytes as two f16 pairs, exact.
//  I8: bytes (0, 2) and (1, 3): q + 128 in the mantissa of 1024 + (q + 128), minus
//  1152.  Masking, the sign bias and the exponent are one three-input operation.
//  E4M3: bytes (0, 1) and (2, 3) through the hardware's conversion.
template <int FMT>
__device__ __forceinline__ void to_h2(uint32_t x, uint32_t& a, uint32_t& b) {
  if (FMT == NT_KV8_I8) {
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));
    const uint32_t even = and_xor(x, 0x00FF00FFu, 0x64806480u), odd = and_xor(x >> 8, 0x00FF00FFu, 0x64806480u);
    const __half2 h0 = __hsub2(*reinterpret_cast<const __half2*>(&even), bias);
    const __half2 h1 = __hsub2(*reinterpret_cast<const __half2*>(&odd), bias);
    a = *reinterpret_cast<const uint32_t*>(&h0);
    b = *reinterpret_cast<const uint32_t*>(&h1);
  } else {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(a) : "h"(uint16_t(x & 0xFFFFu)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"(uint16_t(x >> 16)));
  }
}
// the byte of the first pair's second value (the other pair holds the other two)
template <int FMT>
constexpr int kPairStep = FMT == NT_KV8_I8 ? 2 : 1;
// words of two rows -> a word whose to_h2 pairs are (row 0, row 1) of bytes 0 and 1 (half 0) or 2 and 3
template <int FMT>
__device__ __forceinline__ uint32_t interleave8(uint32_t r0, uint32_t r1, int half) {
  return FMT == NT_KV8_I8 ? __byte_perm(r0, r1, half ? 0x7632 : 0x5410) : __byte_perm(r0, r1, half ? 0x7362 : 0x5140);
}

// four bytes -> values over the scale
template <int FMT>
__device__ __forceinline__ float4 unpack8(uint32_t x) {
  uint32_t lo, hi;
  to_h2<FMT>(x, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return FMT == NT_KV8_I8 ? make_float4(a.x, b.x, a.y, b.y) : make_float4(a.x, a.y, b.x, b.y);
}

// ---- write ---------------------------------------------------------------------
constexpr int kAppendThreads = 256;

struct AppendArgs {
  const void* src[2];        // K, V rows
  int64_t tok_stride, head_stride;
  uint8_t* dst[2];
  float* scale[2];
  int8_t *kmin, *kmax;       // nullable
  int64_t n, pos, kv_stride, nb;
  const int64_t* pos_dev;
  unsigned* err;
};

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

__device__ __forceinline__ float max_nan(float a, float b) {  // the larger; NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 h2f(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2*>(&h)); }

struct AppendShared {
  float red[kAppendThreads / 32];
  float smin[kAppendThreads / 32][128], smax[kAppendThreads / 32][128];
};

// One CTA per (block, head, K or V).  Its rows stay in registers from the load to
// the store: the largest |x| is reduced over the CTA between them, so the source
// is read once.  Rows the block already holds are loaded in the same round and
// restated only when the scale grows.  FULL: the rows are the whole block, and no
// row is tested.  Prompts are bound by HBM (32,767 F32 rows of 8 x 128: 50 us, 335 MB
// at 6.7 TB/s; 131,072 F16 rows to E4M3: 120 us, 805 MB at 6.7 TB/s); a single token
// by the latency of its two memory round trips (2.35 us).
template <int FMT, int HD, typename T, bool FULL>
__device__ __forceinline__ void append_block(const AppendArgs& a, AppendShared& sh, int64_t pos, int64_t blk, int r0,
                                             int r1) {
  constexpr int VEC = 16 / int(sizeof(T));    // channels per thread: 16 bytes of the source
  constexpr int TR = HD / VEC;                // threads per row
  constexpr int RP = kAppendThreads / TR;     // rows per pass
  constexpr int NP = kB / RP;
  constexpr int W = kAppendThreads / 32;
  const int64_t p0 = blk * kB;
  const int h = blockIdx.y, w = blockIdx.z;
  const int tr = threadIdx.x % TR, row = threadIdx.x / TR, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T* src = static_cast<const T*>(w ? a.src[1] : a.src[0]) + int64_t(h) * a.head_stride +
                 (p0 - pos) * a.tok_stride + VEC * tr;
  uint8_t* dst = (w ? a.dst[1] : a.dst[0]) + (int64_t(h) * a.kv_stride + p0) * HD + VEC * tr;
  float* scale = (w ? a.scale[1] : a.scale[0]) + int64_t(h) * a.nb + blk;

  // row r of the block, this thread's channels: the source's, or (below r0) the cache's
  const auto load_row = [&](int r) {
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (FULL || (r >= r0 && r < r1)) {
      x = *reinterpret_cast<const uint4*>(src + r * a.tok_stride);
    } else if (r < r0) {
      x.x = *reinterpret_cast<const uint32_t*>(dst + r * HD);
      if (VEC == 8) x.y = *reinterpret_cast<const uint32_t*>(dst + r * HD + 4);
    }
    return x;
  };
  uint4 raw[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) raw[i] = load_row(row + i * RP);
  const float t_old = !FULL && r0 > 0 ? *scale : 0.f;
  // channels 4 k .. 4 k + 3 of a loaded row: the source's values, or over the old scale the cache's
  const auto values = [&](const uint4& x, int r, int k, float v[4]) {
    if (!FULL && r < r0) {
      const float4 f = unpack8<FMT>(k ? x.y : x.x);
      v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else if (VEC == 4) {
      v[0] = __uint_as_float(x.x), v[1] = __uint_as_float(x.y);
      v[2] = __uint_as_float(x.z), v[3] = __uint_as_float(x.w);
    } else {
      const float2 y = h2f(k ? x.z : x.x), z = h2f(k ? x.w : x.y);
      v[0] = y.x, v[1] = y.y, v[2] = z.x, v[3] = z.y;
    }
  };
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    if (!FULL && row + i * RP < r0) continue;
    if (VEC == 4) {
      float v[4];
      values(raw[i], row + i * RP, 0, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) amax = max_nan(amax, fabsf(v[j]));
    } else {
      const __half2* x = reinterpret_cast<const __half2*>(&raw[i]);
      const __half2 m = __hmax2_nan(__hmax2_nan(__habs2(x[0]), __habs2(x[1])), __hmax2_nan(__habs2(x[2]), __habs2(x[3])));
      const float2 f = __half22float2(m);
      amax = max_nan(amax, max_nan(f.x, f.y));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (lane == 0) sh.red[warp] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < W; ++i) amax = max_nan(amax, sh.red[i]);
  const bool clean = amax <= 3.402823466e38f;
  if (!clean) {
    // a NaN or an infinity: the scale follows the finite values.  Here and below the
    // rows are loaded again, in loops that are not unrolled: this rare case's code in
    // the loops of the others cost every call (one token 2.48 against 2.35 us, the
    // 131,072-row conversion 129.8 against 119.7).
    if (threadIdx.x == 0) flag_error(a.err, kErrNonFinite);
    amax = 0.f;
#pragma unroll 1
    for (int r = row; r < r1; r += RP) {
      if (r < r0) continue;
      const uint4 x = load_row(r);
#pragma unroll
      for (int k = 0; k < VEC / 4; ++k) {
        float v[4];
        values(x, r, k, v);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (fabsf(v[j]) <= 3.402823466e38f) amax = fmaxf(amax, fabsf(v[j]));
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    __syncthreads();
    if (lane == 0) sh.red[warp] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < W; ++i) amax = fmaxf(amax, sh.red[i]);
  }
  // A block begun elsewhere may have any scale: it goes on at the next power of two,
  // and its rows are restated to it like those of a block that grows.
  const float t = fmaxf(kv8_scale<FMT>(amax), pow2_ceil(t_old));
  const float inv = pow2_inv(t), restate = t_old * inv;
  if (threadIdx.x == 0) *scale = t;

  const bool sums = w == 0 && a.kmin;
  // bounds of the stored values (plus `offset`), exact in f16; pair j: channels ch and ch + PS
  constexpr bool HALF = FULL && VEC == 8;
  constexpr int PS = HALF ? 1 : kPairStep<FMT>;
  float offset = 0.f;
  __half2 lo[VEC / 2], hi[VEC / 2];
#pragma unroll
  for (int j = 0; j < VEC / 2; ++j) {
    lo[j] = __half2half2(__ushort_as_half(0x7C00));  // +inf
    hi[j] = __half2half2(__ushort_as_half(0xFC00));
  }
  const auto bound = [&](int j, uint32_t z) {
    const __half2 y = *reinterpret_cast<const __half2*>(&z);
    lo[j] = __hmin2(lo[j], y);
    hi[j] = __hmax2(hi[j], y);
  };
  // one row: packed, stored, bounded.  CLEAN: finite values; else NaN is stored as 0 and an
  // infinity as the largest value, clamped over the scale, where that cannot overflow
  const auto put_row = [&](auto clean_row, int r, const uint4& x) {
    constexpr bool CLEAN = decltype(clean_row)::value;
    const bool old = !FULL && r < r0;
    uint32_t packed[VEC / 4];
#pragma unroll
    for (int k = 0; k < VEC / 4; ++k) {
      float v[4];
      values(x, r, k, v);
      if (!CLEAN && !old) {
        constexpr float top = FMT == NT_KV8_I8 ? 127.f : 448.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = v[j] != v[j] ? 0.f : fminf(fmaxf(v[j] * inv, -top), top);
      }
      packed[k] = pack8<FMT>(v, old ? restate : CLEAN ? inv : 1.f);
      if (sums) {
        uint32_t z[2];
        to_h2<FMT>(packed[k], z[0], z[1]);
        if (PS != kPairStep<FMT>) {
          const uint32_t y = __byte_perm(z[0], z[1], 0x5410);
          z[1] = __byte_perm(z[0], z[1], 0x7632);
          z[0] = y;
        }
        bound(2 * k, z[0]);
        bound(2 * k + 1, z[1]);
      }
    }
    if (!old || restate != 1.f) {
      if (VEC == 4)
        *reinterpret_cast<uint32_t*>(dst + r * HD) = packed[0];
      else
        *reinterpret_cast<uint2*>(dst + r * HD) = make_uint2(packed[0], packed[VEC / 4 - 1]);
    }
  };
  if (HALF && clean && inv <= 32768.f) {
    // F16 rows stay F16: the product with a power of two is exact down to the f16
    // subnormals, which are far below half of the least 8-bit value; I8 adds 1.5 *
    // 2^10 in the same step, which rounds to the whole number in the low byte
    const __half2 inv2 = __half2half2(__float2half_rn(inv)), magic = __half2half2(__ushort_as_half(0x6600));
    if (FMT == NT_KV8_I8) offset = 1536.f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const __half2* x = reinterpret_cast<const __half2*>(&raw[i]);
      uint32_t packed[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t z[2];
        if (FMT == NT_KV8_I8) {
          const __half2 q0 = __hfma2(x[2 * k], inv2, magic), q1 = __hfma2(x[2 * k + 1], inv2, magic);
          z[0] = *reinterpret_cast<const uint32_t*>(&q0);
          z[1] = *reinterpret_cast<const uint32_t*>(&q1);
          packed[k] = __byte_perm(z[0], z[1], 0x6420);
        } else {
          const __half2 q0 = __hmul2(x[2 * k], inv2), q1 = __hmul2(x[2 * k + 1], inv2);
          uint16_t b0, b1;
          asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(b0) : "r"(*reinterpret_cast<const uint32_t*>(&q0)));
          asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(b1) : "r"(*reinterpret_cast<const uint32_t*>(&q1)));
          packed[k] = uint32_t(b0) | (uint32_t(b1) << 16);
          if (sums) to_h2<FMT>(packed[k], z[0], z[1]);
        }
        if (sums) {
          bound(2 * k, z[0]);
          bound((2 * k + 1) % (VEC / 2), z[1]);
        }
      }
      *reinterpret_cast<uint2*>(dst + (row + i * RP) * HD) = make_uint2(packed[0], packed[1]);
    }
  } else if (clean) {
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (FULL || row + i * RP < r1) put_row(std::true_type{}, row + i * RP, raw[i]);
  } else {
#pragma unroll 1
    for (int r = row; r < r1; r += RP) put_row(std::false_type{}, r, load_row(r));
  }
  if (!sums) return;
#pragma unroll
  for (int o = TR; o < 32; o <<= 1)
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) {
      lo[j] = __hmin2(lo[j], __shfl_xor_sync(0xffffffffu, lo[j], o));
      hi[j] = __hmax2(hi[j], __shfl_xor_sync(0xffffffffu, hi[j], o));
    }
  if (lane < TR) {
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) {
      const int ch = VEC * tr + 4 * (j / 2) + (j & 1) * (3 - PS);
      const float2 l = __half22float2(lo[j]), u = __half22float2(hi[j]);
      sh.smin[warp][ch] = l.x - offset;
      sh.smin[warp][ch + PS] = l.y - offset;
      sh.smax[warp][ch] = u.x - offset;
      sh.smax[warp][ch + PS] = u.y - offset;
    }
  }
  __syncthreads();
  if (threadIdx.x >= HD) return;
  float l = sh.smin[0][threadIdx.x], u = sh.smax[0][threadIdx.x];
#pragma unroll
  for (int i = 1; i < W; ++i) {
    l = fminf(l, sh.smin[i][threadIdx.x]);
    u = fmaxf(u, sh.smax[i][threadIdx.x]);
  }
  if (FMT == NT_KV8_E4M3) {  // whole numbers of 4 scale steps, rounded outwards: still bounds
    l = floorf(l * 0.25f);
    u = ceilf(u * 0.25f);
  }
  const int64_t at = (int64_t(h) * a.nb + blk) * HD + threadIdx.x;
  a.kmin[at] = int8_t(__float2int_rn(l));
  a.kmax[at] = int8_t(__float2int_rn(u));
}

template <int FMT, int HD, typename T>
__global__ void __launch_bounds__(kAppendThreads) kv8_append_kernel(const AppendArgs a) {
  __shared__ AppendShared sh;
  pdl_wait();
  pdl_trigger();
  const int64_t pos = a.pos_dev ? *a.pos_dev : a.pos;
  if (pos < 0 || pos > a.kv_stride - a.n) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) flag_error(a.err, kErrPosRange);
    return;
  }
  const int64_t blk = pos / kB + blockIdx.x, p0 = blk * kB;
  const int r0 = int(max(pos, p0) - p0);
  const int64_t end = min(pos + a.n, p0 + kB) - p0;
  if (end <= r0) return;
  if (r0 == 0 && end == kB)
    append_block<FMT, HD, T, true>(a, sh, pos, blk, 0, kB);
  else
    append_block<FMT, HD, T, false>(a, sh, pos, blk, r0, int(end));
}

// ---- read back -----------------------------------------------------------------
constexpr int kReadThreads = 256;
constexpr int kReadUnroll = 4;

struct ReadArgs {
  const uint8_t* src[2];
  const float* scale[2];
  void* dst[2];  // either may be null
  int64_t pos, n, kv_stride, nb, head_stride;
};

// Each thread turns VEC bytes into 16 bytes of values, kReadUnroll times.  Bound by
// HBM: 131,072 positions of 8 x 128 E4M3 to F16, 116 us (805 MB at 6.9 TB/s).
template <int FMT, int HD, typename T>
__global__ void __launch_bounds__(kReadThreads) kv8_read_kernel(const ReadArgs a) {
  constexpr int VEC = 16 / int(sizeof(T));
  pdl_wait();
  pdl_trigger();
  const int h = blockIdx.y, w = blockIdx.z;
  void* out = w ? a.dst[1] : a.dst[0];
  if (!out) return;
  const uint8_t* src = (w ? a.src[1] : a.src[0]) + (int64_t(h) * a.kv_stride + a.pos) * HD;
  const float* scale = (w ? a.scale[1] : a.scale[0]) + int64_t(h) * a.nb;
  T* dst = static_cast<T*>(out) + int64_t(h) * a.head_stride;
  const int64_t units = a.n * (HD / VEC);
  const int64_t u0 = int64_t(blockIdx.x) * (kReadThreads * kReadUnroll) + threadIdx.x;
  uint32_t x[kReadUnroll][VEC / 4];
  float t[kReadUnroll];
#pragma unroll
  for (int i = 0; i < kReadUnroll; ++i) {
    const int64_t u = u0 + i * kReadThreads;
    if (u >= units) continue;
    if (VEC == 4) {
      x[i][0] = *reinterpret_cast<const uint32_t*>(src + u * VEC);
    } else {
      const uint2 r = *reinterpret_cast<const uint2*>(src + u * VEC);
      x[i][0] = r.x;
      x[i][VEC / 4 - 1] = r.y;
    }
    t[i] = scale[(a.pos + u / (HD / VEC)) / kB];
  }
#pragma unroll
  for (int i = 0; i < kReadUnroll; ++i) {
    const int64_t u = u0 + i * kReadThreads;
    if (u >= units) continue;
    const float4 f = unpack8<FMT>(x[i][0]);
    uint4 o;
    if (VEC == 4) {
      o = make_uint4(__float_as_uint(f.x * t[i]), __float_as_uint(f.y * t[i]), __float_as_uint(f.z * t[i]),
                     __float_as_uint(f.w * t[i]));
    } else {
      const float4 g = unpack8<FMT>(x[i][VEC / 4 - 1]);
      const __half2 h0 = __floats2half2_rn(f.x * t[i], f.y * t[i]), h1 = __floats2half2_rn(f.z * t[i], f.w * t[i]);
      const __half2 h2 = __floats2half2_rn(g.x * t[i], g.y * t[i]), h3 = __floats2half2_rn(g.z * t[i], g.w * t[i]);
      o = make_uint4(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1),
                     *reinterpret_cast<const uint32_t*>(&h2), *reinterpret_cast<const uint32_t*>(&h3));
    }
    *reinterpret_cast<uint4*>(dst + u * VEC) = o;
  }
}

// ---- attention -----------------------------------------------------------------
// Scores and outputs on the tensor cores (mma.sync m16n8k16, f16 products, fp32
// sums) with fp32-level operands.  The cached values are exact in f16.  A row of
// q (and of the probabilities) is split into hi = f16(x), lo = f16(x - hi), which
// carries 22 bits; the M = 16 rows of an MMA are the hi parts of 8 rows and, 8
// below, their lo parts, so the two halves of a product meet in one thread:
// accumulators c0 + c2 and c1 + c3.  The parts of a probability times its V scale stop
// at f16's smallest step: 2^-33 of the largest such product is what is lost of each position.
//
// Fragments come without a transpose: MMA k and n indices are ours to name.  Lane
// (n = lane / 4, c = lane % 4), a step of 16 U tokens:
//  - Q K^T: B column n of n-tile u (0 .. 2 U - 1) is token 4 U (n / 2) + 2 u + n % 2;
//    the lane reads bytes 16 c .. 16 c + 15 (+ 64 for the upper half) of that row, and
//    word w of a 16-byte piece is its k-slots of k-step w.
//  - the scores of row n land in lane (n, c) for tokens 4 U c .. 4 U c + 4 U - 1;
//  - P V: those tokens are the lane's k-slots; it reads bytes n HD/8 .. + HD/8 - 1 of
//    their V rows, and byte i of them is B column n of n-tile i, i.e. output channel
//    n HD/8 + i.
//
// Each warp walks its own steps: one bulk copy brings a step's K and one its V.  The
// next step's K is copied while the warp works on the probabilities and V, the next V
// while it works on K; no barrier joins the warps.
//
// Long sequences are bound by HBM (32 q heads over 8 of 128 channels, I8: 1,000,003
// positions 290 us, 7.06 TB/s; 131,071 47.3 us, of which about 9 are the ramp, the
// tail and the combine); short ones by the latency of launch, copy, step and merge
// (1088 positions 5.4 us); several queries by the chain of a 16-row step (8 queries of
// 32 heads, 16,381 positions 24.3 us, tensor pipe at 40%).  Eight warps of 128
// registers and two CTAs an SM: fewer registers spill, a second buffer per warp
// changes nothing.
constexpr int kAttnWarps = 8;
constexpr float kPTop = 8.f, kLUnit = 0x1p-13f;                   // see the softmax
constexpr float kSlack = 6.f, kFar = 90.f, kMid = (kFar - kSlack) / 2, kLift = 110.f;
constexpr float kLowest = -3.402823466e38f;  // the merges' maximum of nothing: 2^(-inf - kLowest) is 0
constexpr int kMaxCluster = 16;

struct AttnKv8Args {
  const float* q;
  const uint8_t *k, *v;
  const float *ks, *vs;
  float* out;
  float* part;         // [query * n_qh + head][S][HD], unnormalised outputs in fragment order
  float2* ml;          // [query * n_qh + head][S]: (max, sum)
  const int32_t* idx;  // sparse: [query][n_kvh][n_sel]
  int n_sel;
  int n_qh, n_kvh, G, nq, S;
  int chunks;          // row chunks of 8 R rows: per KV head (dense), per query and KV head (sparse)
  int inv_g;           // ceil(2^16 / G): r / G = r inv_g >> 16 for the rows (at most 256) of a call
  int64_t n_pos, kv_stride, nb;
  const int64_t* pos_dev;
  unsigned* err;
  int cluster;         // the splits of a head are one cluster and join in shared memory
  int stall;           // test hook: issue no bulk copies; the waits give up after kStallSpin tries
};

// positions query 0 sees, held to the cache
__device__ __forceinline__ int64_t seen_positions(const AttnKv8Args& a) {
  int64_t n = a.pos_dev ? *a.pos_dev + 1 : a.n_pos;
  if (n < 0 || n > a.kv_stride - (a.nq - 1)) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) flag_error(a.err, kErrPosRange);
    n = n < 0 ? 0 : a.kv_stride - (a.nq - 1);
  }
  return n;
}

// steps per CTA for `steps` warp steps over S splits: both launches compute it, so an
// unused split is never read
__device__ __forceinline__ int split_steps(int steps, int S) {
  const int even = (steps + S - 1) / S;
  return even < kAttnWarps ? kAttnWarps : even;
}

__device__ __forceinline__ void mma16816(float c[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// the same from zero
__device__ __forceinline__ void mma16816_zero(float c[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(0.f));
}

// whether phase `parity` of an mbarrier has completed, without waiting
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// a + b on two floats at once
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 z, x, y;\n\t"
      "mov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\t"
      "mov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// hi and lo f16 parts of two values
__device__ __forceinline__ void split_h2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

// two floats into the shared memory of CTA `rank` of this cluster, at this CTA's address `at`
__device__ __forceinline__ void st_cluster(uint32_t at, int rank, float2 v) {
  uint32_t to;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(at), "r"(rank));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(v.x), "f"(v.y) : "memory");
}

// shared memory: q fragments [R][HD / 16][32] x 16, (max, sum) [2][warps][8 R], what
// the other CTAs of a cluster send, each warp's room for one step's K and V; at the
// end, in its place, the warps' outputs [warps][R][HD / 8][32] x 8
template <int HD, int R, int U>
struct AttnKv8Smem {
  static constexpr size_t q = 0;
  static constexpr size_t ml = q + size_t(R) * (HD / 16) * 512;
  static constexpr size_t push = ml + size_t(2) * kAttnWarps * 8 * R * 4;           // from the cluster: outputs
  static constexpr size_t push_ml = push + size_t(R) * (HD / 8) * 256;               // and (max, sum) [splits][8 R]
  static constexpr size_t ring = push_ml + size_t(kMaxCluster) * 8 * R * 8;
  static constexpr size_t stage = size_t(16 * U) * HD * 2;           // K, then V
  static constexpr size_t outs = size_t(R) * (HD / 8) * 256;         // one warp's outputs
  static constexpr size_t bytes = ring + kAttnWarps * (stage > outs ? stage : outs);
};

template <int FMT, int HD, int R, int U, bool SPARSE>
__global__ void __launch_bounds__(kAttnWarps * 32, R == 1 ? 2 : 1) attn_kv8_kernel(const AttnKv8Args a) {
  using L = AttnKv8Smem<HD, R, U>;
  constexpr int kStep = 16 * U;      // tokens per warp step
  constexpr int KS = HD / 16;        // k-steps of Q K^T
  constexpr int NT = HD / 8;         // n-tiles of P V
  constexpr int KP = HD / 64;        // 16-byte pieces of a K row per lane
  constexpr int VW = HD / 32;        // words of a V row per lane
  constexpr int ROWS = 8 * R;
  constexpr int CH = U == 1 ? 2 : 1; // accumulators per score tile: at least four chains of MMAs
  extern __shared__ __align__(16) uint8_t sm8[];
  uint4* qa = reinterpret_cast<uint4*>(sm8 + L::q);
  __shared__ float s_amax[R * KS][8];  // by k-step and row
  __shared__ __align__(8) uint64_t bars[kAttnWarps][2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = lane >> 2, c = lane & 3;
  // what needs no input runs before the wait for the kernel in front
  if (a.cluster) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // our shared memory may be written
  const uint8_t* sk = sm8 + L::ring + size_t(warp) * L::stage;  // this warp's K rows of a step
  const uint8_t* sv = sk + kStep * HD;                           // and its V rows
  const uint32_t bar = smem_u32(&bars[warp][0]);                 // K, V
  const uint64_t pol = policy_evict_first();
  if (lane == 0) {
    mbar_init(bar, 1);
    mbar_init(bar + 8, 1);
    fence_barrier_init();
  }
  __syncwarp();
  pdl_wait();
  pdl_trigger();
  const int g = blockIdx.x, s = blockIdx.y;
  const int qi0 = SPARSE ? blockIdx.z / a.chunks : 0;
  const int row0 = (SPARSE ? blockIdx.z % a.chunks : blockIdx.z) * ROWS;
  const int rows = min(ROWS, (SPARSE ? a.G : a.nq * a.G) - row0);
  const int n_pos = int(seen_positions(a));  // positions fit 30 bits
  // row r of this chunk: query and head
  const auto query_of = [&](int r) { return SPARSE ? qi0 : ((row0 + r) * a.inv_g) >> 16; };
  const auto vec_of = [&](int r) {
    const int qi = query_of(r);
    return int64_t(qi) * a.n_qh + g * a.G + (SPARSE ? row0 + r : row0 + r - qi * a.G);
  };
  const int tokens = n_pos + query_of(rows - 1);  // the last row sees the most
  const int steps = SPARSE ? a.n_sel * (kB / kStep) : (tokens + kStep - 1) / kStep;
  const int per = split_steps(steps, a.S);
  const int st0 = s * per, st1 = min(steps, st0 + per);
  if (!a.cluster && st0 >= st1 && s > 0) return;

  // this thread's q values, requested before the copies of K and V fill the memory system
  constexpr int QI = (R * KS + kAttnWarps - 1) / kAttnWarps;  // fragments per thread
  float4 qv[QI];
#pragma unroll
  for (int i = 0; i < QI; ++i) {
    const int f = warp + i * kAttnWarps, j = f % KS, r = f / KS * 8 + n;
    qv[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (f < R * KS && r < rows) qv[i] = load4(a.q + vec_of(r) * HD + 64 * (j >> 2) + 16 * c + 4 * (j & 3));
  }
  const uint8_t* kg = a.k + int64_t(g) * a.kv_stride * HD;
  const uint8_t* vg = a.v + int64_t(g) * a.kv_stride * HD;
  const float* ksg = a.ks + int64_t(g) * a.nb;
  const float* vsg = a.vs + int64_t(g) * a.nb;
  const int32_t* list = SPARSE ? a.idx + (int64_t(qi0) * a.n_kvh + g) * a.n_sel : nullptr;
  const int blocks_seen = (tokens + kB - 1) / kB;

  // first token of step st (tokens: nothing to do)
  const auto step_token = [&](int st) {
    if (!SPARSE) return st < st1 ? st * kStep : tokens;
    if (st >= st1) return tokens;
    const int b = __ldcg(list + st / (kB / kStep));
    return b < 0 || b >= blocks_seen ? tokens : min(tokens, b * kB + st % (kB / kStep) * kStep);
  };
  // the copy of one step's K (which 0) or V (1), rows below `tokens` only
  const auto copy = [&](const uint8_t* from, int which, int t0) {
    if (t0 >= tokens || lane != 0) return;
    const uint32_t bytes = min(kStep, tokens - t0) * HD, on = bar + 8 * which;
    mbar_arrive_expect_tx(on, bytes);
    if (!a.stall) bulk_g2s(smem_u32(which ? sv : sk), from + int64_t(t0) * HD, bytes, on, pol);
  };
  int st = st0 + warp;
  int t0 = step_token(st), t1 = step_token(st + kAttnWarps);  // this step's first token, the next one's
  uint32_t phase = 0;
  const auto wait = [&](int which) {
    const uint32_t on = bar + 8 * which;
    if (mbar_test(on, phase)) return true;
    const int cap = a.stall ? kStallSpin : kMaxSpin;
    const bool ok = __all_sync(0xffffffffu, mbar_wait(on, phase, cap));
    if (!ok) {  // flag it, wait (bounded) for the copies still in flight, go on to the merge
      if (lane == 0) flag_error(a.err, kErrWaitTimeout);
      mbar_wait(on, phase, cap);
      if (which == 0)
        mbar_wait(bar + 8, phase, cap);  // this step's V
      else if (t1 < tokens)
        mbar_wait(bar, phase ^ 1, cap);  // the next step's K
    }
    return ok;
  };
  const auto scales = [&](int t0) {
    return t0 < tokens ? make_float2(__ldcg(ksg + t0 / kB), __ldcg(vsg + t0 / kB)) : make_float2(0.f, 0.f);
  };
  copy(kg, 0, t0);
  copy(vg, 1, t0);
  float2 kvs = scales(t0);

  // q: each row scaled by a power of two to amax in [2^13, 2^14), split, laid out as
  // fragments: warp w holds k-step w % KS of every row
#pragma unroll
  for (int i = 0; i < QI; ++i) {
    const int f = warp + i * kAttnWarps;
    if (f >= R * KS) continue;
    float x = fmaxf(fmaxf(fabsf(qv[i].x), fabsf(qv[i].y)), fmaxf(fabsf(qv[i].z), fabsf(qv[i].w)));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
    if (c == 0) s_amax[f][n] = x;
  }
  __syncthreads();
  int qe[R];  // q of row 8 t + n times 2^qe
#pragma unroll
  for (int t = 0; t < R; ++t) {
    float x = s_amax[t * KS][n];
#pragma unroll
    for (int j = 1; j < KS; ++j) x = fmaxf(x, s_amax[t * KS + j][n]);
    qe[t] = min(100, 140 - int(__float_as_uint(x) >> 23));
  }
#pragma unroll
  for (int i = 0; i < QI; ++i) {
    const int f = warp + i * kAttnWarps;
    if (f >= R * KS) continue;
    const float sc = __uint_as_float(uint32_t((R == 1 || f < KS ? qe[0] : qe[R - 1]) + 127) << 23);
    const float4 x = qv[i];
    uint4 y;
    split_h2(x.x * sc, (kPairStep<FMT> == 2 ? x.z : x.y) * sc, y.x, y.y);
    split_h2((kPairStep<FMT> == 2 ? x.y : x.z) * sc, x.w * sc, y.z, y.w);
    qa[f * 32 + lane] = y;
  }
  __syncthreads();
  float rscale[R];      // scores to the base-2 exponent
  int limit[R];         // positions row n sees
  float m[R], l[R];
  float2 o[R][NT];      // row n, channels 2 c (HD / 8) + i and (2 c + 1) (HD / 8) + i
#pragma unroll
  for (int t = 0; t < R; ++t) {
    const int r = t * 8 + n;
    // log2(e) / sqrt(HD)
    rscale[t] = __uint_as_float(uint32_t(127 - qe[t]) << 23) * (1.44269504088896f * rsqrtf(float(HD)));
    limit[t] = r < rows ? n_pos + query_of(r) : 0;
    m[t] = -INFINITY;
    l[t] = 0.f;
#pragma unroll
    for (int i = 0; i < NT; ++i) o[t][i] = make_float2(0.f, 0.f);
  }
  const int fewest = SPARSE ? tokens : n_pos + query_of(0);  // positions every row sees
  for (; st < st1; st += kAttnWarps) {
    const int t2 = step_token(st + 2 * kAttnWarps);
    const float2 kvs1 = scales(t1);
    // ---- scores
    float sc[R][2 * U][CH][4];
    if (t0 < tokens) {
      if (!wait(0)) break;
#pragma unroll
      for (int t = 0; t < R; ++t)
#pragma unroll
        for (int u = 0; u < 2 * U; ++u)
#pragma unroll
          for (int e = 0; e < CH; ++e) sc[t][u][e][0] = sc[t][u][e][1] = sc[t][u][e][2] = sc[t][u][e][3] = 0.f;
#pragma unroll
      for (int p = 0; p < KP; ++p) {
        uint4 kw[2 * U];
#pragma unroll
        for (int u = 0; u < 2 * U; ++u)
          kw[u] = *reinterpret_cast<const uint4*>(sk + (4 * U * (n >> 1) + 2 * u + (n & 1)) * HD + 64 * p + 16 * c);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint4 af[R];
#pragma unroll
          for (int t = 0; t < R; ++t) af[t] = qa[(t * KS + 4 * p + j) * 32 + lane];
#pragma unroll
          for (int u = 0; u < 2 * U; ++u) {
            uint32_t b0, b1;
            to_h2<FMT>(j == 0 ? kw[u].x : j == 1 ? kw[u].y : j == 2 ? kw[u].z : kw[u].w, b0, b1);
#pragma unroll
            for (int t = 0; t < R; ++t) mma16816(sc[t][u][j % CH], af[t], b0, b1);
          }
        }
      }
    }
    __syncwarp();  // this step's K is in registers and used
    copy(kg, 0, t1);
    uint4 pf[R][U];
    if (t0 < tokens) {
      // ---- online softmax.  The f16 operand of P V is a probability times the block's
      // V scale vs = vn 2^lv, 1 <= vn < 2, so the running m follows s + lv and the operand
      // is p vn with p = 2^(s + lv - m + kPTop).  m is a whole number (base is exact) and is
      // left behind by up to kSlack before the accumulators are rescaled to a new one:
      // the operand then stays below 2^(kPTop + kSlack + 1), the largest f16 exponent, and a
      // warp rescales once or twice in a sequence instead of at every new maximum.  The sum
      // l takes p 2^-lv in units of 2^13, which keep it within fp32 for every scale that
      // the cache can hold (2^26 weights of the largest exponent at 2^-100, one at 2^122).
      // Where s + lv is kFar below m (an all-zero block beside large ones) the outputs
      // gain nothing, and l takes the exponentials lifted by kLift, out of reach of the
      // underflow.  Registers hold m - kMid: one comparison finds both cases.
      const float vs = kvs.y;
      const uint32_t ve = min(max(__float_as_uint(vs) >> 23, 27u), 249u);  // 2^-100 .. 2^122
      const float lv = __uint_as_float(0x4B000000u + ve) - (8388608.f + 127.f);
      const float il = __uint_as_float((254u - ve) << 23), vn = vs * il, lu = il * kLUnit;
#pragma unroll
      for (int t = 0; t < R; ++t) {
        const float f = rscale[t] * kvs.x;
        float p[4 * U];
#pragma unroll
        for (int x = 0; x < 2 * U; ++x) {
          const float* v = sc[t][x][0];
          float2 y = add2(make_float2(v[0], v[1]), make_float2(v[2], v[3]));
          if (CH == 2) {
            const float* z = sc[t][x][CH - 1];
            y = add2(y, add2(make_float2(z[0], z[1]), make_float2(z[2], z[3])));
          }
          y = mul2(y, make_float2(f, f));
          p[2 * x] = y.x;
          p[2 * x + 1] = y.y;
        }
        if (t0 + kStep > fewest) {
          const int left = limit[t] - t0 - 4 * U * c;
#pragma unroll
          for (int x = 0; x < 4 * U; ++x) p[x] = x < left ? p[x] : -INFINITY;
        }
        float mx = p[0];
#pragma unroll
        for (int x = 1; x < 4 * U; ++x) mx = fmaxf(mx, p[x]);
        float ml = m[t] - lv;
        if (__any_sync(0xffffffffu, fabsf(mx - ml) > kMid + kSlack)) {
          float mn = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 2)) + lv;
          mn = fmaxf(m[t], floorf(mn) - kMid);
          const float down = m[t] == -INFINITY ? -INFINITY : m[t] - mn;
          const float corr = ex2(fmaxf(down, -kLift));
          l[t] = l[t] * corr * ex2(fminf(down + kLift, 0.f));  // in two steps: it may be large
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            o[t][i].x *= corr;
            o[t][i].y *= corr;
          }
          m[t] = mn;
          ml = mn - lv;
          if (ml - mx > kMid + kSlack) {
            const float lifted = (kPTop - kMid + kLift) - ml;
            float2 far = make_float2(0.f, 0.f);
#pragma unroll
            for (int x = 0; x < 4 * U; x += 2) {
              const float2 e = add2(make_float2(p[x], p[x + 1]), make_float2(lifted, lifted));
              far = add2(far, make_float2(ex2(e.x), ex2(e.y)));
              p[x] = p[x + 1] = -INFINITY;
            }
            l[t] = fmaf((far.x + far.y) * lu, ex2(-kLift), l[t]);
          }
        }
        const float base = m[t] == -INFINITY ? 0.f : (kPTop - kMid) - ml;
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float2 y[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            y[x] = add2(make_float2(p[4 * u + 2 * x], p[4 * u + 2 * x + 1]), make_float2(base, base));
            y[x] = make_float2(ex2(y[x].x), ex2(y[x].y));
            sum = add2(sum, y[x]);
            y[x] = mul2(y[x], make_float2(vn, vn));
          }
          split_h2(y[0].x, y[0].y, pf[t][u].x, pf[t][u].y);
          split_h2(y[1].x, y[1].y, pf[t][u].z, pf[t][u].w);
        }
        l[t] = fmaf(sum.x + sum.y, lu, l[t]);
      }
    }
    if (t0 < tokens) {
      if (!wait(1)) break;
      phase ^= 1;
      // ---- P V: words of two tokens interleaved into (token, token + 1) pairs per
      // channel.  Each step's products start from zero and are added to the output
      // in fp32: the tensor cores round their sums towards zero, and a bias of one
      // such rounding per step would grow with the length (1,000,003 positions:
      // error 4.3e-6 with one running accumulator).
#pragma unroll
      for (int w = 0; w < VW; w += 2) {
        uint32_t vw[4 * U][2];
#pragma unroll
        for (int x = 0; x < 4 * U; ++x) {
          const uint2 r = *reinterpret_cast<const uint2*>(sv + (4 * U * c + x) * HD + n * (HD / 8) + 4 * w);
          vw[x][0] = r.x;
          vw[x][1] = r.y;
        }
        if (t0 + kStep > tokens) {  // rows past the end were not copied: their bytes must not meet the zeros of p
#pragma unroll
          for (int x = 0; x < 4 * U; ++x)
            if (t0 + 4 * U * c + x >= tokens) vw[x][0] = vw[x][1] = 0u;
        }
#pragma unroll
        for (int h = 0; h < 4; ++h) {  // half (h % 2) of word h / 2: two channels
          float acc[R][2][4];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            uint32_t b0[2], b1[2];
            to_h2<FMT>(interleave8<FMT>(vw[4 * u][h >> 1], vw[4 * u + 1][h >> 1], h & 1), b0[0], b0[1]);
            to_h2<FMT>(interleave8<FMT>(vw[4 * u + 2][h >> 1], vw[4 * u + 3][h >> 1], h & 1), b1[0], b1[1]);
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int t = 0; t < R; ++t) {
                if (u == 0)
                  mma16816_zero(acc[t][e], pf[t][u], b0[e], b1[e]);
                else
                  mma16816(acc[t][e], pf[t][u], b0[e], b1[e]);
              }
          }
#pragma unroll
          for (int t = 0; t < R; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float* x = acc[t][e];
              float2& y = o[t][4 * w + 2 * h + e];
              y = add2(y, add2(make_float2(x[0], x[1]), make_float2(x[2], x[3])));
            }
        }
      }
    }
    __syncwarp();  // and its V
    copy(vg, 1, t1);
    t0 = t1;
    t1 = t2;
    kvs = kvs1;
  }

  // ---- merge the warps
  __syncthreads();  // every warp is done with its K and V
  float* mm = reinterpret_cast<float*>(sm8 + L::ml);  // [warps][ROWS] max
  float* mll = mm + kAttnWarps * ROWS;                // [warps][ROWS] sum
  float2* outs = reinterpret_cast<float2*>(sm8 + L::ring);
#pragma unroll
  for (int t = 0; t < R; ++t) {
    l[t] += __shfl_xor_sync(0xffffffffu, l[t], 1);
    l[t] += __shfl_xor_sync(0xffffffffu, l[t], 2);
    if (!(l[t] >= 0x1p-60f && l[t] <= 0x1p20f)) {
      // (very small or very large V scales) m takes over the exponent of l, down to -60, and
      // l and o lose it: in the merges the weights 2^(m - M) then underflow only where l does
      // not matter either
      const uint32_t k = max(__float_as_uint(l[t]) & 0x7F800000u, 67u << 23);
      const float down = __uint_as_float((254u << 23) - k);
      l[t] *= down;
      m[t] += float(int(k >> 23) - 127);
#pragma unroll
      for (int i = 0; i < NT; ++i) o[t][i] = mul2(o[t][i], make_float2(down, down));
    }
    if (c == 0) {
      mm[warp * ROWS + t * 8 + n] = m[t];
      mll[warp * ROWS + t * 8 + n] = l[t];
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) outs[(size_t(warp) * R * NT + t * NT + i) * 32 + lane] = o[t][i];
  }
  __syncthreads();
  const bool whole = a.S == 1 || (per >= steps && !a.cluster);  // one split: the output itself
  // of the R NT fragment tiles, `own` belong to each CTA of a cluster
  const int own = a.cluster ? R * NT / a.S : 1;
  const uint32_t push = smem_u32(sm8 + L::push), push_ml = smem_u32(sm8 + L::push_ml);
  if (a.cluster) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
#pragma unroll
  for (int t = 0; t < R; ++t) {
    const int r = t * 8 + n;
    if (r >= rows && !a.cluster) continue;
    float f[kAttnWarps], M = kLowest, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
      f[w] = mm[w * ROWS + r];
      M = fmaxf(M, f[w]);
    }
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
      f[w] = ex2(f[w] - M);
      sum = fmaf(mll[w * ROWS + r], f[w], sum);
    }
    const int64_t vec = vec_of(r);
    const float inv = !whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int i = warp; i < NT; i += kAttnWarps) {
      float2 acc = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kAttnWarps; ++w) {
        const float2 x = outs[(size_t(w) * R * NT + t * NT + i) * 32 + lane];
        acc.x = fmaf(x.x, f[w], acc.x);
        acc.y = fmaf(x.y, f[w], acc.y);
      }
      if (a.cluster) {
        const int tile = t * NT + i;
        st_cluster(push + ((s * own + tile % own) * 32 + lane) * 8, tile / own, acc);
      } else if (whole) {
        a.out[vec * HD + (HD / 8) * (2 * c) + i] = acc.x * kLUnit * inv;
        a.out[vec * HD + (HD / 8) * (2 * c + 1) + i] = acc.y * kLUnit * inv;
      } else {
        *reinterpret_cast<float2*>(a.part + (vec * a.S + s) * HD + (i * 4 + c) * 2) = acc;
      }
    }
    if (a.cluster) {
      for (int d = c + 4 * warp; d < a.S; d += 4 * kAttnWarps)
        st_cluster(push_ml + (s * ROWS + r) * 8, d, make_float2(M, sum));
    } else if (!whole && warp == 0 && c == 0) {
      a.ml[vec * a.S + s] = make_float2(M, sum);
    }
  }
  if (!a.cluster) return;
  // ---- merge the cluster's splits: this CTA's tiles of every split have arrived
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  const float2* pushed = reinterpret_cast<const float2*>(sm8 + L::push);
  const float2* pushed_ml = reinterpret_cast<const float2*>(sm8 + L::push_ml);
  for (int k = warp; k < own; k += kAttnWarps) {
    const int tile = s * own + k, r = tile / NT * 8 + n, i = tile % NT;
    if (r >= rows) continue;
    float2 y[kMaxCluster], z[kMaxCluster];  // all in flight together
    float M = kLowest, sum = 0.f;
#pragma unroll
    for (int x = 0; x < kMaxCluster; ++x) {
      y[x] = x < a.S ? pushed_ml[x * ROWS + r] : make_float2(-INFINITY, 0.f);
      z[x] = x < a.S ? pushed[(x * own + k) * 32 + lane] : make_float2(0.f, 0.f);
    }
#pragma unroll
    for (int x = 0; x < kMaxCluster; ++x) M = fmaxf(M, y[x].x);
    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
    for (int x = 0; x < kMaxCluster; ++x) {
      const float f = ex2(y[x].x - M);
      sum = fmaf(y[x].y, f, sum);
      acc.x = fmaf(z[x].x, f, acc.x);
      acc.y = fmaf(z[x].y, f, acc.y);
    }
    const int64_t vec = vec_of(r);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    a.out[vec * HD + (HD / 8) * (2 * c) + i] = acc.x * kLUnit * inv;
    a.out[vec * HD + (HD / 8) * (2 * c + 1) + i] = acc.y * kLUnit * inv;
  }
}

// the splits' partials of one row into the output: one thread per channel
constexpr int kMaxSplits = 512;
template <int HD, bool SPARSE>
__global__ void __launch_bounds__(HD) attn_kv8_combine_kernel(const AttnKv8Args a, int rows_per_chunk, int step) {
  __shared__ float wts[kMaxSplits];
  __shared__ float red[HD / 32];
  pdl_wait();
  pdl_trigger();
  const int qh = blockIdx.x, qi = blockIdx.y, d = threadIdx.x, lane = d & 31, warp = d >> 5;
  const int n_pos = int(seen_positions(a));
  int tokens = n_pos + qi;
  if (!SPARSE) {  // the chunk of this row ends at its last row's query
    const int r = qi * a.G + qh % a.G, last = min(a.nq * a.G, (r / rows_per_chunk + 1) * rows_per_chunk) - 1;
    tokens = n_pos + last / a.G;
  }
  const int steps = SPARSE ? a.n_sel * (kB / step) : (tokens + step - 1) / step;
  const int per = split_steps(steps, a.S);
  if (per >= steps) return;
  const int used = (steps + per - 1) / per;
  const int64_t vec = int64_t(qi) * a.n_qh + qh;
  const float2* ml = a.ml + vec * a.S;
  const float* part = a.part + vec * a.S * HD + d;
  // this channel of the first 16 splits and the splits' (max, sum), all in flight together
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = i < used ? __ldcg(part + int64_t(i) * HD) : 0.f;
  float2 x[kMaxSplits / HD];
  float M = kLowest;
#pragma unroll
  for (int i = 0; i < kMaxSplits / HD; ++i) {
    x[i] = d + i * HD < used ? __ldcg(ml + d + i * HD) : make_float2(-INFINITY, 0.f);
    M = fmaxf(M, x[i].x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) red[warp] = M;
  __syncthreads();
  M = red[0];
#pragma unroll
  for (int w = 1; w < HD / 32; ++w) M = fmaxf(M, red[w]);
  __syncthreads();
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxSplits / HD; ++i) {
    const float f = ex2(x[i].x - M);
    if (d + i * HD < used) wts[d + i * HD] = f;
    sum = fmaf(x[i].y, f, sum);
  }
  sum = warp_sum(sum);
  if (lane == 0) red[warp] = sum;
  __syncthreads();
  sum = red[0];
#pragma unroll
  for (int w = 1; w < HD / 32; ++w) sum += red[w];
  float acc = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < used) acc = fmaf(v[i], wts[i], acc);
  for (int i0 = 16; i0 < used; i0 += 16) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = i0 + i < used ? __ldcg(part + int64_t(i0 + i) * HD) : 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i0 + i < used) acc = fmaf(v[i], wts[i0 + i], acc);
  }
  // fragment order (n-tile, lane pair, column) -> channel
  const int ch = (HD / 8) * (d & 7) + (d >> 3);
  a.out[vec * HD + ch] = acc * kLUnit * (sum == 0.f ? 0.f : 1.f / sum);
}

using AttnKv8Kernel = void (*)(AttnKv8Args);
struct AttnKv8Variant {
  AttnKv8Kernel kernel;
  size_t smem;
};
template <int FMT, int HD, bool SPARSE>
AttnKv8Variant attn_kv8_pick(int R, int U) {
  if (R == 1 && U == 1) return {attn_kv8_kernel<FMT, HD, 1, 1, SPARSE>, AttnKv8Smem<HD, 1, 1>::bytes};
  if (R == 1) return {attn_kv8_kernel<FMT, HD, 1, 2, SPARSE>, AttnKv8Smem<HD, 1, 2>::bytes};
  return {attn_kv8_kernel<FMT, HD, 2, 2, SPARSE>, AttnKv8Smem<HD, 2, 2>::bytes};
}
template <bool SPARSE>
AttnKv8Variant attn_kv8_for(int fmt, int hd, int R, int U) {
  if (fmt == NT_KV8_I8)
    return hd == 128 ? attn_kv8_pick<NT_KV8_I8, 128, SPARSE>(R, U) : attn_kv8_pick<NT_KV8_I8, 64, SPARSE>(R, U);
  return hd == 128 ? attn_kv8_pick<NT_KV8_E4M3, 128, SPARSE>(R, U) : attn_kv8_pick<NT_KV8_E4M3, 64, SPARSE>(R, U);
}

// ---- block selection -----------------------------------------------------------
// The largest score that any key within a block's channel bounds could have with
// head h is sum_d max(q_d kmin_d, q_d kmax_d) = sum_d max(q_d, 0) kmax_d +
// min(q_d, 0) kmin_d: linear in the two halves of q, so the group's heads are
// added first and a block costs 2 HD products whatever the group size.  With q as
// 12-bit integers every sum is a whole number below 2^31: the scores, and with
// them the choice, do not depend on the order of additions.
constexpr int kSelWide = 1024, kSelNarrow = 256;  // threads of a selection
constexpr int kSelNarrowBlocks = kSelNarrow;      // most blocks of the narrow one: one a thread
// most CTAs of a selection's cluster, an SM each: larger clusters of 8 heads do not all
// fit on the GPU at once (15,626 blocks: 8 CTAs 17.8 us, 12 16.5, 14 22.3, 16 21.1).  Of
// fewer heads they do, and 12 is not the best (15,626 blocks of 4 heads: 8 CTAs 17.0 us,
// 12 15.5, 16 14.3; of one head 15.0, 13.7, 12.8).
constexpr int kSelCluster = 12;

struct SelectArgs {
  const float* q;
  const int8_t *kmin, *kmax;
  const float* ks;
  uint32_t* keys;    // [query][n_kvh][nb]: scratch, when the keys of a head do not fit in shared memory
  int32_t* idx;      // [query][n_kvh][n_sel]
  int n_qh, n_kvh, G, nq, n_sel, n_first, n_last;
  int64_t n_pos, kv_stride, nb;
  const int64_t* pos_dev;
  unsigned* err;
};

__device__ __forceinline__ int64_t seen_positions(const SelectArgs& a) {
  AttnKv8Args t{};
  t.pos_dev = a.pos_dev;
  t.n_pos = a.n_pos;
  t.nq = a.nq;
  t.kv_stride = a.kv_stride;
  t.err = a.err;
  return seen_positions(t);
}

// order-preserving key of a score; NaN ranks below everything
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0u;
  const uint32_t b = __float_as_uint(v);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// blocks a warp scores per pass: HD / 8 lanes share a block, four blocks at a time each
template <int HD>
constexpr int kScorePass = 4 * 32 / (HD / 8);

// The keys of one head's blocks for one query, by CTA `rank` of `ranks`, each to
// put(block, key).  A lane holds 8 channels of a block; four blocks are loaded and
// summed together: their lanes' sums are exchanged so that lane j (mod 4) of a group
// ends with block j, in 5 or 4 shuffles for the four.
template <int NT, int HD, typename Ready, typename Put>
__device__ __forceinline__ void score_blocks(const SelectArgs& a, int g, int qi, int blocks, int rank, int ranks,
                                             Ready ready, Put put) {
  constexpr int LB = HD / 8, BW = 32 / LB;
  constexpr int W = NT / 32;
  __shared__ float red[W];
  __shared__ int sums[2][HD];            // group sums of max(qi, 0) and min(qi, 0)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, part = lane % LB, sub = lane / LB;
  const int stride = ranks * W * kScorePass<HD>;
  const int64_t head = int64_t(g) * a.nb;
  const int8_t* pmax = a.kmax + head * HD + part * 8;
  const int8_t* pmin = a.kmin + head * HD + part * 8;
  int b0 = (rank * W + warp) * kScorePass<HD>;  // the warp's blocks b0 + j BW + sub, j < 4
  uint2 hi[4], lo[4];
  float ks;
  const auto load = [&](int at) {  // in flight while q is prepared or the last four are summed
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t b = min(at + j * BW + sub, blocks - 1);
      hi[j] = *reinterpret_cast<const uint2*>(pmax + b * HD);
      lo[j] = *reinterpret_cast<const uint2*>(pmin + b * HD);
    }
    ks = a.ks[head + min(at + (part & 3) * BW + sub, blocks - 1)];
  };
  load(b0);
  const float* q = a.q + (int64_t(qi) * a.n_qh + g * a.G) * HD;
  constexpr int QR = 16 * HD / NT;  // q values per thread, at most
  float x[QR];
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < QR; ++i) {
    const int at = tid + i * NT;
    x[i] = at < a.G * HD ? q[at] : 0.f;
    const float v = fabsf(x[i]);
    if (v <= 3.402823466e38f) m = fmaxf(m, v);
  }
  for (int i = tid; i < 2 * HD; i += NT) (&sums[0][0])[i] = 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red[warp] = m;
  __syncthreads();
  m = red[lane % W];
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float inv = pow2_inv(pow2_scale<10, 0x7FE000u>(m));  // 2047 = 1.99902 * 2^10
#pragma unroll
  for (int i = 0; i < QR; ++i) {
    const int v = x[i] != x[i] ? 0 : __float2int_rn(fminf(fmaxf(x[i] * inv, -2047.f), 2047.f));
    if (v) atomicAdd(&sums[v < 0][(tid + i * NT) % HD], v);
  }
  __syncthreads();
  int p2[4], n2[4];  // pairs of 16-bit sums (16 heads of 2047 fit)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int d = part * 8 + 2 * i;
    p2[i] = (sums[0][d] & 0xFFFF) | (sums[0][d + 1] << 16);
    n2[i] = (sums[1][d] & 0xFFFF) | (sums[1][d + 1] << 16);
  }
  ready();
  for (; b0 < blocks; b0 += stride) {
    int v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      int acc = __dp2a_lo(p2[0], int(hi[j].x), 0);
      acc = __dp2a_hi(p2[1], int(hi[j].x), acc);
      acc = __dp2a_lo(p2[2], int(hi[j].y), acc);
      acc = __dp2a_hi(p2[3], int(hi[j].y), acc);
      acc = __dp2a_lo(n2[0], int(lo[j].x), acc);
      acc = __dp2a_hi(n2[1], int(lo[j].x), acc);
      acc = __dp2a_lo(n2[2], int(lo[j].y), acc);
      v[j] = __dp2a_hi(n2[3], int(lo[j].y), acc);
    }
    const float t = ks;
    load(b0 + stride);
    // odd lanes keep blocks 1 and 3, then lanes with bit 1 the upper of the two
    const bool o1 = part & 1, o2 = part & 2;
    const int k0 = (o1 ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, o1 ? v[0] : v[1], 1);
    const int k1 = (o1 ? v[3] : v[2]) + __shfl_xor_sync(0xffffffffu, o1 ? v[2] : v[3], 1);
    int acc = (o2 ? k1 : k0) + __shfl_xor_sync(0xffffffffu, o2 ? k0 : k1, 2);
#pragma unroll
    for (int o = 4; o < LB; o <<= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    const int b = b0 + (part & 3) * BW + sub;
    if (b < blocks && part < 4)
      put(b, b < a.n_first || b >= blocks - a.n_last ? kForced : order_key(__int2float_rn(acc) * t));
  }
}

// One cluster per (KV head, query): its CTAs score the head's blocks and put the
// keys into the first CTA's shared memory, which selects.  Bound by the latency of
// its phases (65 blocks 3.3 us) and, for long sequences, about equally by reading the
// bounds from the cluster's SMs and by the choice in one SM (15,626 blocks of 8
// heads 16.6 us: 3.6 launch and q, 6 scoring 32 MB, 7 choice).
template <int NT, int HD>
__global__ void __launch_bounds__(NT) kv8_select_kernel(const SelectArgs a) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ SelShared<NT> sh;
  pdl_wait();
  pdl_trigger();
  const int ranks = gridDim.x, rank = blockIdx.x;  // the grid is one cluster wide
  const int g = blockIdx.y, qi = blockIdx.z;
  const int blocks = int(kv8_blocks(seen_positions(a) + qi));
  int32_t* idx = a.idx + (int64_t(qi) * a.n_kvh + g) * a.n_sel;
  if (blocks <= a.n_sel) {  // uniform over the cluster
    for (int i = rank * NT + threadIdx.x; i < a.n_sel; i += ranks * NT) idx[i] = i < blocks ? i : -1;
    return;
  }
  if (ranks == 1) {
    score_blocks<NT, HD>(a, g, qi, blocks, 0, 1, [] {}, [&](int b, uint32_t k) { keys[b] = k; });
    __syncthreads();
  } else {
    uint32_t first;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(first) : "r"(smem_u32(keys)));
    // no CTA writes into the first one before it runs
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    score_blocks<NT, HD>(
        a, g, qi, blocks, rank, ranks, [] { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); },
        [&](int b, uint32_t k) {
          asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(first + 4u * uint32_t(b)), "r"(k) : "memory");
        });
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank) return;
  }
  if (NT == kSelNarrow) {  // launched for at most kSelNarrowBlocks
    rank_blocks<NT>(a, blocks, idx, sh, keys);
    return;
  }
  const auto key = [&](int b) { return keys[b]; };
  // Keys in registers where a thread has up to five (8 heads, against shared memory: 1024
  // blocks 6.2 and 7.5 us, 1100 7.55 and 7.25, 5120 8.7 and 9.45); more of them cost more
  // than they save (17 a thread: 10,000 blocks 14.6 against 12.95, 17,408 17.0 and 16.7;
  // 33: 30,000 26.1 and 24.1).  54,784 blocks take 47 us.
  if (blocks <= NT) select_blocks<NT, 1>(a, blocks, idx, sh, key);
  else if (blocks <= 5 * NT) select_blocks<NT, 5>(a, blocks, idx, sh, key);
  else select_blocks<NT, 0>(a, blocks, idx, sh, key);
}

// the same in two launches with the keys in scratch, for heads whose keys do not
// fit in shared memory
template <int NT, int HD>
__global__ void __launch_bounds__(NT) kv8_score_kernel(const SelectArgs a) {
  pdl_wait();
  pdl_trigger();
  const int g = blockIdx.y, qi = blockIdx.z;
  const int blocks = int(kv8_blocks(seen_positions(a) + qi));
  if (blocks == 0) return;
  uint32_t* out = a.keys + (int64_t(qi) * a.n_kvh + g) * a.nb;
  score_blocks<NT, HD>(a, g, qi, blocks, blockIdx.x, gridDim.x, [] {}, [&](int b, uint32_t k) { out[b] = k; });
}
template <int NT>
__global__ void __launch_bounds__(NT) kv8_select_scratch_kernel(const SelectArgs a) {
  __shared__ SelShared<NT> sh;
  pdl_wait();
  pdl_trigger();
  const int g = blockIdx.y, qi = blockIdx.z;
  const int blocks = int(kv8_blocks(seen_positions(a) + qi));
  int32_t* idx = a.idx + (int64_t(qi) * a.n_kvh + g) * a.n_sel;
  if (blocks <= a.n_sel) {
    for (int i = threadIdx.x; i < a.n_sel; i += NT) idx[i] = i < blocks ? i : -1;
    return;
  }
  const uint32_t* keys = a.keys + (int64_t(qi) * a.n_kvh + g) * a.nb;
  select_blocks<NT, 0>(a, blocks, idx, sh, [&](int b) { return __ldcg(keys + b); });
}

}  // namespace

// ---------------------------------------------------------------------------------
// launchers (arguments already validated by the C ABI layer)

nt_status launch_kv8_append(Ctx* c, const nt_kv8& kv, int src_fmt, const void* k, const void* v, int64_t n,
                            int64_t tok_stride, int64_t head_stride, int64_t pos, const int64_t* pos_dev,
                            cudaStream_t st) {
  AppendArgs a{};
  a.src[0] = k;
  a.src[1] = v;
  a.tok_stride = tok_stride;
  a.head_stride = head_stride;
  a.dst[0] = static_cast<uint8_t*>(kv.k);
  a.dst[1] = static_cast<uint8_t*>(kv.v);
  a.scale[0] = kv.kscale;
  a.scale[1] = kv.vscale;
  a.kmin = kv.kmin;
  a.kmax = kv.kmax;
  a.n = n;
  a.pos = pos;
  a.pos_dev = pos_dev;
  a.kv_stride = kv.kv_stride;
  a.nb = kv8_blocks(kv.kv_stride);
  a.err = c->err_flag;
  // blocks the rows can touch: exact for a host position, the worst offset for a device one
  const int64_t o0 = pos_dev ? kB - 1 : pos % kB;
  const dim3 grid(unsigned((o0 + n + kB - 1) / kB), kv.n_kvh, 2), block(kAppendThreads);
  using K = void (*)(AppendArgs);
  const bool i8 = kv.fmt == NT_KV8_I8, h128 = kv.head_dim == 128;
  K kern;
  if (src_fmt == NT_F32)
    kern = i8 ? (h128 ? kv8_append_kernel<NT_KV8_I8, 128, float> : kv8_append_kernel<NT_KV8_I8, 64, float>)
              : (h128 ? kv8_append_kernel<NT_KV8_E4M3, 128, float> : kv8_append_kernel<NT_KV8_E4M3, 64, float>);
  else
    kern = i8 ? (h128 ? kv8_append_kernel<NT_KV8_I8, 128, __half> : kv8_append_kernel<NT_KV8_I8, 64, __half>)
              : (h128 ? kv8_append_kernel<NT_KV8_E4M3, 128, __half> : kv8_append_kernel<NT_KV8_E4M3, 64, __half>);
  return cuda_check(c, launch_k(c, kern, grid, block, 0, st, a), "8-bit cache write launch");
}

nt_status launch_kv8_read(Ctx* c, const nt_kv8& kv, int64_t pos, int64_t n, int dst_fmt, void* k, void* v,
                          int64_t head_stride, cudaStream_t st) {
  ReadArgs a{};
  a.src[0] = static_cast<const uint8_t*>(kv.k);
  a.src[1] = static_cast<const uint8_t*>(kv.v);
  a.scale[0] = kv.kscale;
  a.scale[1] = kv.vscale;
  a.dst[0] = k;
  a.dst[1] = v;
  a.pos = pos;
  a.n = n;
  a.kv_stride = kv.kv_stride;
  a.nb = kv8_blocks(kv.kv_stride);
  a.head_stride = head_stride;
  const int vec = dst_fmt == NT_F32 ? 4 : 8;
  const int64_t units = n * (kv.head_dim / vec), per = kReadThreads * kReadUnroll;
  const dim3 grid(unsigned((units + per - 1) / per), kv.n_kvh, 2), block(kReadThreads);
  using K = void (*)(ReadArgs);
  const bool i8 = kv.fmt == NT_KV8_I8, h128 = kv.head_dim == 128;
  K kern;
  if (dst_fmt == NT_F32)
    kern = i8 ? (h128 ? kv8_read_kernel<NT_KV8_I8, 128, float> : kv8_read_kernel<NT_KV8_I8, 64, float>)
              : (h128 ? kv8_read_kernel<NT_KV8_E4M3, 128, float> : kv8_read_kernel<NT_KV8_E4M3, 64, float>);
  else
    kern = i8 ? (h128 ? kv8_read_kernel<NT_KV8_I8, 128, __half> : kv8_read_kernel<NT_KV8_I8, 64, __half>)
              : (h128 ? kv8_read_kernel<NT_KV8_E4M3, 128, __half> : kv8_read_kernel<NT_KV8_E4M3, 64, __half>);
  return cuda_check(c, launch_k(c, kern, grid, block, 0, st, a), "8-bit cache read launch");
}

// launch_k with a cluster shape (1, 1, 1: none)
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(const Ctx* c, void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                           dim3 cluster, Args&&... args) {
  if (cluster.x * cluster.y * cluster.z == 1) return launch_k(c, kernel, grid, block, smem, st, std::forward<Args>(args)...);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster.x;
  attr[0].val.clusterDim.y = cluster.y;
  attr[0].val.clusterDim.z = cluster.z;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = (c->pdl && !c->pdl_hold) ? 2 : 1;
  c->pdl_hold = false;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

nt_status launch_attn_kv8(Ctx* c, const nt_kv8& kv, const float* q, float* out, int n_qh, int64_t n_pos, int nq,
                          const int64_t* pos_dev, const int32_t* idx, int n_sel, char* scratch, size_t scratch_bytes,
                          cudaStream_t st) {
  AttnKv8Args a{};
  a.q = q;
  a.k = static_cast<const uint8_t*>(kv.k);
  a.v = static_cast<const uint8_t*>(kv.v);
  a.ks = kv.kscale;
  a.vs = kv.vscale;
  a.out = out;
  a.idx = idx;
  a.n_sel = n_sel;
  a.n_qh = n_qh;
  a.n_kvh = kv.n_kvh;
  a.G = n_qh / kv.n_kvh;
  a.inv_g = (65536 + a.G - 1) / a.G;
  a.nq = nq;
  a.n_pos = n_pos;
  a.kv_stride = kv.kv_stride;
  a.nb = kv8_blocks(kv.kv_stride);
  a.pos_dev = pos_dev;
  a.err = c->err_flag;
  const bool sparse = idx != nullptr;
  const int rows = sparse ? a.G : a.G * nq;
  const int R = rows > 8 ? 2 : 1;
  a.chunks = (rows + 8 * R - 1) / (8 * R);
  const int z = sparse ? a.chunks * nq : a.chunks;
  // splits: the grid fills the SMs once (two CTAs each, one with R = 2), no more
  // than the longest sequence has work for, and what the scratch holds
  const int64_t most = sparse ? int64_t(n_sel) * kB : (pos_dev ? kv.kv_stride : n_pos + nq - 1);
  int64_t S = int64_t(c->num_sms) * (R == 1 ? 2 : 1) / (int64_t(kv.n_kvh) * z);
  if (S > kMaxSplits) S = kMaxSplits;
  if (S < 1) S = 1;
  const auto useful = [&](int u) { return std::max<int64_t>(1, (most + 16 * kAttnWarps * u - 1) / (16 * kAttnWarps * u)); };
  const size_t vecs = size_t(n_qh) * nq, row = vecs * (kv.head_dim * 4 + 8);
  // Up to 768 positions a split, the splits of a head run as one cluster of at most 16
  // and join in shared memory: one launch instead of two (2 us of host time; on the
  // GPU, 8 KV heads, 1024 positions 5.0 against 5.7 us, 12,000 13.2 against 15.7,
  // 16,384 15.8 against 14.3).  The CTAs of R = 2 fill an SM each, so their clusters
  // take at most half of the SMs.
  const int64_t groups = int64_t(kv.n_kvh) * z;
  const int64_t widest = std::min<int64_t>({kMaxCluster, R * kv.head_dim / 8, S, R == 1 ? S : c->num_sms / 2 / groups});
  int64_t C = 1;
  while (C < useful(R) && 2 * C <= widest) C *= 2;
  a.cluster = useful(2) > 1 && C > 1 && most <= 768 * C;
  if (a.cluster) S = C;
  // Steps of 32 tokens where every warp has one, else of 16, which give more warps
  // work (two launches, 8 KV heads: 32,768 positions 19.9 against 21.0 us, 1024 6.5
  // against 5.7); a cluster's few warps take 16 up to 640 positions a split (4160
  // positions 8.1 against 8.6 us, 12,000 13.2 against 13.6).  One CTA a head does up
  // to 256 positions in one step (4.4 us; two CTAs of shorter steps 4.9).
  const int64_t long_from = a.cluster ? 640 * S : 32 * kAttnWarps * S;
  const int U = R == 2 || most <= 32 * kAttnWarps || most >= long_from ? 2 : 1;
  if (!a.cluster) S = std::min<int64_t>({S, useful(U), std::max<int64_t>(1, int64_t(scratch_bytes / row))});
  a.S = int(S);
  a.part = reinterpret_cast<float*>(scratch);
  a.ml = reinterpret_cast<float2*>(scratch + vecs * S * kv.head_dim * 4);
  a.stall = take_stall(st);
  const AttnKv8Variant kern = sparse ? attn_kv8_for<true>(kv.fmt, kv.head_dim, R, U)
                                     : attn_kv8_for<false>(kv.fmt, kv.head_dim, R, U);
  nt_status s = cuda_check(c, launch_cluster(c, kern.kernel, dim3(kv.n_kvh, a.S, z), dim3(kAttnWarps * 32), kern.smem,
                                             st, dim3(1, a.cluster ? a.S : 1, 1), a),
                           "8-bit attention launch");
  if (s || a.S == 1 || a.cluster) return s;  // the output is written
  using Combine = void (*)(AttnKv8Args, int, int);
  Combine comb = kv.head_dim == 128 ? (sparse ? attn_kv8_combine_kernel<128, true> : attn_kv8_combine_kernel<128, false>)
                              : (sparse ? attn_kv8_combine_kernel<64, true> : attn_kv8_combine_kernel<64, false>);
  return cuda_check(c, launch_k(c, comb, dim3(n_qh, nq), dim3(kv.head_dim), 0, st, a, 8 * R, 16 * U),
                    "8-bit attention combine launch");
}

// dynamic shared memory of a selection, its static part held back
constexpr size_t kSelStatic = 13312;

static bool kv8_select_fits(const Ctx* c, int64_t blocks) {
  return size_t(blocks) * sizeof(uint32_t) + kSelStatic <= c->smem_optin;
}

size_t kv8_score_bytes(const Ctx* c, const nt_kv8& kv, int64_t n_pos, int nq, bool pos_on_device) {
  const int64_t nb = kv8_blocks(kv.kv_stride);
  const int64_t most = pos_on_device ? nb : kv8_blocks(n_pos + nq - 1);
  return kv8_select_fits(c, most) ? 0 : size_t(nq) * kv.n_kvh * size_t(nb) * sizeof(uint32_t);
}

nt_status launch_kv8_select(Ctx* c, const nt_kv8& kv, const float* q, int n_qh, int64_t n_pos, int nq,
                            const int64_t* pos_dev, int n_sel, int n_first, int n_last, int32_t* idx, char* scratch,
                            cudaStream_t st) {
  SelectArgs a{};
  a.q = q;
  a.kmin = kv.kmin;
  a.kmax = kv.kmax;
  a.ks = kv.kscale;
  a.keys = reinterpret_cast<uint32_t*>(scratch);
  a.idx = idx;
  a.n_qh = n_qh;
  a.n_kvh = kv.n_kvh;
  a.G = n_qh / kv.n_kvh;
  a.nq = nq;
  a.n_sel = n_sel;
  a.n_first = n_first;
  a.n_last = n_last;
  a.n_pos = n_pos;
  a.kv_stride = kv.kv_stride;
  a.nb = kv8_blocks(kv.kv_stride);
  a.pos_dev = pos_dev;
  a.err = c->err_flag;
  const int64_t blocks = pos_dev ? a.nb : kv8_blocks(n_pos + nq - 1);
  const bool h128 = kv.head_dim == 128;
  const int64_t pass = int64_t(kSelWide / 32) * (h128 ? kScorePass<128> : kScorePass<64>);  // blocks a CTA scores at a time
  const int64_t groups = int64_t(kv.n_kvh) * nq;
  if (blocks <= kSelNarrowBlocks)
    return cuda_check(c, launch_k(c, h128 ? kv8_select_kernel<kSelNarrow, 128> : kv8_select_kernel<kSelNarrow, 64>,
                                  dim3(1, kv.n_kvh, nq), dim3(kSelNarrow), size_t(blocks + 3) * sizeof(uint32_t), st, a),
                      "block select launch");
  if (kv8_select_fits(c, blocks)) {
    // CTAs per cluster: a pass of work for each, and the grid within the SMs
    const int ranks = int(std::max<int64_t>(1, std::min<int64_t>({kSelCluster, (blocks + pass - 1) / pass, c->num_sms / groups})));
    return cuda_check(c, launch_cluster(c, h128 ? kv8_select_kernel<kSelWide, 128> : kv8_select_kernel<kSelWide, 64>,
                                        dim3(ranks, kv.n_kvh, nq), dim3(kSelWide), size_t(blocks) * sizeof(uint32_t),
                                        st, dim3(ranks, 1, 1), a),
                      "block select launch");
  }
  int64_t gx = (blocks + pass - 1) / pass;
  const int64_t fill = (int64_t(c->num_sms) * 2 + groups - 1) / groups;
  gx = gx > fill ? fill : gx;
  nt_status s = cuda_check(c, launch_k(c, h128 ? kv8_score_kernel<kSelWide, 128> : kv8_score_kernel<kSelWide, 64>,
                                       dim3(unsigned(gx), kv.n_kvh, nq), dim3(kSelWide), 0, st, a),
                           "block score launch");
  if (s) return s;
  return cuda_check(c, launch_k(c, kv8_select_scratch_kernel<kSelWide>, dim3(1, kv.n_kvh, nq), dim3(kSelWide), 0, st, a),
                    "block select launch");
}

nt_status configure_kv8(Ctx* c) {
  for (const auto k : {kv8_select_kernel<kSelWide, 64>, kv8_select_kernel<kSelWide, 128>}) {
    nt_status s = cuda_check(c, cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     int(c->smem_optin - kSelStatic)),
                             "block select shared-memory attribute");
    if (!s) s = cuda_check(c, cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1),
                           "block select cluster attribute");
    if (s) return s;
  }
  for (int fmt : {NT_KV8_I8, NT_KV8_E4M3})
    for (int hd : {64, 128})
      for (int v = 0; v < 6; ++v) {
        const int R = v < 4 ? 1 : 2, U = v < 2 ? 1 : 2;
        const AttnKv8Variant k = v & 1 ? attn_kv8_for<true>(fmt, hd, R, U) : attn_kv8_for<false>(fmt, hd, R, U);
        nt_status s = cuda_check(
            c, cudaFuncSetAttribute(k.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(k.smem)),
            "8-bit attention shared-memory attribute");
        if (!s)
          s = cuda_check(c, cudaFuncSetAttribute(k.kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1),
                         "8-bit attention cluster attribute");
        if (s) return s;
      }
  return NT_OK;
}

}  // namespace nt
