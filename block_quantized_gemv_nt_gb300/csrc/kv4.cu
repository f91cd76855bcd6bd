// kv4.cu — the paged 4-bit KV cache of several requests: rows quantised into their
// slots and read back, and the attention of each request's rows over its own pages.
// It stands beside the F16 cache ("Ntransformer", en.unwiki.net, roadmap) and the
// 8-bit one (kv8.cu).
//
// A page holds 64 positions.  Per page and KV head there is one block: the K half,
// then the V half, each 64 rows of HD / 2 bytes and 64 HD / 32 scales.  Channels 8 j
// .. 8 j + 7 of a row are one word, channel 8 j + n its nibble n.  The order inside a
// half is the one in which the attention's MMA fragments read it (see there):
//  - K row t at t HD / 2; scale (t, group) at ((t % 8) NG + group) 8 + t / 8
//  - V word j of row t: plane j % WPL, line swap(t), word j / WPL of the line, where
//    WPL = HD / 64 and swap(t) puts t, t + 2, t + 4, t + 6 of every 8 side by side;
//    scale (t, group) at (group 4 + t / 2 % 4) 16 + t / 16 4 + t / 8 % 2 2 + t % 2
//
// A scale has at most 8 significant bits and a code at most 3, so every value is exact
// in f16: the attention multiplies the scale in as it unpacks, and its products lose
// nothing.  (Half of the least E2M1 scale would not be; the cache holds those scales
// doubled, kStored d, and what is read or attended to is halved in fp32.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <algorithm>

#include "nt_internal.cuh"
#include "ops.cuh"

namespace nt {
namespace {

constexpr int kPg = NT_KV4_PAGE;
constexpr float kTopScale = 2720.f;
template <int FMT>
constexpr float kStored = FMT == NT_KV4_E2M1 ? 2.f : 1.f;

template <int HD>
struct Kv4Block {
  static constexpr int NG = HD / 32;                  // scales of a row
  static constexpr int row = HD / 2;                  // bytes of a row's codes
  static constexpr int scales = kPg * row;            // the scales' place in a half
  static constexpr int half = scales + kPg * NG * 2;  // bytes of the K or V half
  static constexpr int bytes = 2 * half;
  static constexpr int WPL = HD / 64;                 // V words of a line's lane: planes
};
__host__ __device__ constexpr int kv4_swap(int t) { return (t & ~7) | ((t & 1) << 2) | ((t >> 1) & 3); }

// byte of word j of row t, and of the scale of (t, group), in the K (0) or V (1) half
template <int HD>
__device__ __forceinline__ int kv4_word_at(int which, int t, int j) {
  using B = Kv4Block<HD>;
  if (which == 0) return t * B::row + 4 * j;
  return (j % B::WPL) * (kPg * 32) + kv4_swap(t) * 32 + (j / B::WPL) * 4;
}
template <int HD>
__device__ __forceinline__ int kv4_scale_at(int which, int t, int group) {
  using B = Kv4Block<HD>;
  const int at = which == 0 ? ((t & 7) * B::NG + group) * 8 + (t >> 3)
                            : (group * 4 + ((t >> 1) & 3)) * 16 + (t >> 4) * 4 + ((t >> 3) & 1) * 2 + (t & 1);
  return B::scales + 2 * at;
}

// ---- codes -----------------------------------------------------------------------
// (x & m) | b as one three-input operation
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t m, uint32_t b) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "r"(m), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }

// I4: nibble i of either 16-bit half of x, in bits 6..9 of 0x4C00: the f16 number 16 + code
template <int I>
__device__ __forceinline__ __half2 i4_biased(uint32_t x) {
  const uint32_t y = I == 0 ? x << 6 : I == 1 ? x << 2 : I == 2 ? x >> 2 : x >> 6;
  return as_h2(and_or(y, 0x03C003C0u, 0x4C004C00u));
}
// E2M1: the four bytes of x, two codes each, through the hardware's conversion
__device__ __forceinline__ void e2m1_to_h2(uint32_t x, uint32_t h[4]) {
  asm("{\n\t.reg .b8 p, q, r, s;\n\tmov.b32 {p, q, r, s}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, p;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, q;\n\tcvt.rn.f16x2.e2m1x2 %2, r;\n\tcvt.rn.f16x2.e2m1x2 %3, s;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(x));
}
// a word's 8 values times kStored, exact in f16, as pairs (0, 1), (2, 3), (4, 5), (6, 7) of its channels
template <int FMT>
__device__ __forceinline__ void unpack4(uint32_t x, __half2 d2, uint32_t v[4]) {
  if (FMT == NT_KV4_I4) {
    const __half2 off = __hmul2(d2, __float2half2_rn(-24.f));
    const uint32_t p[4] = {as_u32(__hfma2(i4_biased<0>(x), d2, off)), as_u32(__hfma2(i4_biased<1>(x), d2, off)),
                           as_u32(__hfma2(i4_biased<2>(x), d2, off)), as_u32(__hfma2(i4_biased<3>(x), d2, off))};
    v[0] = __byte_perm(p[0], p[1], 0x5410);  // channels i (low halves) and i + 4
    v[1] = __byte_perm(p[2], p[3], 0x5410);
    v[2] = __byte_perm(p[0], p[1], 0x7632);
    v[3] = __byte_perm(p[2], p[3], 0x7632);
  } else {
    e2m1_to_h2(x, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = as_u32(__hmul2(as_h2(v[i]), d2));
  }
}

// the largest (smallest) of three; NaN if one is
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min3_nan(float a, float b, float c) {
  float r;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// the scale: d0 held to the largest, rounded to 8 bits, then to f16
__device__ __forceinline__ float scale8(float d0) {
  d0 = fminf(fmaxf(d0, -kTopScale), kTopScale);
  return __half2float(__float2half_rn(__bfloat162float(__float2bfloat16_rn(d0))));
}
// a / 6 so that its rounding to 8 bits is that of the exact quotient: an fp32 quotient
// halfway between two of them is moved to the side on which the exact one lies
__device__ __forceinline__ float sixth(float a) {
  const float q = __fdiv_rn(a, 6.f);
  uint32_t u = __float_as_uint(q);
  if ((u & 0xFFFFu) == 0x8000u) {
    const float rest = fmaf(-6.f, q, a);
    u += rest > 0.f ? 1u : rest < 0.f ? ~0u : 0u;
  }
  return __uint_as_float(u);
}

// The codes of 8 values over the scale d (inv about 1 / d, 0 for d = 0), as a word, decided
// by products of the borders and d, which are exact in fp32.
template <int FMT>
__device__ __noinline__ uint32_t codes4_exact(float4 a, float4 b, float d, float inv) {
  uint32_t w = 0;
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    const float v = i == 0 ? a.x : i == 1 ? a.y : i == 2 ? a.z : i == 3 ? a.w : i == 4 ? b.x : i == 5 ? b.y : i == 6 ? b.z : b.w;
    uint32_t code;
    if (FMT == NT_KV4_I4) {
      float q = rintf(fminf(fmaxf(v * inv, -9.f), 9.f));
      // x / d - q, as x - q d with the sign of d; exact wherever it is near half of d
      const float rest = copysignf(1.f, d) * fmaf(-q, d, v), half = 0.5f * fabsf(d);
      if (fabsf(rest) > half || (fabsf(rest) == half && (int(q) & 1))) q += rest > 0.f ? 1.f : -1.f;
      code = inv == 0.f ? 8u : uint32_t(int(fminf(fmaxf(q, -8.f), 7.f)) + 8);
    } else {
      const float m = fabsf(v);
      code = (m > 0.25f * d) + (m >= 0.75f * d) + (m > 1.25f * d) + (m >= 1.75f * d) + (m > 2.5f * d) + (m >= 3.5f * d) +
             (m > 5.f * d);
      code = (inv == 0.f ? 0u : code) | (v < 0.f ? 8u : 0u);
    }
    w |= code << (4 * i);
  }
  return w;
}

// The same where the scale has its 8 bits and is below the largest one: the products x inv
// are within 2^-22 of the quotients, which are at most 8 (6) and a 2^-8th.  Where one of
// them is that near a border the exact products decide again.
template <int FMT>
__device__ __forceinline__ uint32_t codes4(const float x[8], float d, float inv) {
  if (FMT == NT_KV4_I4) {
    // x / d + 200.5: of 192 + 8 + the quotient, the whole part's low 4 bits are the code,
    // rounded half up; 16 bits of the rest stand below them, and a border is where they are 0
    uint32_t z[8], least = ~0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      z[i] = __float_as_uint(fminf(fmaf(x[i], inv, 200.5f), 207.9375f));
      least = min(least, z[i] * 65536u + (8u << 16));
    }
    if (least < (16u << 16)) {
      const float half = 0.5f * fabsf(d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t u = z[i] & 0xFFFF0000u;                 // 200 + the rounded quotient
        const float rest = copysignf(1.f, d) * fmaf(200.f - __uint_as_float(u), d, x[i]);
        const bool move = fabsf(rest) > half || (fabsf(rest) == half && (u & 0x10000u));
        z[i] = min(move ? (rest > 0.f ? u + 0x10000u : u - 0x10000u) : u, 0x434F0000u);  // 207: code 15
      }
    }
    const uint32_t e0 = __byte_perm(z[0], z[2], 0x0062), e1 = __byte_perm(z[4], z[6], 0x0062);
    const uint32_t o0 = __byte_perm(z[1], z[3], 0x0062), o1 = __byte_perm(z[5], z[7], 0x0062);
    const uint32_t even = __byte_perm(e0, e1, 0x5410), odd = __byte_perm(o0, o1, 0x5410);
    return and_or(even, 0x0F0F0F0Fu, (odd << 4) & 0xF0F0F0F0u);
  }
  // the codes of products a little larger and a little smaller: where they differ, the border is near
  const auto pack = [&](float by) {
    uint32_t w;
    asm("{\n\t.reg .b8 p, q, r, s;\n\tcvt.rn.satfinite.e2m1x2.f32 p, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 q, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 r, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 s, %8, %7;\n\tmov.b32 %0, {p, q, r, s};\n\t}"
        : "=r"(w)
        : "f"(x[0] * by), "f"(x[1] * by), "f"(x[2] * by), "f"(x[3] * by), "f"(x[4] * by), "f"(x[5] * by), "f"(x[6] * by),
          "f"(x[7] * by));
    return w;
  };
  uint32_t w = pack(inv * (1.f + 0x1p-20f));
  for (uint32_t diff = w ^ pack(inv * (1.f - 0x1p-20f)); diff;) {
    const int at = (__ffs(diff) - 1) & ~3, i = at >> 2;
    const uint32_t up = (w >> at) & 7u;
    uint32_t h[4];
    e2m1_to_h2(up | ((up - 1u) << 4), h);
    const float2 g = __half22float2(as_h2(h[0]));
    float m = x[0];
#pragma unroll
    for (int k = 1; k < 8; ++k) m = k == i ? x[k] : m;
    m = fabsf(m);
    const float border = 0.5f * (g.x + g.y) * d;
    if (m < border || (m == border && (up & 1u))) w -= 1u << at;
    diff &= ~(15u << at);
  }
  return w;
}

// The same of F16 values.  One of them is on a border (k + 1/2) d, 12 bits, or at least a
// 2^-12th of it away: the quotient after one correction, which is exact on borders and within
// 2^-22 of itself elsewhere, rounds as the exact one does.
template <int FMT>
__device__ __forceinline__ uint32_t codes4_f16(const float x[8], float d, float inv) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] = x[i] * inv;
    y[i] = fmaf(fmaf(-y[i], d, x[i]), inv, y[i]);
  }
  uint32_t w;
  if (FMT == NT_KV4_I4) {
    uint32_t z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = __float_as_uint(fminf(y[i], 7.f) + 12582920.f);  // 1.5 * 2^23 + 8: the code in the low bits
    const uint32_t a = __byte_perm(z[1] * 16u + z[0], z[3] * 16u + z[2], 0x0040);
    w = __byte_perm(a, __byte_perm(z[5] * 16u + z[4], z[7] * 16u + z[6], 0x0040), 0x5410);
  } else {
    asm("{\n\t.reg .b8 p, q, r, s;\n\tcvt.rn.satfinite.e2m1x2.f32 p, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 q, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 r, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 s, %8, %7;\n\tmov.b32 %0, {p, q, r, s};\n\t}"
        : "=r"(w)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  }
  return w;
}

// ---- write and read back ------------------------------------------------------------
// A thread has 16 channels of a row, two words of codes: half of a group.
constexpr int kRowThreads = 256;
template <typename T>
constexpr int kRowPasses = sizeof(T) == 4 ? 2 : 4;  // rows a thread has in flight: 128 bytes

struct Kv4RowsArgs {
  char* row[2];  // K, V rows (either may be null when read)
  int64_t tok_stride, head_stride;  // bytes
  uint8_t* data;
  const int64_t* slots;
  int64_t n_tok, n_slots;
  int n_kvh;
  bool wide;     // rows start at multiples of 32 bytes
  unsigned* err;
};

// the two words j, j + 1 (j even) of row t of a half
template <int HD>
__device__ __forceinline__ void store_words(uint8_t* half, int which, int t, int j, uint32_t a, uint32_t b) {
  if (which && HD == 128) {  // a plane each
    *reinterpret_cast<uint32_t*>(half + kv4_word_at<HD>(1, t, j)) = a;
    *reinterpret_cast<uint32_t*>(half + kv4_word_at<HD>(1, t, j + 1)) = b;
  } else {
    *reinterpret_cast<uint2*>(half + kv4_word_at<HD>(which, t, j)) = make_uint2(a, b);
  }
}
template <int HD>
__device__ __forceinline__ uint2 load_words(const uint8_t* half, int which, int t, int j) {
  if (which && HD == 128)
    return make_uint2(*reinterpret_cast<const uint32_t*>(half + kv4_word_at<HD>(1, t, j)),
                      *reinterpret_cast<const uint32_t*>(half + kv4_word_at<HD>(1, t, j + 1)));
  return *reinterpret_cast<const uint2*>(half + kv4_word_at<HD>(which, t, j));
}

// 16 values of a row as they are loaded
template <typename T>
struct Raw16 {
  uint32_t w[4 * sizeof(T)];
};
template <typename T>
__device__ __forceinline__ void load16(const char* p, bool wide, Raw16<T>& v) {
  if (wide) {
#pragma unroll
    for (int i = 0; i < 4 * int(sizeof(T)); i += 8)
      asm("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
          : "=r"(v.w[i]), "=r"(v.w[i + 1]), "=r"(v.w[i + 2]), "=r"(v.w[i + 3]), "=r"(v.w[i + 4]), "=r"(v.w[i + 5]),
            "=r"(v.w[i + 6]), "=r"(v.w[i + 7])
          : "l"(p + 4 * i)
          : "memory");
    return;
  }
#pragma unroll
  for (int i = 0; i < int(sizeof(T)); ++i) {
    const uint4 a = reinterpret_cast<const uint4*>(p)[i];
    v.w[4 * i] = a.x, v.w[4 * i + 1] = a.y, v.w[4 * i + 2] = a.z, v.w[4 * i + 3] = a.w;
  }
}
__device__ __forceinline__ void floats(const Raw16<float>& r, float v[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r.w[i]);
}
__device__ __forceinline__ void floats(const Raw16<__half>& r, float v[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = __half22float2(as_h2(r.w[i]));
    v[2 * i] = f.x, v[2 * i + 1] = f.y;
  }
}
// the largest and the smallest value over the two threads of a group; NaN if one is
__device__ __forceinline__ void extremes(const Raw16<float>& r, float& hi, float& lo) {
  float v[16];
  floats(r, v);
  hi = lo = v[0];
#pragma unroll
  for (int i = 1; i < 15; i += 2) {
    hi = max3_nan(hi, v[i], v[i + 1]);
    lo = min3_nan(lo, v[i], v[i + 1]);
  }
  const float up = max3_nan(hi, v[15], v[15]), dn = min3_nan(lo, v[15], v[15]);
  const float a = __shfl_xor_sync(0xffffffffu, up, 1), b = __shfl_xor_sync(0xffffffffu, dn, 1);
  hi = max3_nan(up, a, a);
  lo = min3_nan(dn, b, b);
}
__device__ __forceinline__ void extremes(const Raw16<__half>& r, float& hi, float& lo) {
  __half2 up = as_h2(r.w[0]), dn = up;
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    up = __hmax2_nan(up, as_h2(r.w[i]));
    dn = __hmin2_nan(dn, as_h2(r.w[i]));
  }
  const uint32_t a = as_u32(up), b = as_u32(__hneg2(dn));
  __half2 m = __hmax2_nan(as_h2(__byte_perm(a, b, 0x5410)), as_h2(__byte_perm(a, b, 0x7632)));  // (largest, - smallest)
  m = __hmax2_nan(m, as_h2(__shfl_xor_sync(0xffffffffu, as_u32(m), 1)));
  const float2 f = __half22float2(m);
  hi = f.x;
  lo = -f.y;
}
__device__ __forceinline__ float about_inverse(float d) {  // within 2^-23; 0 for 0
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return d != 0.f ? r : 0.f;
}

// One CTA: kRowPasses * 4096 / HD tokens of one head's K or V.  Where rows are few, two
// round trips of latency (16 rows of 8 heads 1.9 us, a bare launch 1.0); where they are
// many, HBM: 32,767 F32 rows of 8 heads 48 us, 303 MB, 6.3 TB/s.  Of F16 rows there is
// half as much to read for the same arithmetic, and instruction issue bounds them: 131,072
// in 132 us, 671 MB, 5.1 TB/s, the issue slots 82% and the integer pipe 57% busy; with four
// rows a thread and four CTAs an SM (64 registers), as here, faster than with two rows
// (134) or one (161).
template <int FMT, int HD, typename T>
__global__ void __launch_bounds__(kRowThreads, 4) kv4_append_kernel(const Kv4RowsArgs a) {
  using B = Kv4Block<HD>;
  constexpr int TR = HD / 16;  // threads of a row
  constexpr int RP = kRowThreads / TR, NP = kRowPasses<T>;
  constexpr float kMax = 3.402823466e38f;
  pdl_wait();
  pdl_trigger();
  const int j = 2 * (threadIdx.x % TR), h = blockIdx.y, which = blockIdx.z;
  const int64_t tok0 = int64_t(blockIdx.x) * (RP * NP) + threadIdx.x / TR;
  const char* src = (which ? a.row[1] : a.row[0]) + h * a.head_stride + int(sizeof(T)) * 8 * j;
  int64_t slot[NP];
  Raw16<T> x[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) slot[i] = tok0 + i * RP < a.n_tok ? a.slots[tok0 + i * RP] : -1;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    if (slot[i] >= a.n_slots) {
      if (j == 0) flag_error(a.err, kErrPaged);
      slot[i] = -1;
    }
#pragma unroll
    for (uint32_t& w : x[i].w) w = 0u;
    if (slot[i] >= 0) load16(src + (tok0 + i * RP) * a.tok_stride, a.wide, x[i]);
  }
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    if (!__any_sync(0xffffffffu, slot[i] >= 0)) continue;
    float hi, lo, v[16];
    extremes(x[i], hi, lo);
    floats(x[i], v);
    const bool clean = hi <= kMax && lo >= -kMax;  // the same for the group's two threads
    if (__any_sync(0xffffffffu, !clean)) {
      float up = hi, dn = lo;
      if (!clean) {  // NaN becomes 0, an infinity leaves the scale alone
        flag_error(a.err, kErrNonFinite4);
        up = dn = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          if (v[k] != v[k]) v[k] = 0.f;
          if (fabsf(v[k]) <= kMax) up = fmaxf(up, v[k]), dn = fminf(dn, v[k]);
          v[k] = fminf(fmaxf(v[k], -1e38f), 1e38f);
        }
      }
      hi = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 1));
      lo = fminf(dn, __shfl_xor_sync(0xffffffffu, dn, 1));
    }
    const float d = scale8(FMT == NT_KV4_I4 ? (hi >= -lo ? hi : lo) * -0.125f : sixth(fmaxf(hi, -lo)));
    const float inv = about_inverse(d);
    // a scale that lost bits to f16's least numbers, or is the largest, may leave quotients beyond the codes
    const bool plain = clean && (d == 0.f || (fabsf(d) >= 0x1p-16f && fabsf(d) < kTopScale));
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float* y = v + 8 * k;
      if (!plain)
        w[k] = codes4_exact<FMT>(make_float4(y[0], y[1], y[2], y[3]), make_float4(y[4], y[5], y[6], y[7]), d, inv);
      else
        w[k] = sizeof(T) == 4 ? codes4<FMT>(y, d, inv) : codes4_f16<FMT>(y, d, inv);
    }
    if (slot[i] < 0) continue;
    const uint64_t page = uint64_t(slot[i]) / kPg;
    const int t = int(slot[i]) & (kPg - 1);
    uint8_t* half = a.data + (page * a.n_kvh + h) * B::bytes + which * B::half;
    store_words<HD>(half, which, t, j, w[0], w[1]);
    if (j % 4 == 0) *reinterpret_cast<__half*>(half + kv4_scale_at<HD>(which, t, j / 4)) = __float2half_rn(d * kStored<FMT>);
  }
}

// The way back: 131,072 F16 rows of 8 heads 105 us, 6.4 TB/s.
template <int FMT, int HD, typename T>
__global__ void __launch_bounds__(kRowThreads) kv4_read_kernel(const Kv4RowsArgs a) {
  using B = Kv4Block<HD>;
  constexpr int TR = HD / 16;
  constexpr int RP = kRowThreads / TR, NP = kRowPasses<T>;
  pdl_wait();
  pdl_trigger();
  const int j = 2 * (threadIdx.x % TR), h = blockIdx.y, which = blockIdx.z;
  char* out = which ? a.row[1] : a.row[0];
  if (!out) return;
  out += h * a.head_stride + int(sizeof(T)) * 8 * j;
  const int64_t tok0 = int64_t(blockIdx.x) * (RP * NP) + threadIdx.x / TR;
  int64_t slot[NP];
  uint2 w[NP];
  __half d[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) slot[i] = tok0 + i * RP < a.n_tok ? a.slots[tok0 + i * RP] : -1;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    if (slot[i] >= a.n_slots) {
      if (j == 0) flag_error(a.err, kErrPaged);
      slot[i] = -1;
    }
    if (slot[i] < 0) continue;
    const uint64_t page = uint64_t(slot[i]) / kPg;
    const int t = int(slot[i]) & (kPg - 1);
    const uint8_t* half = a.data + (page * a.n_kvh + h) * B::bytes + which * B::half;
    w[i] = load_words<HD>(half, which, t, j);
    d[i] = *reinterpret_cast<const __half*>(half + kv4_scale_at<HD>(which, t, j / 4));
  }
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    if (slot[i] < 0) continue;
    uint32_t v[8];
    unpack4<FMT>(w[i].x, __half2half2(d[i]), v);
    unpack4<FMT>(w[i].y, __half2half2(d[i]), v + 4);
    char* to = out + (tok0 + i * RP) * a.tok_stride;
    uint32_t y[4 * sizeof(T)];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (sizeof(T) == 4) {
        const float2 f = __half22float2(as_h2(v[k]));
        y[2 * k % (4 * sizeof(T))] = __float_as_uint(f.x * (1.f / kStored<FMT>));
        y[(2 * k + 1) % (4 * sizeof(T))] = __float_as_uint(f.y * (1.f / kStored<FMT>));
      } else {
        y[k] = FMT == NT_KV4_E2M1 ? as_u32(__hmul2(as_h2(v[k]), __float2half2_rn(1.f / kStored<FMT>))) : v[k];
      }
    }
    if (a.wide) {
#pragma unroll
      for (int k = 0; k < 4 * int(sizeof(T)); k += 8)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + 4 * k), "r"(y[k]), "r"(y[k + 1]),
                     "r"(y[k + 2]), "r"(y[k + 3]), "r"(y[k + 4]), "r"(y[k + 5]), "r"(y[k + 6]), "r"(y[k + 7])
                     : "memory");
    } else {
#pragma unroll
      for (int k = 0; k < int(sizeof(T)); ++k)
        reinterpret_cast<uint4*>(to)[k] = make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
    }
  }
}

// ---- attention -----------------------------------------------------------------------
// Scores and outputs on the tensor cores (mma.sync m16n8k16, f16 products, fp32 sums)
// with fp32-level operands.  K and V are the A operands: 16 positions by 16 channels of
// K, 16 channels by 16 positions of V, exact in f16 with their scales.  A column pair
// (2 r, 2 r + 1) of the B operand holds hi = f16(x) and lo, the rest x - hi, of query row r
// (or of its probabilities, there times kLo), which together carry 22 bits: of q down to 2^-17
// of the row's largest value, of probabilities to 2^-22 of the largest.  A tile of 8 columns is
// 4 rows (NT tiles: 4 NT rows), and the two parts of a product meet in one thread.
//
// Fragments come without a transpose in shared memory: the names of MMA rows and k slots
// are ours.  Lane (g = lane / 4, c = lane % 4), 16 positions 16 m .. of a page:
//  - K: the lane reads rows 16 m + g and 16 m + 8 + g, channels c HD / 4 .. of them; word
//    w, pairs 2 u and 2 u + 1 of either row are its part of k-step (w, u).
//  - S^T: the lane then has the scores of those positions with row c of each tile.
//  - P: (hi, lo) of a position and row is one register, an 8 x 8 transpose in the
//    registers (movmatrix) turns them into the B fragment whose k slots are positions.
//  - V: the lane reads word w of channels g HD / 8 .. of rows 16 m + 2 c, + 1, + 8, + 9;
//    channel n of the word is MMA row g or g + 8 of m-tile n % 4 (I4) or n / 2 (E2M1).
//
// Work: the steps (a page of one KV head for one chunk of 4 NT query rows) of all requests
// in one line, the same number to each warp, whatever the requests' lengths.  A warp walks
// its steps with an online softmax; where it begins or ends inside an item (request, head, chunk) it leaves a partial (m, l, o).  The CTA joins
// its warps' partials of one item, and the last CTA to arrive at an item that several
// share joins theirs, in the order of the line: nothing depends on who arrives when.
//
// A step is a whole page: each warp has the K and the V half of one in shared memory and
// the next page's halves on their way in the same places as soon as it has used them; with
// steps of 32 or 16 positions the joins and the copies' round trips cost more than the
// shorter steps save (4160 positions 17.7 and 22.8 us, whole pages 13.3 then).
//
// What bounds it.  Up to 4 rows (a decode step): instruction issue, before HBM.  A page of
// a head is 9216 bytes and about 1180 warp instructions for E2M1 (hardware conversion and
// one multiply a pair), 1390 for I4 (shift, mask, fused multiply-add a pair); 1,000,003
// positions of 8 heads take 186 and 212 us, 6.2 and 5.4 TB/s, the tensor cores 23..25%
// busy, the integer pipe half.  Two CTAs of 8 warps an SM; with 16 warps in one CTA these took
// 178 and 202 where two of 8 took 184 and 209, but 64 requests of up to 8000 positions (107,693
// in all) 36.8 and not 34.4.  Some 13 us of a call in line are its prologue and the join through
// global memory (131,071 positions 40.5 us, 22.2 of them bytes).  8 rows (verify passes): one
// CTA of 8 warps an SM with 255 registers, tensor cores 33%, issue 45%; the dependent
// products and conversions of 8 warps do not fill more (16 ragged requests of 64 query
// heads and up to 5 rows 59 us; with 12 warps 67, with 16 rows a step 76, with unpacked
// tiles shared by all warps 71).  Why not tcgen05: its 128 rows take two pages, unpacked to
// f16 tiles in shared memory, and scores, probabilities and outputs then pass between warps
// through TMEM and shared memory; that chain took 2.8 us a step, the ragged requests 122 us,
// and 2000 rows over 4000 positions 1044 us, where 8 rows a step took 1122 (chunks in order).
constexpr int kMaxCtas = 512;                 // one counter each
constexpr float kPTop = 8.f, kSlack = 6.f;    // probabilities are up to 2^(kPTop + kSlack), in f16's range
constexpr float kLowest = -3.402823466e38f;
constexpr int64_t kMaxSteps = int64_t(1) << 28;
constexpr int kMaxCluster = 8;
constexpr int kOwnSteps = 2, kSharedSteps = 3;  // most steps a warp takes of an item that is a CTA's, or a cluster's own
constexpr int kJoin = 16;                     // partials of an item that a join has in flight together

struct AttnKv4Args {
  const float* q;
  const uint8_t* data;
  float* out;
  const int32_t *q_start, *held, *table;
  float* part;         // [CTA][2][rows][HD]
  float2* ml;          // [CTA][2][rows]
  unsigned* counters;  // [CTA], zero at rest
  unsigned* err;
  int64_t max_pages, n_pages, n_tok;
  uint64_t inv_g;      // ceil(2^32 / G): row / G = row inv_g >> 32 below 2^28 rows
  int n_req, n_qh, n_kvh, G;
  int cluster_log;     // of CTAs
  int stall;
};

__device__ __forceinline__ void mma16816(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the same from zero
__device__ __forceinline__ void mma16816_zero(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A weight's f16 parts: hi to nearest, and what that left, exact in fp32, times 2^11.  So the
// lower part is as large as hi's own steps allow, and small weights keep theirs: each is off by
// 2^-22 of itself or by 2^-36, which is 2^-44 of the largest.  (Not scaled, the lower part of
// weights below 2^-22 of the largest was lost, up to 2^-6 of a tail of equal ones; scaling it
// costs 0.5 to 1.5% of the time.)
constexpr float kLo = 0x1p11f;
// (hi, lo) of x and of y, a register each
__device__ __forceinline__ void hi_lo(float x, float y, uint32_t& of_x, uint32_t& of_y) {
  const __half2 hi = __floats2half2_rn(x, y);
  const float2 f = __half22float2(hi);
  float2 rest;  // (x - f.x) kLo, (y - f.y) kLo
  asm("{\n\t.reg .b64 a, b, m, n;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 m, {%6, %6};\n\t"
      "mov.b64 n, {%7, %7};\n\tmul.rn.f32x2 a, a, m;\n\tfma.rn.f32x2 a, b, n, a;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(rest.x), "=f"(rest.y)
      : "f"(x), "f"(y), "f"(f.x), "f"(f.y), "f"(kLo), "f"(-kLo));
  const __half2 lo = __floats2half2_rn(rest.x, rest.y);
  of_x = __byte_perm(as_u32(hi), as_u32(lo), 0x5410);
  of_y = __byte_perm(as_u32(hi), as_u32(lo), 0x7632);
}
// 8 bytes at this CTA's shared address `at` in the CTA `rank` of the cluster
__device__ __forceinline__ float2 ld_cluster(uint32_t at, int rank) {
  float2 v;
  asm volatile("{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %2, %3;\n\tld.shared::cluster.v2.f32 {%0, %1}, [a];\n\t}"
               : "=f"(v.x), "=f"(v.y)
               : "r"(at), "r"(rank)
               : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// an arrival that orders what this CTA wrote before it and reads what earlier ones wrote
__device__ __forceinline__ unsigned arrive_counter(unsigned* at) {
  unsigned old;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(at) : "memory");
  return old;
}

// a request: its first row, rows and positions, held to what the arguments allow, and
// the steps of it and of those before it
struct Req {
  int row0, rows, len, steps;
};

// shared memory: each warp's K and V halves; its partial of the item that it found
// begun; the requests.  At the end the warps' last partials lie in their own K and V halves.
template <int HD, int NT, int kWarps>
struct AttnKv4Smem {
  static constexpr int ROWS = 4 * NT;
  static constexpr int line = HD + 4;                                  // floats of a row of a partial
  static constexpr size_t slot = size_t(ROWS) * line * 4 + ROWS * 8;   // then (m, l) of each row
  static constexpr size_t ring = 0;
  static constexpr size_t first = size_t(kWarps) * Kv4Block<HD>::bytes;
  static constexpr size_t reqs = first + kWarps * slot;
  static_assert(slot <= size_t(Kv4Block<HD>::bytes), "a partial fits a warp's halves");
  static constexpr int max_ctas = 4096 / ROWS < kMaxCtas ? 4096 / ROWS : kMaxCtas;
  static_assert(max_ctas * ROWS * 8 + kWarps * 32 * 16 <= first, "a join's weights and sums fit the ring");
  static_assert(reqs % 16 == 0, "requests are read as 16 bytes");
};

// an item, and the step of it that comes next
struct Item {
  int r, h;          // request, KV head
  int row0, at;      // the chunk's first row: of q the request's, of the request's (query, head) rows
  int rows, q_rows;  // rows of the chunk, queries of the request
  int len, steps, j;
};

template <int FMT, int HD, int NT, int kWarps, int CTAS>
__global__ void __launch_bounds__(kWarps * 32, CTAS) attn_kv4_kernel(const AttnKv4Args a) {
  using B = Kv4Block<HD>;
  using L = AttnKv4Smem<HD, NT, kWarps>;
  constexpr int ROWS = 4 * NT;
  constexpr int WK = HD / 32;  // K words of a lane and row
  constexpr int KS = HD / 16;  // k-steps of the scores
  constexpr int CW = HD / 8;   // output channels of a lane and row
  extern __shared__ __align__(16) uint8_t sm4[];
  __shared__ __align__(8) uint64_t bars[kWarps][2];
  __shared__ int seg_item[2 * kWarps];   // item (its first step) of a warp's partials, -1: none
  __shared__ Item seg_of[2 * kWarps];
  __shared__ int64_t wsum[kWarps];
  __shared__ unsigned arrived;
  Req* const reqs = reinterpret_cast<Req*>(sm4 + L::reqs);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const uint32_t bar = smem_u32(&bars[warp][0]);
  const int cluster_rank = blockIdx.x & ((1 << a.cluster_log) - 1);
  const uint64_t pol = policy_evict_first();
  if (lane == 0) {
    mbar_init(bar, 1);
    mbar_init(bar + 8, 1);
    fence_barrier_init();
    seg_item[2 * warp] = seg_item[2 * warp + 1] = -1;
  }
  pdl_wait();
  pdl_trigger();

  // x / d; both below 2^21, as a rule, and then exact in fp32 up to one
  const auto divide = [](unsigned x, unsigned d) {
    if (x >= 1u << 21) return x / d;
    unsigned q = __float2uint_rz(__uint2float_rn(x) * about_inverse(__uint2float_rn(d)));
    q -= q * d > x;
    return q + ((q + 1) * d <= x);
  };
  // ---- the requests and the sums of their pages' steps
  int64_t total64 = 0;
  const auto read_req = [&](int r, int64_t& v) {
    Req x{0, 0, 0, 0};
    v = 0;
    if (r < a.n_req) {
      const int b = a.q_start[r], e = a.q_start[r + 1], n = a.held[r];
      const int64_t cap = a.max_pages * kPg;
      const bool rows_ok = b >= 0 && e >= b && e <= a.n_tok, len_ok = n >= 0 && n <= cap;
      x.row0 = b;
      x.rows = rows_ok ? e - b : 0;
      x.len = len_ok ? n : n < 0 ? 0 : int(cap);
      if (!(rows_ok && len_ok) && blockIdx.x == 0) flag_error(a.err, kErrPaged);
      v = ((int64_t(x.rows) * a.G + ROWS - 1) / ROWS) * a.n_kvh * max(1, (x.len + kPg - 1) / kPg);
      v = min(v, kMaxSteps + 1);  // so that the sums cannot overflow
    }
    return x;
  };
  const auto scan = [&](int64_t v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += x;
    }
    return v;
  };
  // Few requests, whose items all find a CTA or a cluster of their own and are not much longer
  // than its warps: then no item is joined through global memory (16 requests of up to 500
  // positions, 1247 in all, 7.4 us, in line 9.4; 1088 positions of one 7.8 in clusters of 8, 9.3
  // of 2, in line 10.2; 4160 10.6 and in line 12.8).
  int own_r = -1, own_it = 0;  // the request and item of it that this CTA, or its cluster, has; -1: steps in line
  bool for_cluster = false;    // the cluster has it
  if (a.n_req <= 32) {  // every warp by itself: all write the same
    int64_t v;
    Req x = read_req(lane, v);
    const int64_t mine = v;
    v = scan(v);
    total64 = __shfl_sync(0xffffffffu, v, 31);
    x.steps = int(min(v, kMaxSteps));
    if (lane < a.n_req) reqs[lane] = x;
    __syncwarp();
    const int pages = max(1, (x.len + kPg - 1) / kPg), longest = __reduce_max_sync(0xffffffffu, mine ? pages : 0);
    if (longest <= (kSharedSteps * kWarps << a.cluster_log) && total64 <= int64_t(gridDim.x) * longest) {
      int items = int(divide(unsigned(mine), pages));
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, items, o);
        if (lane >= o) items += y;
      }
      const int all = __shfl_sync(0xffffffffu, items, 31);
      for_cluster = longest > kWarps && all <= int(gridDim.x) >> a.cluster_log;
      if (for_cluster || (longest <= kOwnSteps * kWarps && all <= int(gridDim.x))) {
        const int me = for_cluster ? blockIdx.x >> a.cluster_log : blockIdx.x;
        own_r = __popc(__ballot_sync(0xffffffffu, items <= me));
        if (own_r == 32) return;
        own_it = me - (own_r ? __shfl_sync(0xffffffffu, items, own_r - 1) : 0);
      }
    }
  } else {
    for (int r0 = 0; r0 < a.n_req; r0 += kWarps * 32) {
      int64_t v;
      Req x = read_req(r0 + tid, v);
      v = scan(v);
      if (lane == 31) wsum[warp] = v;
      __syncthreads();
      v += total64;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) v += wsum[w];
        total64 += wsum[w];
      }
      x.steps = int(min(v, kMaxSteps));
      if (r0 + tid < a.n_req) reqs[r0 + tid] = x;
      __syncthreads();
    }
  }
  if (total64 > kMaxSteps) {
    if (blockIdx.x == 0 && tid == 0) flag_error(a.err, kErrTooMuch);
    return;
  }
  const int warps = gridDim.x * kWarps;
  // the CTA's steps, and of each warp the same number
  const int total = int(total64);
  int cta0, cta1, per, own_first = 0;
  if (own_r >= 0) {
    const int pages = max(1, (reqs[own_r].len + kPg - 1) / kPg);
    cta0 = (own_r ? reqs[own_r - 1].steps : 0) + own_it * pages;
    cta1 = cta0 + pages;
    own_first = cta0;
    if (for_cluster) {
      const int each = (pages + (1 << a.cluster_log) - 1) >> a.cluster_log;
      cta0 = min(cta1, cta0 + cluster_rank * each);
      cta1 = min(cta1, cta0 + each);
    }
    per = (cta1 - cta0 + kWarps - 1) / kWarps;
  } else {
    per = max(1, int(divide(total + warps - 1, warps)));
    cta0 = min(int64_t(total), int64_t(blockIdx.x) * (kWarps * per));
    cta1 = min(total, cta0 + kWarps * per);
    if (cta0 >= cta1) return;
  }
  const int s0 = min(cta1, cta0 + warp * per), s1 = min(cta1, s0 + per);

  const auto query_of = [&](int row) { return int((uint64_t(unsigned(row)) * a.inv_g) >> 32); };
  const auto locate = [&](int s) {
    int lo = -1, hi = a.n_req - 1;  // the first request whose sum is above s
    if (own_r >= 0) hi = own_r, lo = hi - 1;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (reqs[mid].steps > s) hi = mid; else lo = mid;
    }
    const Req q = reqs[hi];
    const int before = hi ? reqs[hi - 1].steps : 0;
    Item x;
    x.r = hi;
    x.len = q.len;
    x.row0 = q.row0;
    x.q_rows = q.rows;
    x.steps = max(1, (q.len + kPg - 1) / kPg);
    const unsigned chunks = unsigned(q.rows * a.G + ROWS - 1) / ROWS, off = unsigned(s - before);
    const unsigned it = divide(off, x.steps), h = divide(it, chunks);
    x.j = int(off - it * x.steps);
    x.h = int(h);
    // a prompt's first chunks see little of it and its last ones all: taken in turn from
    // either end, so that each warp's share of the line is as much work (4000 rows of 4000
    // positions 1313 us, in order 2177; 2000 rows of up to 4000 positions 924 and 1123)
    const unsigned k = it - h * chunks;
    x.at = int(k & 1 ? chunks - 1 - k / 2 : k / 2) * ROWS;
    x.rows = min(ROWS, q.rows * a.G - x.at);
    return x;
  };
  // positions that row `row` of the chunk sees
  const auto seen = [&](const Item& x, int row) { return x.len - (x.q_rows - 1 - query_of(x.at + row)); };
  // the offset of its vector in q and out
  const auto vec_of = [&](const Item& x, int row) {
    const int qi = query_of(x.at + row);
    return (int64_t(x.row0 + qi) * a.n_qh + x.h * a.G + (x.at + row - qi * a.G)) * HD;
  };
  uint8_t* const sk = sm4 + L::ring + size_t(warp) * B::bytes;
  const uint8_t* const sv = sk + B::half;
  // the K (0) or V (1) half of block `b`
  const auto copy = [&](const uint8_t* b, int which) {
    if (!b || lane != 0) return;
    mbar_arrive_expect_tx(bar + 8 * which, B::half);
    if (!a.stall) bulk_g2s(smem_u32(which ? sv : sk), b + which * B::half, B::half, bar + 8 * which, pol);
  };
  uint32_t phase = 0;
  bool dead = false;  // a wait ran out: the rest is taken as not seen
  const auto wait = [&](int which, bool next_k) {
    const int cap = a.stall ? kStallSpin : kMaxSpin;
    if (__all_sync(0xffffffffu, mbar_wait(bar + 8 * which, phase, cap))) return true;
    if (lane == 0) flag_error(a.err, kErrWaitTimeout);
    mbar_wait(bar + 8 * which, phase, cap);
    if (which == 0) mbar_wait(bar + 8, phase, cap);
    else if (next_k) mbar_wait(bar, phase ^ 1, cap);
    dead = true;
    return false;
  };
  // 32 entries of an item's table, one a lane, from page `p0` on: blocks, or -1 where a
  // page is not seen or not one of the cache
  const auto entries = [&](const Item& x, int p0, int pages_seen) {
    const int p = p0 + lane;
    if (p >= pages_seen) return -1;
    const int e = a.table[x.r * a.max_pages + p];
    if (e >= 0 && e < a.n_pages) return e;
    flag_error(a.err, kErrPaged);
    return -1;
  };
  const auto block_of = [&](const Item& x, int ent, int j) -> const uint8_t* {
    const int e = __shfl_sync(0xffffffffu, ent, j & 31);
    return e < 0 ? nullptr : a.data + (int64_t(e) * a.n_kvh + x.h) * B::bytes;
  };

  // this lane's channels of the rows that its columns stand for, requested as soon as the item is known
  float qv[NT][HD / 4];
  const auto load_q = [&](const Item& x) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int row = 4 * t + (g >> 1);
      const float* q = a.q + vec_of(x, row) + c * (HD / 4);
#pragma unroll
      for (int i = 0; i < HD / 4; i += 4) {
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row < x.rows) y = *reinterpret_cast<const float4*>(q + i);
        qv[t][i] = y.x, qv[t][i + 1] = y.y, qv[t][i + 2] = y.z, qv[t][i + 3] = y.w;
      }
    }
  };

  Item x{}, nx{};
  const uint8_t* blk = nullptr;
  int ent = -1;
  for (int s = s0; s < s1;) {
    // ---- an item: its rows of q, scaled by a power of two to amax in [2^13, 2^14) and split
    if (s == s0) x = locate(s);
    load_q(x);
    const int tokens = seen(x, x.rows - 1), fewest = seen(x, 0), pages_seen = (tokens + kPg - 1) / kPg;
    if (s == s0) {
      ent = entries(x, x.j & ~31, pages_seen);
      blk = block_of(x, ent, x.j);
      copy(blk, 0);
      copy(blk, 1);
    }
    const int first_j = x.j, last_j = min(x.steps, x.j + (s1 - s));
    uint32_t qf[NT][KS][2];
    float rscale[NT], m[NT], l[NT], o[NT][CW];
    int limit[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float* v = qv[t];
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < HD / 4; ++i) top = fmaxf(top, fabsf(v[i]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = min(100, 140 - int(__float_as_uint(top) >> 23));
      const float sc = __uint_as_float(uint32_t(e + 127) << 23);
#pragma unroll
      for (int w = 0; w < WK; ++w)
#pragma unroll
        for (int p = 0; p < 4; ++p) {  // pair p of word w
          const int i0 = 8 * w + (FMT == NT_KV4_I4 ? p : 2 * p), i1 = 8 * w + (FMT == NT_KV4_I4 ? p + 4 : 2 * p + 1);
          const __half2 hi = __floats2half2_rn(v[i0] * sc, v[i1] * sc);
          const float2 f = __half22float2(hi);
          const __half2 lo = __floats2half2_rn(v[i0] * sc - f.x, v[i1] * sc - f.y);
          qf[t][2 * w + p / 2][p & 1] = as_u32(g & 1 ? lo : hi);
        }
      // of row c of the tile: lanes 8 c .. hold its q
      rscale[t] = __uint_as_float(uint32_t(127 - __shfl_sync(0xffffffffu, e, 8 * c)) << 23) *
                  (1.44269504088896f / kStored<FMT> * rsqrtf(float(HD)));
      limit[t] = 4 * t + c < x.rows ? seen(x, 4 * t + c) : 0;
      m[t] = -INFINITY;
      l[t] = 0.f;
#pragma unroll
      for (int i = 0; i < CW; ++i) o[t][i] = 0.f;
    }
    for (int j = first_j; j < last_j; ++j, ++s) {
      // the next step's block, requested before this step's work
      const uint8_t* nblk = nullptr;
      if (j + 1 < last_j) {
        if (((j + 1) & 31) == 0) ent = entries(x, j + 1, pages_seen);
        if (!dead) nblk = block_of(x, ent, j + 1);
      } else if (s + 1 < s1) {
        nx = locate(s + 1);
        ent = entries(nx, 0, (seen(nx, nx.rows - 1) + kPg - 1) / kPg);
        if (!dead) nblk = block_of(nx, ent, 0);
      }
      bool live = blk != nullptr && !dead;
      const int t0 = j * kPg;
      float sc[NT][4][4];
      if (live) live = wait(0, false);
      if (live) {
        // ---- scores
        const uint4 ksw = *reinterpret_cast<const uint4*>(sk + B::scales + (g * B::NG + (HD == 128 ? c : c >> 1)) * 16);
        const uint32_t ks[4] = {ksw.x, ksw.y, ksw.z, ksw.w};  // rows g + 8 i of the page: two a word
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
          uint32_t kw[2][WK];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint8_t* p = sk + (16 * mt + 8 * e + g) * B::row + c * (HD / 8);
            if (HD == 128) {
              const uint4 y = *reinterpret_cast<const uint4*>(p);
              kw[e][0] = y.x, kw[e][1] = y.y, kw[e][WK - 2] = y.z, kw[e][WK - 1] = y.w;
            } else {
              const uint2 y = *reinterpret_cast<const uint2*>(p);
              kw[e][0] = y.x, kw[e][1] = y.y;
            }
          }
          const __half2 d2[2] = {as_h2(__byte_perm(ks[mt], 0u, 0x1010)), as_h2(__byte_perm(ks[mt], 0u, 0x3232))};
          const __half2 off[2] = {__hmul2(d2[0], __float2half2_rn(-24.f)), __hmul2(d2[1], __float2half2_rn(-24.f))};
#pragma unroll
          for (int w = 0; w < WK; ++w) {
            uint32_t kv[2][4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (FMT == NT_KV4_I4) {
                kv[e][0] = as_u32(__hfma2(i4_biased<0>(kw[e][w]), d2[e], off[e]));
                kv[e][1] = as_u32(__hfma2(i4_biased<1>(kw[e][w]), d2[e], off[e]));
                kv[e][2] = as_u32(__hfma2(i4_biased<2>(kw[e][w]), d2[e], off[e]));
                kv[e][3] = as_u32(__hfma2(i4_biased<3>(kw[e][w]), d2[e], off[e]));
              } else {
                e2m1_to_h2(kw[e][w], kv[e]);
#pragma unroll
                for (int i = 0; i < 4; ++i) kv[e][i] = as_u32(__hmul2(as_h2(kv[e][i]), d2[e]));
              }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint32_t af[4] = {kv[0][2 * u], kv[1][2 * u], kv[0][2 * u + 1], kv[1][2 * u + 1]};
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                if (w == 0 && u == 0)
                  mma16816_zero(sc[t][mt], af, qf[t][0][0], qf[t][0][1]);
                else
                  mma16816(sc[t][mt], af, qf[t][2 * w + u][0], qf[t][2 * w + u][1]);
              }
            }
          }
        }
      }
      __syncwarp();  // this step's K is in registers and used
      if (!dead) copy(nblk, 0);
      uint32_t pf[NT][4][2];
      if (live) {
        // ---- online softmax, base 2: m is left behind by up to kSlack before the sums are rescaled
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float p[8];  // positions 8 i + g of the page
#pragma unroll
          for (int i = 0; i < 8; ++i) p[i] = (sc[t][i / 2][2 * (i & 1)] + sc[t][i / 2][2 * (i & 1) + 1]) * rscale[t];
          if (t0 + kPg > fewest) {
            const int left = limit[t] - t0 - g;
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = 8 * i < left ? p[i] : -INFINITY;
          }
          float mx = p[0];
#pragma unroll
          for (int i = 1; i < 8; ++i) mx = fmaxf(mx, p[i]);
          if (__any_sync(0xffffffffu, mx > m[t] + kSlack)) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const float mn = fmaxf(m[t], mx);
            const float corr = mn == -INFINITY ? 1.f : ex2(m[t] - mn);
            m[t] = mn;
            l[t] *= corr;
#pragma unroll
            for (int i = 0; i < CW; ++i) o[t][i] *= corr;
          }
          const float base = m[t] == -INFINITY ? 0.f : kPTop - m[t];
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            p[i] = ex2(p[i] + base);
            sum += p[i];
          }
          l[t] += sum;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t a, b;
            hi_lo(p[2 * i], p[2 * i + 1], a, b);
            pf[t][i][0] = transpose8(a);
            pf[t][i][1] = transpose8(b);
          }
        }
        live = wait(1, nblk != nullptr);
      }
      if (live) {
        // ---- P V.  Each page's products start from zero and are added to the output in
        // fp32: the tensor cores round their sums towards zero, and that bias would grow
        // with the length.
        const uint4* vsp = reinterpret_cast<const uint4*>(sv + B::scales + ((HD == 128 ? g >> 1 : g >> 2) * 4 + c) * 32);
        const uint4 va = vsp[0], vb = vsp[1];
        uint32_t vs[8] = {va.x, va.y, va.z, va.w, vb.x, vb.y, vb.z, vb.w};  // positions 8 i + 2 c, + 1
        if (t0 + kPg > tokens) {  // positions that no row sees: whatever their bytes are, they count as 0
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int left = tokens - t0 - 8 * i - 2 * c;
            vs[i] = left > 1 ? vs[i] : left == 1 ? vs[i] & 0xFFFFu : 0u;
          }
        }
#pragma unroll
        for (int w = 0; w < B::WPL; ++w) {
          float acc[NT][4][4];
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) {
            uint32_t vv[2][2][4];  // [positions 2 c, + 1 or + 8, + 9][MMA row g or g + 8][m-tile]
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint8_t* p = sv + w * (kPg * 32) + (16 * mt + 8 * e + c) * 32 + g * 4;
              const uint32_t r0 = *reinterpret_cast<const uint32_t*>(p), r1 = *reinterpret_cast<const uint32_t*>(p + 128);
              const __half2 d2 = as_h2(vs[2 * mt + e]);
              if (FMT == NT_KV4_I4) {
                const __half2 off = __hmul2(d2, __float2half2_rn(-24.f));
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                  const uint32_t y = __byte_perm(r0, r1, f ? 0x7632 : 0x5410);
                  vv[e][f][0] = as_u32(__hfma2(i4_biased<0>(y), d2, off));
                  vv[e][f][1] = as_u32(__hfma2(i4_biased<1>(y), d2, off));
                  vv[e][f][2] = as_u32(__hfma2(i4_biased<2>(y), d2, off));
                  vv[e][f][3] = as_u32(__hfma2(i4_biased<3>(y), d2, off));
                }
              } else {
                // bytes of two nibbles: the even (odd) channels of both positions
                const uint32_t even = and_or(r0, 0x0F0F0F0Fu, (r1 << 4) & 0xF0F0F0F0u);
                const uint32_t odd = and_or(r0 >> 4, 0x0F0F0F0Fu, r1 & 0xF0F0F0F0u);
                e2m1_to_h2(even, vv[e][0]);
                e2m1_to_h2(odd, vv[e][1]);
#pragma unroll
                for (int f = 0; f < 2; ++f)
#pragma unroll
                  for (int n = 0; n < 4; ++n) vv[e][f][n] = as_u32(__hmul2(as_h2(vv[e][f][n]), d2));
              }
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const uint32_t af[4] = {vv[0][0][n], vv[0][1][n], vv[1][0][n], vv[1][1][n]};
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                if (mt == 0)
                  mma16816_zero(acc[t][n], af, pf[t][mt][0], pf[t][mt][1]);
                else
                  mma16816(acc[t][n], af, pf[t][mt][0], pf[t][mt][1]);
              }
            }
          }
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              o[t][8 * w + (FMT == NT_KV4_I4 ? n : 2 * n)] += fmaf(acc[t][n][1], 1.f / kLo, acc[t][n][0]);
              o[t][8 * w + (FMT == NT_KV4_I4 ? n + 4 : 2 * n + 1)] += fmaf(acc[t][n][3], 1.f / kLo, acc[t][n][2]);
            }
        }
      }
      __syncwarp();  // and its V
      if (!dead) copy(nblk, 1);
      if (blk) phase ^= 1;
      blk = nblk;
    }
    // ---- the item's end, or the warp's: the output, or a partial
    const bool begun = first_j == 0, ended = last_j == x.steps;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[t] += __shfl_xor_sync(0xffffffffu, l[t], d);
    if (begun && ended && !for_cluster) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (4 * t + c >= x.rows) continue;
        const float inv = l[t] == 0.f ? 0.f : 1.f / kStored<FMT> / l[t];
        float* to = a.out + vec_of(x, 4 * t + c) + g * CW;
#pragma unroll
        for (int i = 0; i < CW; i += 4)
          *reinterpret_cast<float4*>(to + i) =
              make_float4(o[t][i] * inv, o[t][i + 1] * inv, o[t][i + 2] * inv, o[t][i + 3] * inv);
      }
    } else {
      const int which = ended ? 0 : 1;
      uint8_t* base = which ? sk : sm4 + L::first + warp * L::slot;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float* to = reinterpret_cast<float*>(base) + (4 * t + c) * L::line + g * CW;
#pragma unroll
        for (int i = 0; i < CW; i += 4)
          *reinterpret_cast<float4*>(to + i) = make_float4(o[t][i], o[t][i + 1], o[t][i + 2], o[t][i + 3]);
        if (g == 0) reinterpret_cast<float2*>(base + ROWS * L::line * 4)[4 * t + c] = make_float2(m[t], l[t]);
      }
      if (lane == 0) {
        seg_item[2 * warp + which] = s - last_j;
        seg_of[2 * warp + which] = x;
      }
    }
    x = nx;
  }
  __syncthreads();

  // ---- join the warps' partials of one item, (warp, first or last) in the line's order
  const auto slot_of = [&](int i) {
    return i & 1 ? sm4 + L::ring + size_t(i >> 1) * B::bytes : sm4 + L::first + size_t(i >> 1) * L::slot;
  };
  const int mine = lane < 2 * kWarps ? seg_item[lane] : -1;
  const unsigned same = __match_any_sync(0xffffffffu, mine);
  unsigned left = __ballot_sync(0xffffffffu, mine >= 0);
  float* const mine_part = reinterpret_cast<float*>(sm4 + L::reqs + size_t(a.n_req) * sizeof(Req));
  float2* const mine_ml = reinterpret_cast<float2*>(mine_part + ROWS * HD);
  int shared_seg[2] = {-1, -1};  // a partial of the items that other CTAs have parts of: begun elsewhere, ending elsewhere
  while (left) {
    const int i0 = __ffs(left) - 1;
    const unsigned run = __shfl_sync(0xffffffffu, same, i0);
    const int item = __shfl_sync(0xffffffffu, mine, i0);
    left &= ~run;
    const Item& y = seg_of[i0];
    const bool begun = item >= cta0, whole = begun && item + y.steps <= cta1;
    const int side = begun ? 1 : 0;
    for (int e = 2 * tid; e < ROWS * HD; e += kWarps * 64) {
      const int row = e / HD, ch = e % HD;
      // the warps' last partials, then (at most one in a run) the one that a warp found begun, which is the line's last
      float2 ml[kWarps + 1], v[kWarps + 1];
      const int tail = __ffs(run & 0x55555555u) - 1;
#pragma unroll
      for (int w = 0; w <= kWarps; ++w) {
        const int i = w < kWarps ? 2 * w + 1 : tail;
        const bool in = w < kWarps ? run >> (2 * w + 1) & 1u : tail >= 0;
        ml[w] = make_float2(-INFINITY, 0.f);
        v[w] = make_float2(0.f, 0.f);
        if (in) {
          const uint8_t* slot = slot_of(i);
          ml[w] = reinterpret_cast<const float2*>(slot + ROWS * L::line * 4)[row];
          v[w] = *reinterpret_cast<const float2*>(reinterpret_cast<const float*>(slot) + row * L::line + ch);
        }
      }
      float M = kLowest, sum = 0.f;
      float2 acc = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w <= kWarps; ++w) M = fmaxf(M, ml[w].x);
#pragma unroll
      for (int w = 0; w <= kWarps; ++w) {
        const float f = ex2(ml[w].x - M);
        sum = fmaf(ml[w].y, f, sum);
        acc.x = fmaf(v[w].x, f, acc.x);
        acc.y = fmaf(v[w].y, f, acc.y);
      }
      if (for_cluster) {
        *reinterpret_cast<float2*>(mine_part + row * HD + ch) = acc;
        if (ch == 0) mine_ml[row] = make_float2(M, sum);
      } else if (whole) {
        const float inv = sum == 0.f ? 0.f : 1.f / kStored<FMT> / sum;
        if (row < y.rows) *reinterpret_cast<float2*>(a.out + vec_of(y, row) + ch) = make_float2(acc.x * inv, acc.y * inv);
      } else {
        const int64_t at = (int64_t(blockIdx.x) * 2 + side) * ROWS + row;
        *reinterpret_cast<float2*>(a.part + at * HD + ch) = acc;
        if (ch == 0) a.ml[at] = make_float2(M, sum);
      }
    }
    if (!whole) shared_seg[side] = i0;
  }
  if (for_cluster) {
    // ---- the cluster joins its CTAs' partials, each CTA an equal part of the outputs
    if (cta0 >= cta1) {
      for (int e = tid; e < ROWS * HD; e += kWarps * 32) mine_part[e] = 0.f;
      if (tid < ROWS) mine_ml[tid] = make_float2(-INFINITY, 0.f);
    }
    cluster_sync();
    const Item y = locate(own_first);
    const uint32_t at = smem_u32(mine_part), at_ml = smem_u32(mine_ml);
    const int ranks = 1 << a.cluster_log, share = ROWS * HD >> a.cluster_log;
    for (int e = cluster_rank * share + 2 * tid; e < (cluster_rank + 1) * share; e += kWarps * 64) {
      const int row = e / HD;
      float2 ml[kMaxCluster], v[kMaxCluster];
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) {
        ml[k] = k < ranks ? ld_cluster(at_ml + row * 8, k) : make_float2(-INFINITY, 0.f);
        v[k] = k < ranks ? ld_cluster(at + e * 4, k) : make_float2(0.f, 0.f);
      }
      float M = kLowest, sum = 0.f;
      float2 acc = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) M = fmaxf(M, ml[k].x);
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) {
        const float f = ex2(ml[k].x - M);
        sum = fmaf(ml[k].y, f, sum);
        acc.x = fmaf(v[k].x, f, acc.x);
        acc.y = fmaf(v[k].y, f, acc.y);
      }
      const float inv = sum == 0.f ? 0.f : 1.f / kStored<FMT> / sum;
      if (row < y.rows) *reinterpret_cast<float2*>(a.out + vec_of(y, row) + e % HD) = make_float2(acc.x * inv, acc.y * inv);
    }
    cluster_sync();  // no CTA leaves while another reads its shared memory
    return;
  }

  // ---- join the CTAs' partials of an item: the last to arrive does, in the line's order
  for (int side = 0; side < 2; ++side) {
    const int seg = shared_seg[side];
    if (seg < 0) continue;
    const Item& y = seg_of[seg];
    const int item = seg_item[seg];
    const int first = divide(item, kWarps * per), last = divide(item + y.steps - 1, kWarps * per), n = last - first + 1;
    __syncthreads();
    if (tid == 0) {
      arrived = arrive_counter(a.counters + first);
      if (arrived + 1 == unsigned(n)) a.counters[first] = 0u;
    }
    __syncthreads();
    if (arrived + 1 != unsigned(n)) continue;
    // the partial of CTA first + i: its item began there (i = 0), or elsewhere
    const auto part_row = [&](int i, int row) { return (int64_t(first + i) * 2 + (i == 0 ? 1 : 0)) * ROWS + row; };
    if (n <= kJoin) {  // few: all in flight together
      for (int e = 2 * tid; e < y.rows * HD; e += kWarps * 64) {
        const int row = e / HD, ch = e % HD;
        float2 ml[kJoin], v[kJoin];
#pragma unroll
        for (int i = 0; i < kJoin; ++i) {
          ml[i] = i < n ? __ldcg(a.ml + part_row(i, row)) : make_float2(-INFINITY, 0.f);
          v[i] = i < n ? __ldcg(reinterpret_cast<const float2*>(a.part + part_row(i, row) * HD + ch)) : make_float2(0.f, 0.f);
        }
        float M = kLowest, sum = 0.f;
        float2 acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kJoin; ++i) M = fmaxf(M, ml[i].x);
#pragma unroll
        for (int i = 0; i < kJoin; ++i) {
          const float f = ex2(ml[i].x - M);
          sum = fmaf(ml[i].y, f, sum);
          acc.x = fmaf(v[i].x, f, acc.x);
          acc.y = fmaf(v[i].y, f, acc.y);
        }
        const float inv = sum == 0.f ? 0.f : 1.f / kStored<FMT> / sum;
        *reinterpret_cast<float2*>(a.out + vec_of(y, row) + ch) = make_float2(acc.x * inv, acc.y * inv);
      }
      continue;
    }
    // many: the outputs' quads over all threads, S threads a quad where there are more threads
    constexpr int kThreads = kWarps * 32, QUADS = ROWS * HD / 4, S = kThreads > QUADS ? kThreads / QUADS : 1;
    constexpr int kFly = 8;  // loads in flight
    float2* mls = reinterpret_cast<float2*>(sm4 + L::ring);  // (m, l), then in m's place the weight
    __shared__ float inv[ROWS];
    for (int i = tid; i < n * ROWS; i += kThreads) mls[i] = __ldcg(a.ml + part_row(i / ROWS, i % ROWS));
    const int first_quad = tid % QUADS, lane_s = S > 1 ? tid / QUADS : 0;
    const auto quad = [&](int i, int e) {
      return i < n ? __ldcg(reinterpret_cast<const float4*>(a.part + part_row(i, e / (HD / 4)) * HD) + e % (HD / 4))
                   : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    float4 v[kFly];
#pragma unroll
    for (int k = 0; k < kFly; ++k) v[k] = quad(lane_s + k * S, first_quad);
    __syncthreads();
    for (int row = warp; row < ROWS; row += kWarps) {
      float M = kLowest, sum = 0.f;
      for (int i = lane; i < n; i += 32) M = fmaxf(M, mls[i * ROWS + row].x);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
      for (int i = lane; i < n; i += 32) {
        const float2 ml = mls[i * ROWS + row];
        const float f = ex2(ml.x - M);
        mls[i * ROWS + row].x = f;
        sum = fmaf(ml.y, f, sum);
      }
      sum = warp_sum(sum);
      if (lane == 0) inv[row] = sum == 0.f ? 0.f : 1.f / kStored<FMT> / sum;
    }
    __syncthreads();
    for (int e = first_quad; e < QUADS; e += kThreads) {
      const int row = e / (HD / 4);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i0 = lane_s; i0 < n; i0 += kFly * S) {
        if (i0 != lane_s || e != first_quad) {
#pragma unroll
          for (int k = 0; k < kFly; ++k) v[k] = quad(i0 + k * S, e);
        }
#pragma unroll
        for (int k = 0; k < kFly; ++k) {
          const float f = i0 + k * S < n ? mls[(i0 + k * S) * ROWS + row].x : 0.f;
          acc.x = fmaf(v[k].x, f, acc.x);
          acc.y = fmaf(v[k].y, f, acc.y);
          acc.z = fmaf(v[k].z, f, acc.z);
          acc.w = fmaf(v[k].w, f, acc.w);
        }
      }
      if (S > 1) {  // the quad's threads meet behind the weights
        float4* meet = reinterpret_cast<float4*>(sm4 + L::ring + size_t(L::max_ctas) * ROWS * 8);
        if (lane_s) meet[(lane_s - 1) * QUADS + e] = acc;
        __syncthreads();
        if (lane_s) break;
#pragma unroll
        for (int k = 1; k < S; ++k) {
          const float4 y = meet[(k - 1) * QUADS + e];
          acc.x += y.x, acc.y += y.y, acc.z += y.z, acc.w += y.w;
        }
      }
      if (row < y.rows) {
        const float f = inv[row];
        *reinterpret_cast<float4*>(a.out + vec_of(y, row) + 4 * (e % (HD / 4))) =
            make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
      }
    }
    __syncthreads();  // the weights are read before the other side's
  }
}

using RowsKernel = void (*)(Kv4RowsArgs);
template <template <int, int, typename> class Pick>
RowsKernel kv4_rows_for(int fmt, int hd, int row_fmt) {
  if (fmt == NT_KV4_I4)
    return row_fmt == NT_F32 ? (hd == 128 ? Pick<NT_KV4_I4, 128, float>::kernel : Pick<NT_KV4_I4, 64, float>::kernel)
                             : (hd == 128 ? Pick<NT_KV4_I4, 128, __half>::kernel : Pick<NT_KV4_I4, 64, __half>::kernel);
  return row_fmt == NT_F32 ? (hd == 128 ? Pick<NT_KV4_E2M1, 128, float>::kernel : Pick<NT_KV4_E2M1, 64, float>::kernel)
                           : (hd == 128 ? Pick<NT_KV4_E2M1, 128, __half>::kernel : Pick<NT_KV4_E2M1, 64, __half>::kernel);
}
template <int FMT, int HD, typename T>
struct AppendPick {
  static constexpr RowsKernel kernel = kv4_append_kernel<FMT, HD, T>;
};
template <int FMT, int HD, typename T>
struct ReadPick {
  static constexpr RowsKernel kernel = kv4_read_kernel<FMT, HD, T>;
};

Kv4RowsArgs rows_args(const Ctx* c, const nt_kv4& kv, int fmt, void* k, void* v, int64_t n, int64_t tok_stride,
                      int64_t head_stride, const int64_t* slots) {
  const int size = fmt == NT_F32 ? 4 : 2;
  Kv4RowsArgs a{};
  a.row[0] = static_cast<char*>(k);
  a.row[1] = static_cast<char*>(v);
  a.tok_stride = tok_stride * size;
  a.head_stride = head_stride * size;
  a.data = static_cast<uint8_t*>(kv.data);
  a.slots = slots;
  a.n_tok = n;
  a.n_slots = kv.n_pages * kPg;
  a.n_kvh = kv.n_kvh;
  a.wide = aligned(k, 32) && aligned(v, 32) && a.tok_stride % 32 == 0 && a.head_stride % 32 == 0;
  a.err = c->err_flag;
  return a;
}
dim3 rows_grid(const nt_kv4& kv, int fmt, int64_t n) {
  const int64_t per = (fmt == NT_F32 ? kRowPasses<float> : kRowPasses<__half>) * kRowThreads / (kv.head_dim / 16);
  return dim3(unsigned((n + per - 1) / per), kv.n_kvh, 2);
}

using AttnKernel = void (*)(AttnKv4Args);
struct AttnVariant {
  AttnKernel kernel;
  size_t smem;  // without the requests
  int rows, warps, ctas, max_ctas;
};
template <int FMT, int HD, int NT, int WARPS, int CTAS>
AttnVariant attn_variant() {
  return {attn_kv4_kernel<FMT, HD, NT, WARPS, CTAS>, AttnKv4Smem<HD, NT, WARPS>::reqs + 4 * NT * (HD + 2) * 4,
          4 * NT, WARPS, CTAS, AttnKv4Smem<HD, NT, WARPS>::max_ctas};
}
template <int FMT, int HD>
AttnVariant attn_pick(int NT) {
  return NT == 1 ? attn_variant<FMT, HD, 1, 8, 2>() : attn_variant<FMT, HD, 2, 8, 1>();
}
AttnVariant attn_for(int fmt, int hd, int NT) {
  if (fmt == NT_KV4_I4) return hd == 128 ? attn_pick<NT_KV4_I4, 128>(NT) : attn_pick<NT_KV4_I4, 64>(NT);
  return hd == 128 ? attn_pick<NT_KV4_E2M1, 128>(NT) : attn_pick<NT_KV4_E2M1, 64>(NT);
}

}  // namespace

size_t kv4_page_bytes(int head_dim) { return head_dim == 128 ? Kv4Block<128>::bytes : Kv4Block<64>::bytes; }

nt_status launch_kv4_append(Ctx* c, const nt_kv4& kv, int fmt, const void* k, const void* v, int64_t n, int64_t tok_stride,
                            int64_t head_stride, const int64_t* slots, cudaStream_t st) {
  const Kv4RowsArgs a = rows_args(c, kv, fmt, const_cast<void*>(k), const_cast<void*>(v), n, tok_stride, head_stride, slots);
  return cuda_check(c, launch_k(c, kv4_rows_for<AppendPick>(kv.fmt, kv.head_dim, fmt), rows_grid(kv, fmt, n), dim3(kRowThreads), 0,
                                st, a),
                    "4-bit cache write launch");
}

nt_status launch_kv4_read(Ctx* c, const nt_kv4& kv, int fmt, void* k, void* v, int64_t n, int64_t tok_stride,
                          int64_t head_stride, const int64_t* slots, cudaStream_t st) {
  const Kv4RowsArgs a = rows_args(c, kv, fmt, k, v, n, tok_stride, head_stride, slots);
  return cuda_check(c, launch_k(c, kv4_rows_for<ReadPick>(kv.fmt, kv.head_dim, fmt), rows_grid(kv, fmt, n), dim3(kRowThreads), 0,
                                st, a),
                    "4-bit cache read launch");
}

size_t kv4_attn_scratch(int head_dim) {
  // at most 4096 rows of CTAs, two partials each
  return size_t(4096) * 2 * (head_dim * sizeof(float) + sizeof(float2));
}

nt_status launch_attn_kv4(Ctx* c, const nt_kv4& kv, const float* q, float* out, int n_qh, int64_t n_tok, int n_req,
                          const int32_t* q_start, const int32_t* held, const int32_t* table, int64_t max_pages, char* scratch,
                          unsigned* counters, cudaStream_t st) {
  AttnKv4Args a{};
  a.q = q;
  a.data = static_cast<const uint8_t*>(kv.data);
  a.out = out;
  a.q_start = q_start;
  a.held = held;
  a.table = table;
  a.counters = counters;
  a.err = c->err_flag;
  a.max_pages = max_pages;
  a.n_pages = kv.n_pages;
  a.n_tok = n_tok;
  a.n_req = n_req;
  a.n_qh = n_qh;
  a.n_kvh = kv.n_kvh;
  a.G = n_qh / kv.n_kvh;
  a.inv_g = ((uint64_t(1) << 32) + a.G - 1) / a.G;
  a.stall = take_stall(st);
  // By the rows that there is room for; the lengths are the device's.  8 rows a step where the
  // requests have one each cost a second product and leave one CTA an SM (room for five: 16 requests
  // of 1900 positions, 32/8 heads, 22.1 us and not 14.7, of 8000 49.6 and not 40.3); 4 rows a
  // step where they have more read the pages again for each 4.
  const int64_t rows = (n_tok + n_req - 1) / n_req * a.G;
  const int NT = rows <= 4 ? 1 : 2;
  const AttnVariant k = attn_for(kv.fmt, kv.head_dim, NT);
  // Clusters of 8 where no request can be longer than a cluster of its own takes and, by the
  // rows' average, all items find one; else of 2: larger ones do not fill the SMs (1,000,003
  // positions 212 us in clusters of 2, 330 in such of 4: the last of them start when others end).
  // What a request may hold is the tables' width, so a short one in a wide table has clusters of 2
  // or stands in line (256 pages: 1088 positions 9.2 us and not 7.8, 4160 12.8 and not 10.6).
  const int64_t items = n_req * int64_t(kv.n_kvh) * ((rows + k.rows - 1) / k.rows);
  const bool wide = max_pages <= kSharedSteps * k.warps * kMaxCluster && items <= c->kv4_ctas[NT - 1][1] / kMaxCluster;
  a.cluster_log = wide ? 3 : 1;
  const int ctas = std::min(c->kv4_ctas[NT - 1][wide], k.max_ctas) >> a.cluster_log << a.cluster_log;
  a.ml = reinterpret_cast<float2*>(scratch);
  a.part = reinterpret_cast<float*>(scratch + size_t(ctas) * 2 * k.rows * sizeof(float2));
  return cuda_check(c, launch_cluster(c, k.kernel, dim3(ctas), dim3(k.warps * 32), k.smem + size_t(n_req) * sizeof(Req), st,
                                      dim3(1 << a.cluster_log, 1, 1), a),
                    "4-bit attention launch");
}

nt_status configure_kv4(Ctx* c) {
  for (int fmt : {NT_KV4_I4, NT_KV4_E2M1})
    for (int hd : {64, 128})
      for (int NT : {1, 2}) {
        const AttnVariant k = attn_for(fmt, hd, NT);
        nt_status s = cuda_check(
            c, cudaFuncSetAttribute(k.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(k.smem + 1024 * sizeof(Req))),
            "4-bit attention shared-memory attribute");
        if (s) return s;
        // CTAs that run at once in clusters of 2 and of 8, the least of the variants'
        for (int wide : {0, 1}) {
          cudaLaunchConfig_t cfg{};
          const int size = wide ? kMaxCluster : 2;
          cfg.gridDim = dim3(unsigned(k.ctas * c->num_sms / size * size));
          cfg.blockDim = dim3(k.warps * 32);
          cfg.dynamicSmemBytes = k.smem + 1024 * sizeof(Req);
          cudaLaunchAttribute attr[1];
          attr[0].id = cudaLaunchAttributeClusterDimension;
          attr[0].val.clusterDim = {unsigned(size), 1, 1};
          cfg.attrs = attr;
          cfg.numAttrs = 1;
          int n = 0;
          s = cuda_check(c, cudaOccupancyMaxActiveClusters(&n, k.kernel, &cfg), "4-bit attention occupancy");
          if (s) return s;
          int& most = c->kv4_ctas[NT - 1][wide];
          n = std::max(1, n) * size;
          most = most ? std::min(most, n) : n;
        }
      }
  return NT_OK;
}

}  // namespace nt
