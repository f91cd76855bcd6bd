// rope.cu — rotary positions on the rows of several tensors at once ("RoPE",
// fr.news.hada.io, "Fonctionnalités principales"): any positions, pairs adjacent or
// in halves, part of the head, frequencies scaled for long contexts.
#include <cmath>

#include "nt_internal.cuh"
#include "ops.cuh"

namespace nt {
namespace {

constexpr int kRopeThreads = 128;

struct RopeJob {
  const char* x;
  char* y;
  int64_t x_tok, x_head, y_tok, y_head;  // bytes
  int end;                               // heads of this job and those before it
};
struct RopeRowsArgs {
  RopeJob job[3];
  const int32_t* pos;
  int64_t pos0, n_tok;
  int heads, units, turned;  // units of 8 channels in a row, and how many of them turn
  float mag;
  bool in_place;             // the units that do not turn stay where they are
};

// A unit is four pairs: 8 adjacent channels (PAIRS), or channels 4 u .. 4 u + 3 of
// either half (HALVES).  T float: two 16-byte pieces; __half: one, or two of 8 bytes.
template <typename T>
struct Unit {
  float a[4], b[4];  // the pairs
};
__device__ __forceinline__ float2 f2(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2*>(&h)); }
__device__ __forceinline__ uint32_t h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// the raw words of a unit at channel `c0` (and `c1` of the other half)
template <typename T, bool HALVES>
__device__ __forceinline__ void load_unit(const char* row, int c0, int c1, uint4 w[2]) {
  if (sizeof(T) == 4) {
    w[0] = *reinterpret_cast<const uint4*>(row + 4 * c0);
    w[1] = *reinterpret_cast<const uint4*>(row + 4 * c1);
  } else if (HALVES) {
    const uint2 x = *reinterpret_cast<const uint2*>(row + 2 * c0), y = *reinterpret_cast<const uint2*>(row + 2 * c1);
    w[0] = make_uint4(x.x, x.y, y.x, y.y);
  } else {
    w[0] = *reinterpret_cast<const uint4*>(row + 2 * c0);
  }
}
template <typename T, bool HALVES>
__device__ __forceinline__ void store_unit(char* row, int c0, int c1, const uint4 w[2]) {
  if (sizeof(T) == 4) {
    *reinterpret_cast<uint4*>(row + 4 * c0) = w[0];
    *reinterpret_cast<uint4*>(row + 4 * c1) = w[1];
  } else if (HALVES) {
    *reinterpret_cast<uint2*>(row + 2 * c0) = make_uint2(w[0].x, w[0].y);
    *reinterpret_cast<uint2*>(row + 2 * c1) = make_uint2(w[0].z, w[0].w);
  } else {
    *reinterpret_cast<uint4*>(row + 2 * c0) = w[0];
  }
}
template <typename T, bool HALVES>
__device__ __forceinline__ void turn_unit(uint4 w[2], const float c[4], const float s[4]) {
  float v[8];
  if (sizeof(T) == 4) {
    const float x[8] = {__uint_as_float(w[0].x), __uint_as_float(w[0].y), __uint_as_float(w[0].z), __uint_as_float(w[0].w),
                        __uint_as_float(w[1].x), __uint_as_float(w[1].y), __uint_as_float(w[1].z), __uint_as_float(w[1].w)};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = x[i];
  } else {
    const float2 x[4] = {f2(w[0].x), f2(w[0].y), f2(w[0].z), f2(w[0].w)};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = x[i].x, v[2 * i + 1] = x[i].y;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float& a = v[HALVES ? i : 2 * i];
    float& b = v[HALVES ? i + 4 : 2 * i + 1];
    const float t = a;
    a = fmaf(t, c[i], -b * s[i]);
    b = fmaf(t, s[i], b * c[i]);
  }
  if (sizeof(T) == 4) {
    w[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    w[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
  } else {
    w[0] = make_uint4(h2(v[0], v[1]), h2(v[2], v[3]), h2(v[4], v[5]), h2(v[6], v[7]));
  }
}

// One thread: one unit of HEADS heads of one row, which its cosines and sines serve.
// The angle in turns is the position times the plan's 64-bit fraction of a turn, modulo
// 2^64: exact, so far positions lose nothing, and its upper 32 bits are within 2^-33 of a
// turn.  Bound by HBM where rows are many, by a launch and two loads one after the other
// (position, row) where they are few.
template <typename T, bool HALVES, int HEADS>
__global__ void __launch_bounds__(kRopeThreads) rope_rows_kernel(const RopeRowsArgs a, const __grid_constant__ nt_rope_plan plan) {
  __shared__ uint64_t turns[128];
  for (int i = threadIdx.x; i < plan.rot_dim / 2; i += kRopeThreads) turns[i] = plan.turns[i];
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  const int groups = (a.heads + HEADS - 1) / HEADS;
  const int64_t at = int64_t(blockIdx.x) * kRopeThreads + threadIdx.x;
  const int64_t tg = at / a.units;
  const int u = int(at - tg * a.units);
  const int64_t tok = tg / groups;
  const int h0 = int(tg - tok * groups) * HEADS;
  if (tok >= a.n_tok) return;
  const bool turned = u < a.turned;
  if (!turned && a.in_place) return;
  // the unit's first channel, and that of its other half
  const int c0 = HALVES && turned ? 4 * u : 8 * u;
  const int c1 = HALVES && turned ? c0 + plan.rot_dim / 2 : c0 + 4;
  uint4 w[HEADS][2];
  char* to[HEADS];
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    int h = h0 + i;
    to[i] = nullptr;
    if (h >= a.heads) continue;
    const int j = h < a.job[0].end ? 0 : h < a.job[1].end ? 1 : 2;
    const RopeJob& job = j == 0 ? a.job[0] : j == 1 ? a.job[1] : a.job[2];
    h -= j == 0 ? 0 : j == 1 ? a.job[0].end : a.job[1].end;
    to[i] = job.y + tok * job.y_tok + h * job.y_head;
    load_unit<T, HALVES>(job.x + tok * job.x_tok + h * job.x_head, c0, c1, w[i]);
  }
  if (turned) {
    const int64_t p = a.pos ? a.pos[tok] : a.pos0 + tok;
    float c[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t t = uint64_t(p) * turns[4 * u + i];
      sincospif(float(int32_t((t + 0x80000000u) >> 32)) * 0x1p-31f, &s[i], &c[i]);
      c[i] *= plan.mag;
      s[i] *= plan.mag;
    }
#pragma unroll
    for (int i = 0; i < HEADS; ++i) turn_unit<T, HALVES>(w[i], c, s);
  }
#pragma unroll
  for (int i = 0; i < HEADS; ++i)
    if (to[i]) store_unit<T, HALVES>(to[i], c0, c1, w[i]);
}

}  // namespace

nt_status launch_rope_rows(Ctx* c, const nt_rope_plan& plan, int fmt, const nt_rope_job* jobs, int n_jobs, int64_t n_tok,
                           const int32_t* pos, int64_t pos0, cudaStream_t st) {
  RopeRowsArgs a{};
  const int size = fmt == NT_F32 ? 4 : 2;
  a.in_place = true;
  for (int i = 0; i < 3; ++i) {
    if (i < n_jobs) {
      const nt_rope_job& j = jobs[i];
      a.job[i] = {static_cast<const char*>(j.x_dev), static_cast<char*>(j.y_dev), j.x_tok_stride * size,
                  j.x_head_stride * size, j.y_tok_stride * size, j.y_head_stride * size, a.heads + j.n_heads};
      a.heads += j.n_heads;
      a.in_place = a.in_place && j.x_dev == j.y_dev;
    } else {
      a.job[i] = a.job[i - 1];
    }
  }
  a.pos = pos;
  a.pos0 = pos0;
  a.n_tok = n_tok;
  a.units = (a.in_place ? plan.rot_dim : plan.head_dim) / 8;
  a.turned = plan.rot_dim / 8;
  // One head a thread while all of them run at once (F16: half of that), where latency
  // counts (16 rows of 40 heads 1.85 us, with four heads 2.5; 480 F32 rows 4.75 and 5.2, F16
  // 4.75 and 3.9).  Else as many as keep 128 bytes in flight: the turns' cosines and sines
  // cost as much as loading three or four heads (16,381 F32 rows of 40 heads 96.7 us, 6.9
  // TB/s, with one head 114; 8191 F16 rows of 72 heads with eight 49.4, 6.1 TB/s, with four
  // 52, with one 100).
  const bool few = n_tok * a.heads * a.units <= int64_t(c->num_sms) * (fmt == NT_F32 ? 2048 : 1024);
  const int each = few ? 1 : fmt == NT_F32 ? 4 : 8;
  const int64_t threads = n_tok * ((a.heads + each - 1) / each) * a.units;
  const dim3 grid(unsigned((threads + kRopeThreads - 1) / kRopeThreads)), block(kRopeThreads);
  using K = void (*)(RopeRowsArgs, nt_rope_plan);
  const bool halves = plan.layout == NT_ROPE_HALVES;
  K k;
  if (fmt == NT_F32)
    k = few ? (halves ? K(rope_rows_kernel<float, true, 1>) : K(rope_rows_kernel<float, false, 1>))
            : (halves ? K(rope_rows_kernel<float, true, 4>) : K(rope_rows_kernel<float, false, 4>));
  else
    k = few ? (halves ? K(rope_rows_kernel<__half, true, 1>) : K(rope_rows_kernel<__half, false, 1>))
            : (halves ? K(rope_rows_kernel<__half, true, 8>) : K(rope_rows_kernel<__half, false, 8>));
  return cuda_check(c, launch_k(c, k, grid, block, 0, st, a, plan), "rope rows launch");
}

}  // namespace nt

// host arithmetic: no context, no CUDA call
extern "C" nt_status nt_rope_plan_init(const nt_rope_desc* d, nt_rope_plan* plan) {
  if (!d || !plan) return NT_ERR_INVALID_ARG;
  const auto positive = [](double x) { return x > 0 && x <= 1e300; };
  const bool scaled = d->scaling != NT_ROPE_PLAIN, long_context = d->scaling == NT_ROPE_BANDS || d->scaling == NT_ROPE_RAMP;
  if ((d->layout != NT_ROPE_PAIRS && d->layout != NT_ROPE_HALVES) || d->scaling < NT_ROPE_PLAIN || d->scaling > NT_ROPE_RAMP ||
      d->head_dim < 8 || d->head_dim > 256 || d->head_dim % 8 || d->rot_dim < 8 || d->rot_dim > d->head_dim || d->rot_dim % 8 ||
      !positive(d->theta) || d->theta == 1.0 || (scaled && !positive(d->factor)) || (long_context && !positive(d->old_len)) ||
      !(d->mag >= 0 && d->mag <= 1e30) || !(d->low >= 0 && d->low <= 1e300) || !(d->high >= 0 && d->high <= 1e300))
    return NT_ERR_INVALID_ARG;
  const double pi2 = 6.283185307179586, rot = d->rot_dim, s = scaled ? d->factor : 1.0, L = d->old_len;
  const double low = d->low > 0 ? d->low : 1.0, high = d->high > 0 ? d->high : d->scaling == NT_ROPE_RAMP ? 32.0 : 4.0;
  if (long_context && !(high > low)) return NT_ERR_INVALID_ARG;
  if (long_context && !(d->theta > 1.0)) return NT_ERR_INVALID_ARG;
  const int half = d->rot_dim / 2;
  double from = 0, to = 1;
  if (d->scaling == NT_ROPE_RAMP) {
    const auto pair = [&](double t) { return rot * std::log(L / (t * pi2)) / (2.0 * std::log(d->theta)); };
    from = std::fmax(std::floor(pair(high)), 0.0);
    to = std::fmin(std::ceil(pair(low)), rot - 1.0);
    if (!(to > from)) to = from + 0.001;
  }
  const double base = d->scaling == NT_ROPE_BASE ? d->theta * std::pow(s, rot / (rot - 2.0)) : d->theta;
  *plan = nt_rope_plan{};
  for (int i = 0; i < half; ++i) {
    double w = std::pow(base, -2.0 * i / rot);
    if (d->scaling == NT_ROPE_LINEAR) {
      w /= s;
    } else if (d->scaling == NT_ROPE_BANDS) {
      const double k = std::fmin(1.0, std::fmax(0.0, (L * w / pi2 - low) / (high - low)));
      w = w * k + w / s * (1.0 - k);
    } else if (d->scaling == NT_ROPE_RAMP) {
      const double k = std::fmin(1.0, std::fmax(0.0, (i - from) / (to - from)));
      w = w * (1.0 - k) + w / s * k;
    }
    if (d->divisors) {
      if (!positive(d->divisors[i])) return NT_ERR_INVALID_ARG;
      w /= d->divisors[i];
    }
    double turn = w / pi2;
    if (!(turn <= 1e300)) return NT_ERR_INVALID_ARG;
    turn -= std::floor(turn);
    const double scaled_turn = std::ldexp(turn, 64);  // below 2^64; a whole turn after rounding is none
    plan->turns[i] = scaled_turn >= 18446744073709551616.0 ? 0 : uint64_t(scaled_turn);
  }
  plan->layout = d->layout;
  plan->head_dim = d->head_dim;
  plan->rot_dim = d->rot_dim;
  plan->mag = float(d->mag > 0 ? d->mag : d->scaling == NT_ROPE_RAMP && s > 1.0 ? 0.1 * std::log(s) + 1.0 : 1.0);
  return NT_OK;
}
