// kv8_choose.cuh — the choice of blocks by their keys, made by one CTA of NT
// threads.  Nothing here but warp and CTA primitives, so the same source also
// runs on a host that emulates them (tests/c/choose_host.cpp), under schedules
// of the warps that a GPU rarely takes.
#pragma once
#include <cstdint>
#include <type_traits>

namespace nt {

constexpr int kSelBins = 1024;
constexpr uint32_t kForced = 0xFFFFFFFFu;  // key of a block that is taken whatever its score

// The n_sel largest of `blocks` keys, as ascending indices: radix rounds of up to
// ten bits below the keys' common prefix, ending as soon as the chosen bin is taken
// whole; once a bin holds no more keys than there are threads, later rounds look at
// those alone, one a thread; then one scan in index order.  Thread t holds blocks t K .. t K + K - 1 in
// registers (K odd, so that the threads of a warp read different banks), or re-reads
// them every time (K = 0).  key(b): the key of block b.
template <int NT>
struct SelShared {
  unsigned long long wscan[NT / 32];
  int hist[kSelBins];
  int wsum[NT / 32];
  uint32_t wmin[NT / 32], wmax[NT / 32];
  int bin, above, count, listed;
  uint32_t list[NT];
};
template <int NT, int K, typename Args, typename Key>
__device__ __forceinline__ void select_blocks(const Args& a, int blocks, int32_t* idx, SelShared<NT>& sh, Key key) {
  constexpr int W = NT / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunk = K ? K : ((blocks + NT - 1) / NT) | 1;
  const int i0 = min(blocks, tid * chunk), have = min(blocks - i0, chunk);
  uint32_t own[K ? K : 1];
#pragma unroll
  for (int j = 0; j < K; ++j) own[j] = j < have ? key(i0 + j) : 0u;
  const auto each = [&](auto fn) {
    if (K) {
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (j < have) fn(i0 + j, own[j]);
    } else {
      for (int j = 0; j < have; ++j) fn(i0 + j, key(i0 + j));
    }
  };
  int need = a.n_sel - a.n_first - a.n_last;
  uint32_t cut = kForced;  // keys above it are taken, and the first `need` at it
  if (need > 0) {
    uint32_t mn = kForced, mx = 0u;
    each([&](int, uint32_t k) {
      if (k != kForced) {
        mn = min(mn, k);
        mx = max(mx, k);
      }
    });
    mn = __reduce_min_sync(0xffffffffu, mn);
    mx = __reduce_max_sync(0xffffffffu, mx);
    if (lane == 0) {
      sh.wmin[warp] = mn;
      sh.wmax[warp] = mx;
    }
    for (int i = tid; i < kSelBins; i += NT) sh.hist[i] = 0;
    // cleared here alone: the list is made once, and a warp may begin the next round
    // before the others have read its length
    if (tid == 0) sh.listed = 0;
    __syncthreads();
    mn = __reduce_min_sync(0xffffffffu, sh.wmin[lane % W]);
    mx = __reduce_max_sync(0xffffffffu, sh.wmax[lane % W]);
    int bits = mx == mn ? 0 : 32 - __clz(mx ^ mn);
    cut = bits == 32 ? 0u : (mx >> bits) << bits;
    bool short_list = false;  // the keys in question are sh.list
    uint32_t mine = kForced;  // this thread's of them
    while (bits > 0) {
      const int dig = min(10, bits), shift = bits - dig;
      const auto count = [&](uint32_t k) {
        if (k != kForced && (bits == 32 || (k >> bits) == (cut >> bits)))
          atomicAdd(&sh.hist[(k >> shift) & ((1u << dig) - 1u)], 1);
      };
      if (short_list)
        count(mine);
      else
        each([&](int, uint32_t k) { count(k); });
      __syncthreads();
      // thread 0 holds the highest bins
      constexpr int HB = kSelBins / NT;
      int h[HB], sum = 0;
#pragma unroll
      for (int j = 0; j < HB; ++j) {
        h[j] = sh.hist[kSelBins - 1 - tid * HB - j];
        sum += h[j];
      }
      int incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      if (lane == 31) sh.wsum[warp] = incl;
      __syncthreads();
      int before = __reduce_add_sync(0xffffffffu, lane < warp ? sh.wsum[lane % W] : 0) + incl - sum;
#pragma unroll
      for (int j = 0; j < HB; ++j) {
        if (before < need && before + h[j] >= need) {
          sh.bin = kSelBins - 1 - tid * HB - j;
          sh.above = before;
          sh.count = h[j];
        }
        before += h[j];
        sh.hist[kSelBins - 1 - tid * HB - j] = 0;  // for the next round
      }
      __syncthreads();
      cut |= uint32_t(sh.bin) << shift;
      need -= sh.above;
      bits = shift;
      if (sh.count == need) {  // the whole bin: every key from here up (never all keys: n_sel < blocks)
        cut -= 1u;
        need = 0;
        break;
      }
      if (bits > 0 && !short_list && sh.count <= NT) {
        each([&](int, uint32_t k) {
          if (k != kForced && (k >> bits) == (cut >> bits)) sh.list[atomicAdd(&sh.listed, 1)] = k;
        });
        __syncthreads();
        mine = tid < sh.listed ? sh.list[tid] : kForced;
        short_list = true;
      }
    }
  }
  // blocks taken above the cut and (upper half) blocks at it; K > 0 has fewer than 2^16
  using Count = std::conditional_t<(K > 0), uint32_t, unsigned long long>;
  constexpr int H = K > 0 ? 16 : 32;
  Count cnt = 0;
  each([&](int, uint32_t k) { cnt += k == kForced || k > cut ? Count(1) : (k == cut ? Count(1) << H : Count(0)); });
  Count incl = cnt;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Count t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) sh.wscan[warp] = incl;
  __syncthreads();
  Count base = lane < warp ? Count(sh.wscan[lane % W]) : Count(0);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) base += __shfl_xor_sync(0xffffffffu, base, o);
  base += incl - cnt;
  int above = int(base & ((Count(1) << H) - 1)), ties = int(base >> H);
  each([&](int b, uint32_t k) {
    const bool over = k == kForced || k > cut;
    if (!over && (k != cut || ties >= need)) return;
    const int at = above + min(ties, need);
    if (unsigned(at) < unsigned(a.n_sel)) idx[at] = b;  // outside only if the keys changed between two reads of them (K = 0)
    if (over) ++above;
    else ++ties;
  });
}

// The same for at most NT blocks: thread b counts the keys before its own.  keys
// holds up to three more entries than blocks.
template <int NT, typename Args>
__device__ __forceinline__ void rank_blocks(const Args& a, int blocks, int32_t* idx, SelShared<NT>& sh,
                                            uint32_t* keys) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < 3) keys[blocks + tid] = 0u;  // never before a real key
  __syncthreads();
  const uint32_t own = tid < blocks ? keys[tid] : 0u;
  int rank = 0;
#pragma unroll 4
  for (int j = 0; j < blocks; j += 4) {
    const uint4 k = *reinterpret_cast<const uint4*>(keys + j);
    rank += (k.x > own || (k.x == own && j < tid)) + (k.y > own || (k.y == own && j + 1 < tid)) +
            (k.z > own || (k.z == own && j + 2 < tid)) + (k.w > own || (k.w == own && j + 3 < tid));
  }
  const bool take = tid < blocks && rank < a.n_sel;  // a forced block's key is the largest
  const unsigned m = __ballot_sync(0xffffffffu, take);
  if (lane == 0) sh.wsum[warp] = __popc(m);
  __syncthreads();
  int at = __popc(m & ((1u << lane) - 1u));
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) at += w < warp ? sh.wsum[w] : 0;
  if (take) idx[at] = tid;
}

}  // namespace nt
