// pages.cu — block tables and slots of a step of several requests over a paged KV
// cache, from the requests' lengths: the bookkeeping beside the cache ("KV cache",
// fr.news.hada.io, "Fonctionnalités principales"), kept on the device so that a
// captured step needs no host.
#include <algorithm>

#include "nt_internal.cuh"
#include "ops.cuh"

namespace nt {
namespace {

constexpr int kPg = NT_KV4_PAGE;
constexpr int kMaxReq = 1024;
constexpr int64_t kManyRows = 4096;
constexpr int kPagesCluster = 16, kFewThreads = 128;

struct PagesArgs {
  int n_req;
  int32_t* table;
  int64_t max_pages;
  const int32_t *held, *keep, *n_new;
  int32_t* free_pages;
  int64_t n_pages;
  const int32_t* n_free;
  int32_t *held_out, *n_free_out, *q_start;
  int64_t* slots;
  int32_t* positions;
  int64_t n_tok;
  unsigned* err;
};

// inclusive sums over a warp of three values at once
__device__ __forceinline__ void warp_sums(int64_t v[3]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int64_t x = __shfl_up_sync(0xffffffffu, v[i], o);
      if (lane >= o) v[i] += x;
    }
}
// the same over the block; `sums` has a place for each warp, and at the end the sums up to it
__device__ __forceinline__ void block_sums(int64_t v[3], int64_t sums[][3]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  warp_sums(v);
  if (lane == 31)
#pragma unroll
    for (int i = 0; i < 3; ++i) sums[warp][i] = v[i];
  __syncthreads();
  int64_t u[3] = {0, 0, 0};
  if (lane < warp)
#pragma unroll
    for (int i = 0; i < 3; ++i) u[i] = sums[lane][i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < 3; ++i) u[i] += __shfl_xor_sync(0xffffffffu, u[i], o);
#pragma unroll
  for (int i = 0; i < 3; ++i) v[i] += u[i];
}

// what is kept of a request for the phases behind the sums
struct PageReq {
  int64_t items_to, back_to;  // pages to go through, and pages given back: sums up to this request
  int32_t keep, n_new;        // rows [keep, keep + n_new)
  int32_t row0;               // its first row, held to n_tok
  int32_t have;               // its pages before
  int64_t stack;              // page j >= have is stack entry `stack` - j
};
constexpr int64_t kRefused = INT64_MIN;  // a request's `stack`: it gets no slots

// One cluster of CTAs, a thread per request in each: every CTA sums the lengths by
// itself, all of them share the pages.  A lane has one page: it finds its request by
// the sums, takes the page from the stack if it is new, and writes the rows in it
// (its warp does, where there are many).  Bound by latency: loads, three sums, the page
// lists, the rows.
__global__ void __launch_bounds__(kMaxReq) kv4_pages_kernel(const PagesArgs a) {
  __shared__ int64_t sums[32][3];
  __shared__ int64_t total[3];
  __shared__ unsigned long long s_taken;
  __shared__ PageReq req[kMaxReq];
  const int ranks = gridDim.x, rank = blockIdx.x, r = threadIdx.x, last = blockDim.x - 1, lane = r & 31, warp = r >> 5;
  if (r == 0) s_taken = 0;
  pdl_wait();
  pdl_trigger();
  int32_t given = 0;
  int64_t keep = 0, n_new = 0;
  if (r < a.n_req) {
    given = a.held[r];
    keep = a.keep ? a.keep[r] : given;
    n_new = a.n_new[r];
  }
  const int64_t free0 = *a.n_free, top0 = min(max(free0, int64_t(0)), a.n_pages), cap = a.max_pages * kPg;
  // the lengths are read: the others may write over them
  if (ranks > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  int64_t held = given;
  bool bad = held < 0 || held > cap;
  if (bad) held = 0;
  if (keep < 0 || keep > held) bad = true, keep = max(int64_t(0), min(keep, held));
  if (n_new < 0) bad = true, n_new = 0;
  bad = bad || keep + n_new > cap;
  const int64_t have = (held + kPg - 1) / kPg, want = bad ? have : (keep + n_new + kPg - 1) / kPg;
  const int64_t back = max(int64_t(0), have - want), need = max(int64_t(0), want - have);
  int64_t v[3] = {n_new, back, need};
  block_sums(v, sums);
  if (r == last) total[0] = v[0], total[1] = v[1], total[2] = v[2];
  __syncthreads();
  const int64_t rows = min(total[0], a.n_tok), released = total[1];
  // a stack that would outgrow its room holds pages twice: what does not fit is left out
  const int64_t top = min(top0 + released, a.n_pages);
  const bool refused = bad || (need > 0 && v[2] > top);
  if (rank == 0 && (refused || (r == 0 && (total[0] > a.n_tok || top0 != free0 || top != top0 + released))))
    flag_error(a.err, kErrPaged);
  if (need > 0 && !refused) atomicMax(&s_taken, static_cast<unsigned long long>(v[2]));
  const int64_t row0 = min(v[0] - n_new, a.n_tok), shown = min(n_new, a.n_tok - row0);
  // pages to go through: those of its rows (as far as they are written), and all new ones
  const int64_t first = keep / kPg, until = max((keep + shown + kPg - 1) / kPg, refused ? int64_t(0) : need ? want : int64_t(0));
  const int64_t items = n_new > 0 ? max(int64_t(0), until - first) : 0;
  int64_t u[3] = {items, 0, 0};
  __syncthreads();  // the sums' places are read
  block_sums(u, sums);
  if (r < a.n_req)
    req[r] = {u[0], v[1], int32_t(keep), int32_t(min(n_new, int64_t(0x7FFFFFFF) - keep)), int32_t(row0), int32_t(have),
              refused ? kRefused : top - 1 - (v[2] - need) + have};
  if (ranks > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (rank == 0 && r < a.n_req) {
    a.held_out[r] = refused ? given : int32_t(keep + n_new);
    a.q_start[r] = int32_t(row0);
  }
  __syncthreads();
  if (rank == 0 && r == 0) {
    a.q_start[a.n_req] = int32_t(rows);
    *a.n_free_out = int32_t(top - int64_t(s_taken));
  }
  const int W = blockDim.x / 32, at0 = rank * W + warp, step = ranks * W;
  // the request whose sum is the first above i
  const auto find = [&](int64_t i, int64_t PageReq::*to) {
    int lo = -1, hi = a.n_req - 1;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (req[mid].*to > i) hi = mid; else lo = mid;
    }
    return hi;
  };
  if (released) {  // (the same for every CTA)
    for (int64_t i = int64_t(at0) * 32 + lane; i < released; i += int64_t(step) * 32) {
      const int q = find(i, &PageReq::back_to);
      const int64_t j = req[q].have - (req[q].back_to - i);  // its pages want .. have - 1
      if (top0 + i < a.n_pages) a.free_pages[top0 + i] = a.table[q * a.max_pages + j];
    }
    if (ranks > 1)
      asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    else
      __syncthreads();
  }
  const int64_t all = req[a.n_req - 1].items_to;
  const int share = int(min(int64_t(32), (all + step - 1) / step));  // pages a warp has at a time
  for (int64_t i0 = int64_t(at0) * share; i0 < all; i0 += int64_t(step) * share) {
    int32_t row = 0, pos = 0, count = 0, entry = -1;
    if (lane < share && i0 + lane < all) {
      const int q = find(i0 + lane, &PageReq::items_to);
      const PageReq x = req[q];
      const int64_t before = q ? req[q - 1].items_to : 0;
      const int64_t p = x.keep / kPg + (i0 + lane - before);
      if (x.stack != kRefused) {
        if (p < x.have) {
          entry = a.table[q * a.max_pages + p];
        } else {
          entry = __ldcg(a.free_pages + x.stack - p);
          a.table[q * a.max_pages + p] = entry;
        }
      }
      const int64_t lo = max(int64_t(x.keep), p * kPg), hi = min(int64_t(x.keep) + x.n_new, p * kPg + kPg);
      const int64_t at = x.row0 + (lo - x.keep);
      pos = int32_t(lo);
      row = int32_t(min(at, a.n_tok));
      count = int32_t(max(int64_t(0), min(hi - lo, a.n_tok - at)));
    }
    if (!__any_sync(0xffffffffu, count > 4)) {  // a few rows each
      for (int k = 0; k < count; ++k) {
        a.slots[row + k] = entry < 0 ? -1 : int64_t(entry) * kPg + (pos + k) % kPg;
        a.positions[row + k] = pos + k;
      }
      continue;
    }
    for (int k = 0; k < share; ++k) {
      const int n = __shfl_sync(0xffffffffu, count, k);
      if (n == 0) continue;
      const int64_t row_k = __shfl_sync(0xffffffffu, row, k);
      const int pos_k = __shfl_sync(0xffffffffu, pos, k), entry_k = __shfl_sync(0xffffffffu, entry, k);
      const int64_t slot = int64_t(entry_k) * kPg + pos_k % kPg;
#pragma unroll
      for (int i = lane; i < kPg; i += 32)
        if (i < n) {
          a.slots[row_k + i] = entry_k < 0 ? -1 : slot + i;
          a.positions[row_k + i] = pos_k + i;
        }
    }
  }
  for (int64_t i = rows + at0 * 32 + lane; i < a.n_tok; i += int64_t(step) * 32) {
    a.slots[i] = -1;
    a.positions[i] = 0;
  }
}

}  // namespace

nt_status launch_kv4_pages(Ctx* c, int n_req, int32_t* table, int64_t max_pages, const int32_t* held, const int32_t* keep,
                           const int32_t* n_new, int32_t* free_pages, int64_t n_pages, const int32_t* n_free,
                           int32_t* held_out, int32_t* n_free_out, int32_t* q_start, int64_t* slots, int32_t* positions,
                           int64_t n_tok, cudaStream_t st) {
  const PagesArgs a{n_req, table, max_pages, held, keep, n_new, free_pages, n_pages, n_free, held_out, n_free_out, q_start,
                    slots, positions, n_tok, c->err_flag};
  // one CTA where the rows are few, else sixteen, an SM each
  const bool many = n_tok > kManyRows;
  const int ranks = many ? kPagesCluster : 1;
  const int threads = many ? kMaxReq : std::max(kFewThreads, (n_req + 31) / 32 * 32);
  return cuda_check(c, launch_cluster(c, kv4_pages_kernel, dim3(ranks), dim3(threads), 0, st, dim3(ranks, 1, 1), a),
                    "block table launch");
}

nt_status configure_pages(Ctx* c) {
  return cuda_check(c, cudaFuncSetAttribute(kv4_pages_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1),
                    "block table cluster attribute");
}

}  // namespace nt
