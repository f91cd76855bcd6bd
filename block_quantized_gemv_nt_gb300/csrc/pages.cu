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
// Above so many rows a launch of their own writes them, from all SMs, and the tables take a
// cluster: the lists' round trips then run side by side (250 mixed requests with 153,000
// rows: a cluster of 16 writing all 10.0 us, two launches 8.7, with 8 CTAs 9.6, with
// 2 13.8; 1024 requests with 550,000 rows 16.6, 11.1, 11.8, 14.8).
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

__device__ __forceinline__ uint32_t warp_sum_to(uint32_t v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}
// Inclusive sums over the block of N values at once.  A warp's own sum counts for the
// warps behind it as `most` at most (above every bound that the sums are held against),
// so that 32 of them fit 32 bits; `sums` has a place for each warp.
template <int N>
__device__ __forceinline__ void block_sums(uint32_t (&v)[N], const uint32_t (&most)[N], uint32_t sums[][3]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum_to(v[i]);
  if (lane == 31)
#pragma unroll
    for (int i = 0; i < N; ++i) sums[warp][i] = min(v[i], most[i]);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] += __reduce_add_sync(0xffffffffu, lane < warp ? sums[lane][i] : 0u);
}

// what is kept of a request for the phases behind the sums
struct PageReq {
  uint32_t items_to, back_to;  // pages to go through, and pages given back: sums up to this request
  int32_t keep, n_new;         // rows [keep, keep + n_new)
  int32_t row0;                // its first row, held to n_tok
  int32_t have, first, until;  // pages before; pages to go through
  int32_t stack;               // page j >= have is stack entry `stack` - j
};
constexpr int32_t kRefused = INT32_MIN;  // a request's `stack`: it gets no slots

// One cluster of CTAs, a thread per request in each: every CTA sums the lengths by
// itself, all of them share the pages.  A lane has one page: it finds its request by
// the sums, takes the page from the stack if it is new, and writes the rows in it
// (its warp does, where there are many).  ROWS false: of each request's rows only the first
// is written, which tells the launch behind this one where they stand.  Bound by latency:
// loads, sums, page lists, rows.
template <bool ROWS>
__global__ void __launch_bounds__(kMaxReq) kv4_pages_kernel(const PagesArgs a) {
  __shared__ uint32_t sums[32][3];
  __shared__ uint32_t total[2];
  __shared__ uint32_t s_taken;
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
  const int32_t free0 = *a.n_free;
  const int n_pages = int(a.n_pages), n_tok = int(a.n_tok), top0 = min(max(free0, 0), n_pages);
  const int64_t cap = a.max_pages * kPg;
  // the lengths are read: the others may write over them
  if (ranks > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  int64_t held = given;
  bool bad = held < 0 || held > cap;
  if (bad) held = 0;
  if (keep < 0 || keep > held) bad = true, keep = max(int64_t(0), min(keep, held));
  if (n_new < 0) bad = true, n_new = 0;
  bad = bad || keep + n_new > cap;
  const int have = int((held + kPg - 1) / kPg), want = bad ? have : int((keep + n_new + kPg - 1) / kPg);
  const uint32_t back = max(0, have - want), need = max(0, want - have), n = uint32_t(min(n_new, int64_t(n_tok) + 1));
  uint32_t v[3] = {n, back, need};
  const uint32_t most[3] = {uint32_t(n_tok) + 1, uint32_t(n_pages) + 1, uint32_t(n_pages) + 1};
  block_sums(v, most, sums);
  if (r == last) total[0] = v[0], total[1] = v[1];
  __syncthreads();
  const int rows = int(min(total[0], uint32_t(n_tok)));
  const uint32_t released = total[1];
  // a stack that would outgrow its room holds pages twice: what does not fit is left out
  const int top = int(min(uint32_t(top0) + released, uint32_t(n_pages)));
  const bool refused = bad || (need > 0 && v[2] > uint32_t(top));
  if (rank == 0 && (refused || (r == 0 && (total[0] > uint32_t(n_tok) || top0 != free0 || uint32_t(top) != uint32_t(top0) + released))))
    flag_error(a.err, kErrPaged);
  if (need > 0 && !refused) atomicMax(&s_taken, v[2]);
  const int row0 = int(min(v[0] - n, uint32_t(n_tok))), shown = int(min(int64_t(n), int64_t(n_tok) - row0));
  // pages to go through: those of the rows that are written, and all new ones
  int first = int(keep / kPg), until = int((keep + shown + kPg - 1) / kPg);
  if (!shown) first = until = have;
  if (!ROWS) first = until = have;
  if (need && !refused) until = max(until, want);
  uint32_t u[1] = {uint32_t(max(0, until - first))};
  const uint32_t all_most[1] = {1u << 27};  // above the pages of the pool and of the rows together
  __syncthreads();  // the sums' places are read
  block_sums(u, all_most, sums);
  if (r < a.n_req)
    req[r] = {u[0], v[1], int32_t(keep), shown, row0, have, first, until,
              refused ? kRefused : top - 1 - int(v[2] - need) + have};
  if (ranks > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (rank == 0 && r < a.n_req) {
    a.held_out[r] = refused ? given : int32_t(keep + n_new);
    a.q_start[r] = row0;
  }
  __syncthreads();
  if (rank == 0 && r == 0) {
    a.q_start[a.n_req] = rows;
    *a.n_free_out = top - int(s_taken);
  }
  const int W = blockDim.x / 32, at0 = rank * W + warp, step = ranks * W;
  // the request whose sum is the first above i
  const auto find = [&](uint32_t i, uint32_t PageReq::*to) {
    int lo = -1, hi = a.n_req - 1;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (req[mid].*to > i) hi = mid; else lo = mid;
    }
    return hi;
  };
  if (released) {  // (the same for every CTA)
    const int fits = top - top0;
    for (int i = at0 * 32 + lane; i < fits; i += step * 32) {
      const int q = find(i, &PageReq::back_to);
      const int j = req[q].have - int(req[q].back_to - i);  // its pages want .. have - 1
      if (j >= 0) a.free_pages[top0 + i] = a.table[q * a.max_pages + j];
    }
    if (ranks > 1)
      asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    else
      __syncthreads();
  }
  // page p of request q
  const auto entry_of = [&](const PageReq& x, int q, int p) {
    if (x.stack == kRefused) return -1;
    return p < x.have ? a.table[q * a.max_pages + p] : __ldcg(a.free_pages + x.stack - p);
  };
  if (!ROWS && r < a.n_req && r % ranks == rank) {
    const PageReq x = req[r];
    if (x.n_new) {
      const int e = entry_of(x, r, x.keep / kPg);
      a.slots[x.row0] = e < 0 ? -1 : int64_t(e) * kPg + x.keep % kPg;
      a.positions[x.row0] = x.keep;
    }
  }
  const int all = int(min(req[a.n_req - 1].items_to, uint32_t(INT32_MAX)));
  const int share = min(32, (all + step - 1) / step);  // pages a warp has at a time
  for (int i0 = at0 * share; i0 < all; i0 += step * share) {
    int row = 0, pos = 0, count = 0, entry = -1;
    if (lane < share && i0 + lane < all) {
      const int q = find(i0 + lane, &PageReq::items_to);
      const PageReq x = req[q];
      const int p = x.first + (i0 + lane - int(q ? req[q - 1].items_to : 0u));
      if (p < x.until) {
        entry = entry_of(x, q, p);
        if (p >= x.have && x.stack != kRefused) a.table[q * a.max_pages + p] = entry;
        const int64_t lo = max(x.keep, p * kPg), hi = min(int64_t(x.keep) + x.n_new, int64_t(p) * kPg + kPg);
        pos = int(lo);
        row = x.row0 + int(lo) - x.keep;
        count = ROWS ? int(max(int64_t(0), hi - lo)) : 0;
      }
    }
    if constexpr (ROWS) {
      if (!__any_sync(0xffffffffu, count > 4)) {  // a few rows each
        for (int k = 0; k < count; ++k) {
          a.slots[row + k] = entry < 0 ? -1 : int64_t(entry) * kPg + (pos + k) % kPg;
          a.positions[row + k] = pos + k;
        }
        continue;
      }
      for (int k = 0; k < share; ++k) {
        const int n_k = __shfl_sync(0xffffffffu, count, k);
        if (n_k == 0) continue;
        const int row_k = __shfl_sync(0xffffffffu, row, k);
        const int pos_k = __shfl_sync(0xffffffffu, pos, k), entry_k = __shfl_sync(0xffffffffu, entry, k);
        const int64_t slot = int64_t(entry_k) * kPg + pos_k % kPg;
#pragma unroll
        for (int i = lane; i < kPg; i += 32)
          if (i < n_k) {
            a.slots[row_k + i] = entry_k < 0 ? -1 : slot + i;
            a.positions[row_k + i] = pos_k + i;
          }
      }
    }
  }
  if constexpr (ROWS) {
    for (int i = rows + at0 * 32 + lane; i < n_tok; i += step * 32) {
      a.slots[i] = -1;
      a.positions[i] = 0;
    }
  }
}

// The rows of a step with many: each finds its request by q_start, where that stands by its
// first row, and its page in the table.  (A first row is written once more, as it is.)
constexpr int kRowsThreads = 256, kRowsEach = 4;
__global__ void __launch_bounds__(kRowsThreads) kv4_page_rows_kernel(const PagesArgs a) {
  __shared__ int32_t start[kMaxReq + 1];
  pdl_wait();
  pdl_trigger();
  for (int i = threadIdx.x; i <= a.n_req; i += kRowsThreads) start[i] = a.q_start[i];
  __syncthreads();
  const int rows = start[a.n_req], n_tok = int(a.n_tok);
  const int i0 = blockIdx.x * (kRowsThreads * kRowsEach) + threadIdx.x;
  int q[kRowsEach], pos[kRowsEach];
  int64_t slot[kRowsEach];
#pragma unroll
  for (int k = 0; k < kRowsEach; ++k) {
    const int i = i0 + k * kRowsThreads;
    int lo = 0, hi = a.n_req;  // start[lo] <= i < start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= i) lo = mid; else hi = mid;
    }
    q[k] = lo;
    slot[k] = -1;
    pos[k] = 0;
    if (i < rows) {
      pos[k] = __ldcg(a.positions + start[lo]) + (i - start[lo]);
      slot[k] = __ldcg(a.slots + start[lo]);
    }
  }
#pragma unroll
  for (int k = 0; k < kRowsEach; ++k)
    if (slot[k] >= 0) slot[k] = int64_t(__ldcg(a.table + q[k] * a.max_pages + pos[k] / kPg)) * kPg + pos[k] % kPg;
#pragma unroll
  for (int k = 0; k < kRowsEach; ++k) {
    const int i = i0 + k * kRowsThreads;
    if (i >= n_tok) continue;
    a.slots[i] = slot[k];
    a.positions[i] = pos[k];
  }
}

}  // namespace

nt_status launch_kv4_pages(Ctx* c, int n_req, int32_t* table, int64_t max_pages, const int32_t* held, const int32_t* keep,
                           const int32_t* n_new, int32_t* free_pages, int64_t n_pages, const int32_t* n_free,
                           int32_t* held_out, int32_t* n_free_out, int32_t* q_start, int64_t* slots, int32_t* positions,
                           int64_t n_tok, cudaStream_t st) {
  const PagesArgs a{n_req, table, max_pages, held, keep, n_new, free_pages, n_pages, n_free, held_out, n_free_out, q_start,
                    slots, positions, n_tok, c->err_flag};
  const int threads = std::max(kFewThreads, (n_req + 31) / 32 * 32);
  if (n_tok <= kManyRows)
    return cuda_check(c, launch_k(c, kv4_pages_kernel<true>, dim3(1), dim3(threads), 0, st, a), "block table launch");
  nt_status s = cuda_check(c, launch_cluster(c, kv4_pages_kernel<false>, dim3(kPagesCluster), dim3(threads), 0, st,
                                             dim3(kPagesCluster, 1, 1), a),
                           "block table launch");
  if (s) return s;
  const int per = kRowsThreads * kRowsEach;
  return cuda_check(c, launch_k(c, kv4_page_rows_kernel, dim3(unsigned((n_tok + per - 1) / per)), dim3(kRowsThreads), 0, st, a),
                    "slot launch");
}

nt_status configure_pages(Ctx* c) {
  return cuda_check(c, cudaFuncSetAttribute(kv4_pages_kernel<false>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1),
                    "block table cluster attribute");
}

}  // namespace nt
