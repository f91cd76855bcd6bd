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

// an inclusive sum over the block, 64 bits; `sums` has a place for each warp
__device__ __forceinline__ int64_t block_sum_to(int64_t v, int64_t* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  __syncthreads();  // the places' readers of the last sum are done
  if (lane == 31) sums[warp] = v;
  __syncthreads();
  for (int w = 0; w < warp; ++w) v += sums[w];
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One cluster of CTAs, a thread per request in each: every CTA sums the lengths by
// itself, all of them share the page lists and the rows.  Between the phases (pages
// given back, pages taken, slots) a cluster barrier orders what they wrote.
__global__ void __launch_bounds__(kMaxReq) kv4_pages_kernel(const PagesArgs a) {
  __shared__ int64_t sums[32];
  __shared__ int64_t total[2];
  __shared__ int32_t row0[kMaxReq + 1];   // the first row of each request, held to n_tok
  __shared__ int32_t from[kMaxReq];       // the position of its first row; -1 - that where it is refused
  pdl_wait();
  pdl_trigger();
  const int ranks = gridDim.x, rank = blockIdx.x, r = threadIdx.x, last = blockDim.x - 1;
  int64_t held = 0, keep = 0, n_new = 0;
  int32_t given = 0;
  bool bad = false;
  if (r < a.n_req) {
    held = given = a.held[r];
    keep = a.keep ? a.keep[r] : held;
    n_new = a.n_new[r];
  }
  const int64_t top0 = min(max(int64_t(*a.n_free), int64_t(0)), a.n_pages);
  if (held < 0 || held > a.max_pages * kPg) bad = true, held = 0, keep = 0;
  if (keep < 0 || keep > held) bad = true, keep = max(int64_t(0), min(keep, held));
  if (n_new < 0) bad = true, n_new = 0;
  if (keep + n_new > a.max_pages * kPg) bad = true;
  const int64_t have = (held + kPg - 1) / kPg, want = bad ? have : (keep + n_new + kPg - 1) / kPg;
  const int64_t back = max(int64_t(0), have - want), need = max(int64_t(0), want - have);
  const int64_t rows_to = block_sum_to(n_new, sums);
  const int64_t back_to = block_sum_to(back, sums);
  const int64_t need_to = block_sum_to(need, sums);
  if (r == last) total[0] = rows_to, total[1] = back_to;
  row0[r] = int32_t(min(rows_to - n_new, a.n_tok));
  __syncthreads();
  const int64_t rows = min(total[0], a.n_tok);
  if (r == last) row0[a.n_req] = int32_t(rows);
  // a stack that would outgrow its room holds pages twice: what does not fit is left out
  const int64_t top = min(top0 + total[1], a.n_pages);
  const bool refused = bad || (need > 0 && need_to > top);
  from[r] = int32_t(refused ? -1 - keep : keep);
  if (rank == 0 && (refused || (r == 0 && (total[0] > a.n_tok || top0 != *a.n_free || top != top0 + total[1]))))
    flag_error(a.err, kErrPaged);
  // how much the granted requests take: the largest sum that the stack still has
  const int64_t taken = block_sum_to(refused ? 0 : need, sums);

  if (ranks > 1) cluster_sync();  // every CTA has read the lengths
  if (rank == r % ranks && r < a.n_req) {
    for (int64_t j = 0; j < back; ++j)
      if (top0 + back_to - back + j < a.n_pages)
        a.free_pages[top0 + back_to - back + j] = a.table[r * a.max_pages + want + j];
    a.held_out[r] = refused ? given : int32_t(keep + n_new);
    a.q_start[r] = row0[r];
  }
  if (rank == 0 && r == last) {
    a.q_start[a.n_req] = int32_t(rows);
    *a.n_free_out = int32_t(top - taken);
  }
  if (ranks > 1) cluster_sync(); else __syncthreads();
  if (rank == r % ranks && r < a.n_req && !refused)
    for (int64_t j = 0; j < need; ++j)
      a.table[r * a.max_pages + have + j] = __ldcg(a.free_pages + top - 1 - (need_to - need) - j);
  if (ranks > 1) cluster_sync(); else __syncthreads();

  for (int64_t i = int64_t(rank) * blockDim.x + threadIdx.x; i < a.n_tok; i += int64_t(ranks) * blockDim.x) {
    int64_t slot = -1;
    int32_t pos = 0;
    if (i < rows) {
      int lo = 0, hi = a.n_req;  // row0[lo] <= i < row0[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (row0[mid] <= i) lo = mid; else hi = mid;
      }
      const int f = from[lo];
      pos = (f < 0 ? -1 - f : f) + int32_t(i - row0[lo]);
      if (f >= 0) slot = int64_t(__ldcg(a.table + lo * a.max_pages + pos / kPg)) * kPg + pos % kPg;
    }
    a.slots[i] = slot;
    a.positions[i] = pos;
  }
}

}  // namespace

nt_status launch_kv4_pages(Ctx* c, int n_req, int32_t* table, int64_t max_pages, const int32_t* held, const int32_t* keep,
                           const int32_t* n_new, int32_t* free_pages, int64_t n_pages, const int32_t* n_free,
                           int32_t* held_out, int32_t* n_free_out, int32_t* q_start, int64_t* slots, int32_t* positions,
                           int64_t n_tok, cudaStream_t st) {
  const PagesArgs a{n_req, table, max_pages, held, keep, n_new, free_pages, n_pages, n_free, held_out, n_free_out, q_start,
                    slots, positions, n_tok, c->err_flag};
  const int threads = std::max(256, (n_req + 31) / 32 * 32);
  const int ranks = n_tok > 4096 || n_req > 256 ? 8 : 1;
  return cuda_check(c, launch_cluster(c, kv4_pages_kernel, dim3(ranks), dim3(threads), 0, st, dim3(ranks, 1, 1), a),
                    "block table launch");
}

}  // namespace nt
