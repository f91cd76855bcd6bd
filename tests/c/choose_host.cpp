// Runs the choice of blocks (csrc/kv8_choose.cuh) on the host: every thread of
// the CTA is a fiber, warp and CTA primitives are rendezvous, and a schedule says
// who runs next.  Between two rendezvous nothing orders the threads of a CTA, so
// the result has to be the same under every schedule:
//   low    the lowest runnable thread first: thread 0's warp runs ahead of all others
//   high   the highest first: thread 0's warp is the last everywhere
//   mixed  a random one, and random changes at every atomic and key read
//   torn   mixed, and the keys change between reads, as if another call wrote the
//          scratch that holds them: any list may come out, but nothing beside it is written
// Reads cases from stdin:  threads K n_sel n_first n_last blocks schedule seed, then the keys;
// writes the n_sel entries, then 1 if anything beside them was written.
#include <ucontext.h>

#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <functional>
#include <random>
#include <string>
#include <vector>

#define __device__
#define __forceinline__ inline

namespace emu {
struct Dim { unsigned x; } tid;
enum Schedule { kLow, kHigh, kMixed } schedule;
bool torn;
int n;
std::mt19937 rng;
ucontext_t home;
constexpr size_t kStack = 128 << 10;
struct Fiber {
  ucontext_t ctx;
  bool done;
  const unsigned* gate;  // waits until *gate differs from seen
  unsigned seen;
};
std::vector<Fiber> fibers;
std::vector<char> stacks;
struct Warp {
  unsigned long long slot[2][32];
  unsigned gen;
  int arrived;
};
std::vector<Warp> warps;
unsigned cta_gen;
int cta_arrived;
std::function<void()> body;

bool runnable(const Fiber& f) { return !f.done && !(f.gate && *f.gate == f.seen); }
void pause() {
  const unsigned me = tid.x;
  swapcontext(&fibers[me].ctx, &home);
}
void wait_on(const unsigned* gate, unsigned seen) {
  Fiber& f = fibers[tid.x];
  f.gate = gate;
  f.seen = seen;
  pause();
  f.gate = nullptr;
}
void maybe_yield() {
  if (schedule == kMixed && rng() % 4 == 0) pause();
}
void entry() {
  body();
  fibers[tid.x].done = true;
  swapcontext(&fibers[tid.x].ctx, &home);
}
void run(int threads, std::function<void()> fn) {
  n = threads;
  body = std::move(fn);
  fibers.assign(n, Fiber{});
  warps.assign(n / 32, Warp{});
  stacks.resize(n * kStack);
  cta_gen = 0;
  cta_arrived = 0;
  for (int i = 0; i < n; ++i) {
    getcontext(&fibers[i].ctx);
    fibers[i].ctx.uc_stack.ss_sp = stacks.data() + i * kStack;
    fibers[i].ctx.uc_stack.ss_size = kStack;
    fibers[i].ctx.uc_link = &home;
    makecontext(&fibers[i].ctx, entry, 0);
  }
  for (int left = n; left;) {
    int pick = -1;
    const int from = schedule == kMixed ? int(rng() % n) : 0;
    for (int j = 0; j < n && pick < 0; ++j) {
      const int i = schedule == kHigh ? n - 1 - j : (from + j) % n;
      if (runnable(fibers[i])) pick = i;
    }
    if (pick < 0) {
      std::puts("deadlock");
      std::exit(1);
    }
    tid.x = unsigned(pick);
    swapcontext(&home, &fibers[pick].ctx);
    left -= fibers[pick].done;
  }
}

// every lane of the warp brings v; returns the 32 values
template <typename T>
void exchange(T v, T out[32]) {
  Warp& w = warps[tid.x >> 5];
  const unsigned gen = w.gen, lane = tid.x & 31u;
  w.slot[gen & 1][lane] = static_cast<unsigned long long>(v);
  if (++w.arrived == 32) {
    w.arrived = 0;
    ++w.gen;
    if (schedule == kMixed) pause();
  } else {
    wait_on(&w.gen, gen);
  }
  Warp& x = warps[tid.x >> 5];
  for (int i = 0; i < 32; ++i) out[i] = T(x.slot[gen & 1][i]);
}
}  // namespace emu

#define threadIdx emu::tid
using std::max;
using std::min;
struct alignas(16) uint4 { unsigned x, y, z, w; };

inline void __syncthreads() {
  const unsigned gen = emu::cta_gen;
  if (++emu::cta_arrived == emu::n) {
    emu::cta_arrived = 0;
    ++emu::cta_gen;
    emu::pause();
  } else {
    emu::wait_on(&emu::cta_gen, gen);
  }
}
template <typename T>
T __shfl_up_sync(unsigned, T v, int d) {
  T all[32];
  emu::exchange(v, all);
  const int lane = emu::tid.x & 31;
  return all[lane >= d ? lane - d : lane];
}
template <typename T>
T __shfl_xor_sync(unsigned, T v, int d) {
  T all[32];
  emu::exchange(v, all);
  return all[(emu::tid.x & 31) ^ d];
}
template <typename T>
T __reduce_min_sync(unsigned, T v) {
  T all[32];
  emu::exchange(v, all);
  return *std::min_element(all, all + 32);
}
template <typename T>
T __reduce_max_sync(unsigned, T v) {
  T all[32];
  emu::exchange(v, all);
  return *std::max_element(all, all + 32);
}
template <typename T>
T __reduce_add_sync(unsigned, T v) {
  T all[32], s = 0;
  emu::exchange(v, all);
  for (T x : all) s += x;
  return s;
}
inline unsigned __ballot_sync(unsigned, bool v) {
  unsigned all[32], m = 0;
  emu::exchange(unsigned(v), all);
  for (int i = 0; i < 32; ++i) m |= all[i] << i;
  return m;
}
inline int __popc(unsigned v) { return __builtin_popcount(v); }
inline int __clz(unsigned v) { return v ? __builtin_clz(v) : 32; }
inline int atomicAdd(int* p, int v) {
  emu::maybe_yield();
  const int old = *p;
  *p += v;
  return old;
}

#include "kv8_choose.cuh"

struct Args { int n_sel, n_first, n_last; };

template <int NT>
void choose(const Args& a, int K, int blocks, int32_t* idx, uint32_t* keys) {
  static nt::SelShared<NT> sh;
  std::generate_n(reinterpret_cast<unsigned char*>(&sh), sizeof sh, [] { return (unsigned char)emu::rng(); });
  const auto key = [&](int b) {
    emu::maybe_yield();
    return keys[emu::torn && emu::rng() % 2 ? (b * 7LL + 3) % blocks : b];
  };
  emu::run(NT, [&] {
    if (K < 0) nt::rank_blocks<NT>(a, blocks, idx, sh, keys);
    else if (K == 1) nt::select_blocks<NT, 1>(a, blocks, idx, sh, key);
    else if (K == 5) nt::select_blocks<NT, 5>(a, blocks, idx, sh, key);
    else nt::select_blocks<NT, 0>(a, blocks, idx, sh, key);
  });
}

int main() {
  int threads, K, blocks, sched;
  unsigned seed;
  Args a;
  while (std::scanf("%d %d %d %d %d %d %d %u", &threads, &K, &a.n_sel, &a.n_first, &a.n_last, &blocks, &sched, &seed) == 8) {
    emu::torn = sched == 3;
    emu::schedule = emu::Schedule(emu::torn ? 2 : sched);
    emu::rng.seed(seed);
    std::vector<uint4> store((blocks + 3) / 4 + 1);
    uint32_t* keys = reinterpret_cast<uint32_t*>(store.data());
    for (int b = 0; b < blocks; ++b)
      if (std::scanf("%u", keys + b) != 1) return 2;
    const int guard = 2 * blocks + 64;  // a cut that is too low takes up to `blocks` entries
    std::vector<int32_t> idx(a.n_sel + 2 * guard, -7);
    if (threads == 256) choose<256>(a, K, blocks, idx.data() + guard, keys);
    else choose<1024>(a, K, blocks, idx.data() + guard, keys);
    for (int i = 0; i < a.n_sel; ++i) std::printf("%d ", idx[guard + i]);
    const bool beside = std::any_of(idx.begin(), idx.begin() + guard, [](int32_t v) { return v != -7; }) ||
                        std::any_of(idx.end() - guard, idx.end(), [](int32_t v) { return v != -7; });
    std::printf("%d\n", int(beside));
  }
}
