// Runs the packed sequences' walk (seq_walk.cuh) on the host: the 32 lanes of a warp are coroutines that meet at every
// vote or shuffle, and every offset that is read is checked against the array.
#include <ucontext.h>

#include <cstdint>
#include <cstdio>
#include <cstring>
#include <vector>

#define __device__
#define __forceinline__ inline

namespace {

constexpr int kLanes = 32;
constexpr size_t kStack = 64 * 1024;

const int* g_cu;
int g_count;      // offsets in the array
int g_bad;        // 1: read outside the array, 2: lanes at different votes, 3: no end
int64_t g_votes;  // so far
int g_lane;
int g_kind[kLanes], g_value[kLanes], g_from[kLanes], g_result[kLanes];
bool g_done[kLanes];
ucontext_t g_main, g_ctx[kLanes];

int meet(int kind, int value, int from) {
  g_kind[g_lane] = kind;
  g_value[g_lane] = value;
  g_from[g_lane] = from;
  swapcontext(&g_ctx[g_lane], &g_main);
  return g_result[g_lane];
}

int max(int a, int b) { return a > b ? a : b; }
int min(int a, int b) { return a < b ? a : b; }
int __popc(unsigned v) { return __builtin_popcount(v); }
int __ffs(unsigned v) { return __builtin_ffs(int(v)); }
unsigned __ballot_sync(unsigned, bool p) { return unsigned(meet(1, p, 0)); }
bool __any_sync(unsigned, bool p) { return meet(1, p, 0) != 0; }
int __shfl_sync(unsigned, int v, int from) { return meet(2, v, from & 31); }
int __ldg(const int* p) {
  const intptr_t at = (reinterpret_cast<intptr_t>(p) - reinterpret_cast<intptr_t>(g_cu)) / intptr_t(sizeof(int));
  if (at < 0 || at >= g_count) {
    g_bad = 1;
    return 0;
  }
  return *p;
}

}  // namespace

#include "seq_walk.cuh"

namespace {

struct Task {
  const int* cu;
  int S, L, first, step, windows;
  int *whole, *valid, *starts, *ends, *seq;
} g_task;

void lane_main() {
  using namespace mssm;
  const int lane = g_lane;
  const Task& t = g_task;
  SeqWalk walk;
  walk.start(t.cu, t.S, t.L, lane);
  for (int k = 0; k < t.windows; ++k) {
    const int wt = t.first + k * t.step, t0 = wt + lane * kGs, at = k * kLanes + lane;
    t.whole[at] = walk.enter(wt, kLanes * kGs, lane);
    const SeqMask m = walk.masks(wt, t0, lane);
    t.valid[at] = int(m.valid);
    t.starts[at] = int(m.first);
    t.ends[at] = int(m.last);
    for (int e = 0; e < kGs; ++e) t.seq[at * kGs + e] = walk.seq(m, t0, e);
  }
  g_done[lane] = true;
  swapcontext(&g_ctx[lane], &g_main);
}

}  // namespace

// The warp's windows [first + k step, + 256), k < windows, one after another.  Per window and lane: whether the window
// lies inside one sequence, the masks, and the sequence of each of the lane's steps.  Returns 0, or what went wrong.
extern "C" int walk_windows(const int* cu, int S, int L, int first, int step, int windows, int* whole, int* valid, int* starts,
                            int* ends, int* seq) {
  g_cu = cu;
  g_count = S + 1;
  g_bad = 0;
  g_votes = 0;
  g_task = Task{cu, S, L, first, step, windows, whole, valid, starts, ends, seq};
  std::vector<char> stacks(kLanes * kStack);
  for (int l = 0; l < kLanes; ++l) {
    g_done[l] = false;
    getcontext(&g_ctx[l]);
    g_ctx[l].uc_stack.ss_sp = stacks.data() + l * kStack;
    g_ctx[l].uc_stack.ss_size = kStack;
    g_ctx[l].uc_link = nullptr;
    makecontext(&g_ctx[l], lane_main, 0);
  }
  for (;;) {
    for (g_lane = 0; g_lane < kLanes; ++g_lane) swapcontext(&g_main, &g_ctx[g_lane]);
    int done = 0;
    for (int l = 0; l < kLanes; ++l) done += g_done[l];
    if (done == kLanes) return g_bad;
    for (int l = 1; l < kLanes; ++l)
      if (done || g_kind[l] != g_kind[0]) return 2;
    unsigned votes = 0;
    for (int l = 0; l < kLanes; ++l) votes |= unsigned(g_value[l] != 0) << l;
    for (int l = 0; l < kLanes; ++l) g_result[l] = g_kind[0] == 1 ? int(votes) : g_value[g_from[l]];
    if (++g_votes > 400000) return 3;
  }
}
