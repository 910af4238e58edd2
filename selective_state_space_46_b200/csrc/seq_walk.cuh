// Packed sequences: which steps of a thread's window belong to which sequence.  Plain integer arithmetic and warp
// votes, without a CUDA header, so that it can also be compiled for the host and run there lane by lane.
#pragma once

namespace mssm {

constexpr int kGs = 8;  // steps per thread

// The thread's steps [t0, t0 + kGs) that lie in [from, to), where 0 <= from, to < 2^31 - 2^16 and t0 > -2^16
// (so that no difference wraps): bit j for step t0 + j.  Stores rely on it to stay inside the row.
__device__ __forceinline__ unsigned steps_inside(int t0, int from, int to) {
  const int lo = max(from - t0, 0), hi = min(to - t0, kGs);
  return hi > lo ? ((1u << kGs) - 1u) >> (kGs - hi) & ~((1u << lo) - 1u) : 0u;
}

// The largest j in [0, S) with cu[j] <= t (0 if there is none), whatever the offsets hold.
__device__ __forceinline__ int seq_of(const int* cu, int S, int t) {
  int lo = 0, hi = S + 1;
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (__ldg(cu + mid) <= t) lo = mid + 1;
    else hi = mid;
  }
  return max(min(lo - 1, S - 1), 0);
}

// What a window holds of the packed sequences: bit j for step t0 + j.
struct SeqMask {
  unsigned valid, first, last;  // inside a sequence; its first step; its last step
  unsigned offs;                // steps with an offset
  int below;                    // offsets before t0
  bool twice;                   // some step has more than one offset (an empty sequence)
};

// A warp's walk through the offsets, 32 of them in its lanes.  Offsets that are out of order give wrong
// sequences in [0, S) and an end to every loop.
struct SeqWalk {
  const int* cu;
  int S, c0, cS;  // the first and last offset, inside the row whatever they hold
  int base, v;    // the lane's offset is number base + lane

  __device__ __forceinline__ int get(int j) const { return j <= S ? __ldg(cu + j) : 0x7fffffff; }
  __device__ __forceinline__ void start(const int* offsets, int n, int L, int lane) {
    cu = offsets;
    S = n;
    c0 = max(min(__ldg(cu), L), 0);
    cS = max(min(__ldg(cu + n), L), 0);
    base = 0;
    v = get(lane);
  }
  // To the warp's steps [wt, wt + n), up or down the row.  Says whether they lie inside one sequence, with no
  // first or last step.  Neighbouring blocks of offsets share one, so that the last offset in front of the steps and
  // the first behind it are always in the lanes together, also at a block's end.
  __device__ __forceinline__ bool enter(int wt, int n, int lane) {
    unsigned below = __ballot_sync(~0u, v < wt);
    while (below == ~0u) {
      base += 31;
      v = get(base + lane);
      below = __ballot_sync(~0u, v < wt);
    }
    while (below == 0u && base > 0) {
      base -= 31;
      v = get(base + lane);
      below = __ballot_sync(~0u, v < wt);
    }
    const int before = base + __popc(below);
    return !__any_sync(~0u, v >= wt && v <= wt + n) && before >= 1 && before <= S;
  }
  __device__ __forceinline__ SeqMask masks(int wt, int t0, int lane) const {
    SeqMask m{steps_inside(t0, c0, cS), 0u, 0u, 0u, 0, false};
    const int te = wt + 32 * kGs;
    m.below = base + __popc(__ballot_sync(~0u, v < wt));
    int o32 = v;
    for (int at = base;;) {
      unsigned in = __ballot_sync(~0u, o32 >= wt && o32 <= te);
      while (in) {
        const int o = __shfl_sync(~0u, o32, __ffs(in) - 1) - t0;
        in &= in - 1;
        if (o < 0) ++m.below;
        if (o >= 0 && o < kGs) {
          m.twice |= m.offs >> o & 1u;
          m.offs |= 1u << o;
        }
        if (o >= 1 && o <= kGs) m.last |= 1u << (o - 1);
      }
      if (__any_sync(~0u, o32 > te)) break;
      at += 32;
      o32 = get(at + lane);
    }
    m.first = m.offs & m.valid;
    m.last &= m.valid;
    return m;
  }
  // the sequence of step t0 + k
  __device__ __forceinline__ int seq(const SeqMask& m, int t0, int k) const {
    if (m.twice) return seq_of(cu, S, t0 + k);
    return max(min(m.below + __popc(m.offs & ((2u << k) - 1u)) - 1, S - 1), 0);
  }
};

}  // namespace mssm
