// The real-gated linear recurrence: forward scan, backward scan and decode step (sm_100a).
//
//   r = sigmoid(r_raw + r_bias), i = sigmoid(i_raw + i_bias), rate = c softplus(lam)
//   a_t = exp(-rate r_t), beta_t = sqrt(1 - a_t^2), h_t = a_t h_(t-1) + beta_t i_t x_t
//   out_t = h_t silu(z_t)                                               (z optional)
//
// One state per channel, so unlike the 16-state selective scan the path is a stream: 8 bytes of
// bf16 I/O per element (10 with z) against five (six) SFU results.  A row's steps run along the
// lanes: every thread holds kGs consecutive steps (one 16-byte vector of bf16), reduces them to
// the affine map h -> A h + B, and the maps are composed by warp shuffles, across warps through
// shared memory, and from tile to tile by a carry in registers.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "device_common.cuh"

namespace mssm {

constexpr int kGs = 8;             // steps per thread
constexpr float kResetA = -0.0f;   // the decay of a sequence's first step: composes to "ignore what came before"

struct GatedArgs {
  const void *x, *r, *i, *z;       // [Bt, D, L], length stride 1; z may be null
  int64_t x_sb, x_sd, r_sb, r_sd, i_sb, i_sd, z_sb, z_sd;
  void* out;                       // forward: [Bt, D, L]
  int64_t o_sb, o_sd;
  const float *lam, *rb, *ib;      // [D]; biases may be null
  int64_t lam_s, rb_s, ib_s;
  float c;
  const float* h0;                 // [S, D] or null
  int64_t h0_sb, h0_sd;
  float* last;                     // forward: [S, D] or null
  int64_t ls_sb, ls_sd;
  const int* cu;                   // [S + 1] or null: packed sequences of a [1, D, L] row
  int S, Bt, D, L;
  unsigned* err;                   // device error word: bit 2 = inconsistent cu_seqlens
  // backward
  const void* dout;                // [Bt, D, L]
  int64_t g_sb, g_sd;
  const float* dlast;              // [S, D] or null
  int64_t dl_sb, dl_sd;
  void *dx, *dr, *di, *dz;         // [Bt, D, L]
  int64_t dx_sb, dx_sd, dr_sb, dr_sd, di_sb, di_sd, dz_sb, dz_sd;
  float* dh0;                      // [S, D] or null
  int64_t dh_sb, dh_sd;
  float *dlam, *drb, *dib;         // [D] (biases' may be null)
  float* part;                     // [3, Bt, D] row sums of the three when Bt > 1
  int ntiles;                      // tiles of a row and CTA (backward: checkpoints in shared memory)
  int split;                       // CTAs (a cluster) that share a row
};

struct GatedStepArgs {
  float* state;                    // [Bt, D]
  int64_t st_sb, st_sd;
  const void *x, *r, *i, *z;       // [Bt, D]; z may be null
  int64_t x_sb, x_sd, r_sb, r_sd, i_sb, i_sd, z_sb, z_sd;
  void* out;
  int64_t o_sb, o_sd;
  const float *lam, *rb, *ib;
  int64_t lam_s, rb_s, ib_s;
  float c;
  int Bt, D;
};

// ---------------------------------------------------------------- gates and decays

__device__ __forceinline__ float rsqrt_approx(float x) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ f2_t f2s(float v) { return f2(v, v); }

// softplus and the logistic function of a per-channel parameter, once per row: the accurate
// library functions (the rate's relative error multiplies every decay's logarithm).
__device__ __forceinline__ float softplus_exact(float v) { return fmaxf(v, 0.0f) + log1pf(expf(-fabsf(v))); }
__device__ __forceinline__ float logistic_exact(float v) {
  const float e = expf(-fabsf(v));
  return (v >= 0.0f ? 1.0f : e) / (1.0f + e);
}

// per-channel constants of a row
struct GatedRow {
  float rate;    // c softplus(lam)
  float root;    // sqrt(2 rate)
  float cr, ci;  // -log2(e) times the biases
  bool slow;     // some gate may take rate r past the series of the decay: CARE
};

constexpr float kSeriesEnd = 0.25f;

template <typename Args>
__device__ __forceinline__ GatedRow gated_row(const Args& p, int d) {
  GatedRow w;
  w.rate = p.c * softplus_exact(p.lam[d * p.lam_s]);
  w.root = sqrtf(2.0f * w.rate);
  w.cr = p.rb ? -kLog2e * p.rb[d * p.rb_s] : 0.0f;
  w.ci = p.ib ? -kLog2e * p.ib[d * p.ib_s] : 0.0f;
  w.slow = !(w.rate < kSeriesEnd);
  return w;
}

// sigmoid(v) = 1 / p, p = 1 + 2^(-log2(e) v).
//
// The usual path (CARE = false) takes one reciprocal root for all gates of a step,
//   u = 1 / (sqrt(pr) pi pz),  sqrt(r) = u pi pz,  sqrt(r) i = u pz,  1 / pz = (u pi)(pr sqrt(r)),
// and none for sqrt(1 - a^2): with y = rate r, below y = 1/4,
//   sqrt(1 - exp(-2y)) = sqrt(2 rate) sqrt(r) P(y),   P(y) = sqrt((1 - exp(-2y)) / (2y)),
// a polynomial (its reciprocal R is another).  3 SFU results a step, 4 with z; a reciprocal each and two
// roots would be 5 and 7, which is more than the I/O lets the SFU have (2.7 steps a cycle and SM of 10 bytes).
// The polynomials are near-minimax fits on [0, 1/4], relative errors below 2^-27.
//
// `most` collects pr pi^2 pz^2, which has to stay below 2^125 for this; where it does not, or is a NaN, the
// window is computed once more with CARE: a reciprocal for each gate, so every gate falls to the smallest
// normal number before it is zero, and a NaN stays with its own gate.  Rows whose rate reaches 1/4 take
// CARE at once.
constexpr float kGateMost = 4.2535296e37f;  // 2^125

__device__ __forceinline__ f2_t ex2_2(f2_t v) {
  float a, b;
  f2split(v, a, b);
  return f2(ex2f(a), ex2f(b));
}
__device__ __forceinline__ f2_t rcp_2(f2_t v) {
  float a, b;
  f2split(v, a, b);
  return f2(rcpf(a), rcpf(b));
}
__device__ __forceinline__ f2_t rsqrt_2(f2_t v) {
  float a, b;
  f2split(v, a, b);
  return f2(rsqrt_approx(a), rsqrt_approx(b));
}
__device__ __forceinline__ f2_t one_plus(f2_t v) { return add2(v, f2s(1.0f)); }
__device__ __forceinline__ void note_most(float& most, f2_t v) {
  float a, b;
  f2split(v, a, b);
  most = max_nan(most, max_nan(a, b));
}

// CARE: a sigmoid and its complement, which is 1 long before e / (1 + e) overflows
__device__ __forceinline__ void sigmoid_both(f2_t v, f2_t& s, f2_t& c) {
  const f2_t e = ex2_2(v);
  s = rcp_2(one_plus(e));
  const f2_t q = mul2(e, s);
  c = f2(f2lo(e) < 1.0e18f ? f2lo(q) : 1.0f, f2hi(e) < 1.0e18f ? f2hi(q) : 1.0f);
}

// 1 - exp(-y), y < 1/4.  With a = 1 minus it, a is rounded once: a relative error e of a slow decay compounds
// over its memory to e / y, and the SFU exponential's 2^-22 would be felt.
__device__ __forceinline__ f2_t decay_loss(f2_t y) {
  f2_t q = fma2(y, f2s(0.00753015606f), f2s(-0.0415001251f));
  q = fma2(y, q, f2s(0.166652888f));
  q = fma2(y, q, f2s(-0.499999642f));
  q = fma2(y, q, f2s(1.0f));
  return mul2(y, q);
}
__device__ __forceinline__ f2_t root_series(f2_t y) {  // P
  f2_t q = fma2(y, f2s(0.0123667913f), f2s(-0.0622208975f));
  q = fma2(y, q, f2s(0.208310276f));
  q = fma2(y, q, f2s(-0.499999404f));
  return fma2(y, q, f2s(1.0f));
}
__device__ __forceinline__ f2_t root_inverse(f2_t y) {  // R
  f2_t q = fma2(y, f2s(-0.000555377337f), f2s(-0.0210434105f));
  q = fma2(y, q, f2s(0.041683875f));
  q = fma2(y, q, f2s(0.499999553f));
  return fma2(y, q, f2s(1.0f));
}

// CARE: a, sqrt(1 - a^2) and y / sqrt(1 - a^2) for any y.  Above 1/4, 1 - a >= 0.22 and the SFU exponential
// serves.  1 - a^2 = (1 - a)(1 + a) is scaled by 2^40 (v: 2^20) so that the smallest normal number, added
// for a finite root of 0, changes no normal 1 - a^2.
constexpr float kVScale = 1048576.0f;  // 2^20

__device__ __forceinline__ void decay_care(f2_t y, f2_t& a, f2_t& beta, f2_t& y_beta) {
  float y0, y1, m0, m1;
  f2split(y, y0, y1);
  f2split(decay_loss(y), m0, m1);
  const float e0 = ex2f(-kLog2e * y0), e1 = ex2f(-kLog2e * y1);
  const f2_t m = f2(y0 < kSeriesEnd ? m0 : 1.0f - e0, y1 < kSeriesEnd ? m1 : 1.0f - e1);
  a = f2(y0 < kSeriesEnd ? 1.0f - m0 : e0, y1 < kSeriesEnd ? 1.0f - m1 : e1);
  const f2_t v = mul2(m, fma2(a, f2s(kVScale), f2s(kVScale)));
  const f2_t q = rsqrt_2(fma2(v, f2s(kVScale), f2s(1.17549435e-38f)));
  beta = mul2(v, q);
  y_beta = mul2(mul2(y, f2s(kVScale)), q);
}

// A window's a, driven terms b = sqrt(1 - a^2) i x and, with Z, silu(z) (in zz).  Returns `most`.
template <bool Z, bool CARE, int E>
__device__ __forceinline__ float steps(const f2_t (&x)[E / 2], const f2_t (&rr)[E / 2], const f2_t (&ii)[E / 2],
                                       f2_t (&zz)[E / 2], const GatedRow& w, float (&av)[E], float (&bv)[E]) {
  float most = 0.0f;
#pragma unroll
  for (int k = 0; k < E / 2; ++k) {
    const f2_t pr = one_plus(ex2_2(fma2(rr[k], f2s(-kLog2e), f2s(w.cr))));
    const f2_t pi = one_plus(ex2_2(fma2(ii[k], f2s(-kLog2e), f2s(w.ci))));
    const f2_t pz = Z ? one_plus(ex2_2(mul2(zz[k], f2s(-kLog2e)))) : 0;
    f2_t a, b;
    if constexpr (CARE) {
      f2_t beta, unused;
      decay_care(mul2(rcp_2(pr), f2s(w.rate)), a, beta, unused);
      b = mul2(mul2(beta, rcp_2(pi)), x[k]);
      if (Z) zz[k] = mul2(zz[k], rcp_2(pz));
    } else {
      const f2_t t = Z ? mul2(pi, pz) : pi;
      const f2_t all = mul2(mul2(pr, t), t);
      note_most(most, all);
      const f2_t u = rsqrt_2(all), s = mul2(u, t);
      const f2_t y = mul2(mul2(s, s), f2s(w.rate));
      a = fma2(decay_loss(y), f2s(-1.0f), f2s(1.0f));
      b = mul2(mul2(mul2(Z ? mul2(u, pz) : u, f2s(w.root)), root_series(y)), x[k]);
      if (Z) zz[k] = mul2(mul2(mul2(u, pi), mul2(pr, s)), zz[k]);
    }
    f2split(a, av[2 * k], av[2 * k + 1]);
    f2split(b, bv[2 * k], bv[2 * k + 1]);
  }
  return most;
}

// zeros the steps of a window that `valid` leaves out
template <int E>
__device__ __forceinline__ void blank(f2_t (&v)[E / 2], unsigned valid) {
#pragma unroll
  for (int k = 0; k < E / 2; ++k)
    v[k] = f2(valid >> (2 * k) & 1u ? f2lo(v[k]) : 0.0f, valid >> (2 * k + 1) & 1u ? f2hi(v[k]) : 0.0f);
}

// The same for the backward pass.  In: x, r, i, z, dout.  Out: y = rate r (x), 1 - r (r), i x rho (i),
// dout silu'(z) (z), dout silu(z) (g), sqrt(1 - a^2) i (pv), b (1 - i) (cv), a and b.  `valid`: the steps
// that count; y is 0 at the others.
template <bool Z, bool CARE, int E>
__device__ __forceinline__ float steps_grad(f2_t (&xv)[E / 2], f2_t (&rv)[E / 2], f2_t (&iv)[E / 2], f2_t (&zv)[E / 2],
                                            f2_t (&gv)[E / 2], const GatedRow& w, bool whole, unsigned valid,
                                            float (&av)[E], float (&bv)[E], f2_t (&pv)[E / 2], f2_t (&cv)[E / 2]) {
  float most = 0.0f;
#pragma unroll
  for (int k = 0; k < E / 2; ++k) {
    const f2_t ur = fma2(rv[k], f2s(-kLog2e), f2s(w.cr)), ui = fma2(iv[k], f2s(-kLog2e), f2s(w.ci));
    const f2_t uz = Z ? mul2(zv[k], f2s(-kLog2e)) : 0;
    f2_t y, ic, sz = 0, szc = 0, a;
    auto only_valid = [&] {
      if (whole) return;
      f2_t one[1] = {y};
      blank<2>(one, valid >> (2 * k));
      y = one[0];
    };
    if constexpr (CARE) {
      f2_t r, i, beta, y_beta;
      sigmoid_both(ur, r, rv[k]);
      sigmoid_both(ui, i, ic);
      if (Z) sigmoid_both(uz, sz, szc);
      y = mul2(r, f2s(w.rate));
      only_valid();
      decay_care(y, a, beta, y_beta);
      pv[k] = mul2(beta, i);
      iv[k] = mul2(mul2(i, xv[k]), mul2(a, y_beta));
    } else {
      const f2_t er = ex2_2(ur), ei = ex2_2(ui), ez = Z ? ex2_2(uz) : 0;
      const f2_t pr = one_plus(er), pi = one_plus(ei), pz = Z ? one_plus(ez) : 0;
      const f2_t t = Z ? mul2(pi, pz) : pi;
      const f2_t all = mul2(mul2(pr, t), t);
      note_most(most, all);
      const f2_t u = rsqrt_2(all), s = mul2(u, t), r = mul2(s, s), sp = mul2(pr, s);  // sp = 1 / s
      const f2_t si = Z ? mul2(u, pz) : u;                                             // sqrt(r) i
      ic = mul2(ei, mul2(si, sp));
      if (Z) {
        sz = mul2(mul2(u, pi), sp);
        szc = mul2(ez, sz);
      }
      rv[k] = mul2(er, r);
      y = mul2(r, f2s(w.rate));
      only_valid();
      a = fma2(decay_loss(y), f2s(-1.0f), f2s(1.0f));
      const f2_t g = mul2(si, f2s(w.root));
      pv[k] = mul2(g, root_series(y));
      iv[k] = mul2(mul2(mul2(g, f2s(0.5f)), xv[k]), mul2(a, root_inverse(y)));
    }
    const f2_t b = mul2(pv[k], xv[k]);
    xv[k] = y;
    cv[k] = mul2(b, ic);
    if (Z) {
      const f2_t ds = mul2(gv[k], sz);
      gv[k] = mul2(ds, zv[k]);
      zv[k] = mul2(ds, fma2(zv[k], szc, f2s(1.0f)));
    }
    f2split(a, av[2 * k], av[2 * k + 1]);
    f2split(b, bv[2 * k], bv[2 * k + 1]);
  }
  return most;
}

// ---------------------------------------------------------------- a thread's window of a row

// E consecutive elements as stored
template <typename T, int E>
struct Win {
  static constexpr int kVecs = E * int(sizeof(T)) / 16;
  uint4 v[kVecs];
};

// ... and as fp32 pairs
template <typename T, int E>
__device__ __forceinline__ void win_get(const Win<T, E>& w, f2_t (&f)[E / 2]) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int k = 0; k < Win<T, E>::kVecs; ++k) {
      f[4 * k] = f2(bf16lo(w.v[k].x), bf16hi(w.v[k].x));
      f[4 * k + 1] = f2(bf16lo(w.v[k].y), bf16hi(w.v[k].y));
      f[4 * k + 2] = f2(bf16lo(w.v[k].z), bf16hi(w.v[k].z));
      f[4 * k + 3] = f2(bf16lo(w.v[k].w), bf16hi(w.v[k].w));
    }
  } else {
#pragma unroll
    for (int k = 0; k < Win<T, E>::kVecs; ++k) {
      f[2 * k] = f2(__uint_as_float(w.v[k].x), __uint_as_float(w.v[k].y));
      f[2 * k + 1] = f2(__uint_as_float(w.v[k].z), __uint_as_float(w.v[k].w));
    }
  }
}

// Steps [t0, t0 + E) of a row of L steps.  vec: the window's address is 16-byte aligned.  Steps
// outside the row are not read and come back as zero.
template <typename T, int E>
__device__ __forceinline__ Win<T, E> win_load(const T* row, int t0, int L, bool vec) {
  Win<T, E> w;
  if (vec && t0 >= 0 && t0 + E <= L) {
    const uint4* p = reinterpret_cast<const uint4*>(row + t0);
#pragma unroll
    for (int k = 0; k < Win<T, E>::kVecs; ++k) w.v[k] = __ldg(p + k);
    return w;
  }
  uint32_t u[4 * Win<T, E>::kVecs];
#pragma unroll
  for (int k = 0; k < 4 * Win<T, E>::kVecs; ++k) u[k] = 0u;
#pragma unroll
  for (int j = 0; j < E; ++j) {
    const int t = t0 + j;
    if (t < 0 || t >= L) continue;
    if constexpr (sizeof(T) == 2) {
      u[j / 2] |= uint32_t(row[t]) << (16 * (j & 1));
    } else {
      u[j] = __float_as_uint(row[t]);
    }
  }
#pragma unroll
  for (int k = 0; k < Win<T, E>::kVecs; ++k) w.v[k] = make_uint4(u[4 * k], u[4 * k + 1], u[4 * k + 2], u[4 * k + 3]);
  return w;
}

// Stores the steps of `mask` (bit j: step t0 + j, which lies inside the row).
template <typename T, int E>
__device__ __forceinline__ void win_store(T* row, int t0, unsigned mask, bool vec, const f2_t (&f)[E / 2]) {
  if (vec && mask == (1u << E) - 1u) {
    uint4* p = reinterpret_cast<uint4*>(row + t0);
#pragma unroll
    for (int k = 0; k < Win<T, E>::kVecs; ++k) {
      if constexpr (sizeof(T) == 2) {
        p[k] = make_uint4(pack_bf16x2(f2lo(f[4 * k]), f2hi(f[4 * k])), pack_bf16x2(f2lo(f[4 * k + 1]), f2hi(f[4 * k + 1])),
                          pack_bf16x2(f2lo(f[4 * k + 2]), f2hi(f[4 * k + 2])),
                          pack_bf16x2(f2lo(f[4 * k + 3]), f2hi(f[4 * k + 3])));
      } else {
        p[k] = make_uint4(__float_as_uint(f2lo(f[2 * k])), __float_as_uint(f2hi(f[2 * k])),
                          __float_as_uint(f2lo(f[2 * k + 1])), __float_as_uint(f2hi(f[2 * k + 1])));
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < E; ++j) {
    if (!(mask >> j & 1u)) continue;
    const float v = j & 1 ? f2hi(f[j / 2]) : f2lo(f[j / 2]);
    if constexpr (sizeof(T) == 2) {
      row[t0 + j] = f_to_bf16(v);
    } else {
      row[t0 + j] = v;
    }
  }
}

template <typename T>
__device__ __forceinline__ unsigned misalign(const T* p) {
  return unsigned(reinterpret_cast<uintptr_t>(p) & 15u);
}

// ---------------------------------------------------------------- packed sequences

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
  int S, c0, cS;  // the first and last offset
  int base, v;    // the lane's offset is number base + lane

  __device__ __forceinline__ int get(int j) const { return j <= S ? __ldg(cu + j) : 0x7fffffff; }
  __device__ __forceinline__ void start(const int* offsets, int n, int lane) {
    cu = offsets;
    S = n;
    c0 = __ldg(cu);
    cS = __ldg(cu + n);
    base = 0;
    v = get(lane);
  }
  // To the warp's steps [wt, wt + n), up or down the row.  Says whether they lie inside one sequence, with no
  // first or last step.
  __device__ __forceinline__ bool enter(int wt, int n, int lane) {
    unsigned below = __ballot_sync(~0u, v < wt);
    while (below == ~0u) {
      base += 32;
      v = get(base + lane);
      below = __ballot_sync(~0u, v < wt);
    }
    while (below == 0u && base > 0) {
      base -= 32;
      v = get(base + lane);
      below = __ballot_sync(~0u, v < wt);
      if (below == ~0u) break;
    }
    const int before = base + __popc(below);
    return !__any_sync(~0u, v >= wt && v <= wt + n) && below != ~0u && before >= 1 && before <= S;
  }
  template <int E>
  __device__ __forceinline__ SeqMask masks(int wt, int t0, int L, int lane) const {
    SeqMask m{0u, 0u, 0u, 0u, 0, false};
    constexpr unsigned kAll = (1u << E) - 1u;
    const int lo = max(max(c0, 0) - t0, 0), hi = min(min(cS, L) - t0, E);
    if (hi > lo) m.valid = (kAll >> (E - hi)) & ~((1u << lo) - 1u);
    const int te = wt + 32 * E;
    m.below = base + __popc(__ballot_sync(~0u, v < wt));
    int o32 = v;
    for (int at = base;;) {
      unsigned in = __ballot_sync(~0u, o32 >= wt && o32 <= te);
      while (in) {
        const int o = __shfl_sync(~0u, o32, __ffs(in) - 1) - t0;
        in &= in - 1;
        if (o < 0) ++m.below;
        if (o >= 0 && o < E) {
          m.twice |= m.offs >> o & 1u;
          m.offs |= 1u << o;
        }
        if (o >= 1 && o <= E) m.last |= 1u << (o - 1);
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

// ---------------------------------------------------------------- composing affine maps

// (a, b) after (pa, pb): h -> a (pa h + pb) + b.  With packed sequences a negative-zero a is a reset.
template <bool VL>
__device__ __forceinline__ void compose(float& a, float& b, float pa, float pb) {
  if (VL && __float_as_int(a) == int(0x80000000u)) return;
  b = fmaf(a, pb, b);
  a = a * pa;
}

template <bool VL>
__device__ __forceinline__ float apply(float a, float b, float h) {
  if (VL && __float_as_int(a) == int(0x80000000u)) return b;
  return fmaf(a, h, b);
}

// Inclusive composition over a warp's lanes, in lane order (REV: from lane 31 down).
template <bool VL, bool REV>
__device__ __forceinline__ void warp_compose(float& a, float& b, int lane) {
#pragma unroll
  for (int k = 1; k < 32; k *= 2) {
    const float pa = REV ? __shfl_down_sync(~0u, a, k) : __shfl_up_sync(~0u, a, k);
    const float pb = REV ? __shfl_down_sync(~0u, b, k) : __shfl_up_sync(~0u, b, k);
    if (REV ? lane + k < 32 : lane >= k) compose<VL>(a, b, pa, pb);
  }
}

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// writes a pair into the same shared-memory place of another CTA of the cluster
__device__ __forceinline__ void cluster_put(float2* at, unsigned rank, float2 v) {
  unsigned a = unsigned(__cvta_generic_to_shared(at)), r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(r), "f"(v.x), "f"(v.y) : "memory");
}

__device__ __forceinline__ void cluster_put1(float* at, unsigned rank, float v) {
  unsigned a = unsigned(__cvta_generic_to_shared(at)), r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(r), "f"(v) : "memory");
}

constexpr int kMaxSplit = 8;  // CTAs of a cluster that share a row

// The maps that tiles exchange: two sets, used in turn, so one barrier per exchange is enough.
template <int W>
struct CarrySmem {
  float2 warp[2][W];
  float2 cta[2][kMaxSplit];
};

// Carries `h` across a tile of W warps (CL: of a cluster's CTAs): in, the value before the tile; out,
// after it.  a, b: the thread's map.  Returns the value before the thread's own steps.
template <bool VL, bool REV, int W, bool CL>
__device__ __forceinline__ float tile_carry(float a, float b, float& h, CarrySmem<W>& sm, int& flip, int warp, int lane,
                                            int rank, int split) {
  warp_compose<VL, REV>(a, b, lane);
  float ea = REV ? __shfl_down_sync(~0u, a, 1) : __shfl_up_sync(~0u, a, 1);
  float eb = REV ? __shfl_down_sync(~0u, b, 1) : __shfl_up_sync(~0u, b, 1);
  constexpr int edge = REV ? 0 : 31;
  if (lane == 31 - edge) ea = 1.0f, eb = 0.0f;
  if constexpr (W == 1) {
    const float ta = __shfl_sync(~0u, a, edge), tb = __shfl_sync(~0u, b, edge);
    const float mine = apply<VL>(ea, eb, h);
    h = apply<VL>(ta, tb, h);
    return mine;
  } else {
    float2* s = sm.warp[flip];
    if (lane == edge) s[warp] = make_float2(a, b);
    __syncthreads();
    float in = h;
    if constexpr (CL) {
      // the CTA's map, to every CTA of the cluster
      if (warp == 0) {
        float ta = 1.0f, tb = 0.0f;
#pragma unroll
        for (int k = 0; k < W; ++k) {
          const float2 m = s[REV ? W - 1 - k : k];
          float ca = m.x, cb = m.y;
          compose<VL>(ca, cb, ta, tb);
          ta = ca;
          tb = cb;
        }
        if (lane < split) cluster_put(&sm.cta[flip][rank], lane, make_float2(ta, tb));
      }
      cluster_barrier();
      for (int k = 0; k < split; ++k) {
        const int c = REV ? split - 1 - k : k;
        if (c == rank) in = h;
        const float2 m = sm.cta[flip][c];
        h = apply<VL>(m.x, m.y, h);
      }
    }
    float v = in;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const int w = REV ? W - 1 - k : k;
      if (w == warp) in = v;
      const float2 m = s[w];
      v = apply<VL>(m.x, m.y, v);
    }
    if constexpr (!CL) h = v;
    flip ^= 1;
    return apply<VL>(ea, eb, in);
  }
}

// ---------------------------------------------------------------- forward

// Offsets are checked once, by the first CTA; every other use is in bounds whatever they hold.
__device__ __forceinline__ void check_offsets(const int* cu, int S, int L, unsigned* err) {
  bool bad = false;
  for (int j = threadIdx.x; j <= S; j += blockDim.x) {
    const int v = cu[j];
    bad |= v < 0 || v > L || (j < S && cu[j + 1] < v);
  }
  if (bad && err) atomicOr(err, 4u);
}

template <typename T, int E, bool Z>
struct GatedIn {
  Win<T, E> x, r, i, z;
};

constexpr int gated_threads(int W) { return W == 1 ? 128 : 32 * W; }

// the steps of a plain row's window that lie inside the row
template <int E>
__device__ __forceinline__ unsigned row_mask(int t0, int L) {
  const int lo = max(-t0, 0), hi = min(L - t0, E);
  return hi > lo ? ((1u << E) - 1u) >> (E - hi) & ~((1u << lo) - 1u) : 0u;
}

// W warps of a CTA share a row, with CL the CTAs of a cluster do; with W == 1 every warp has its own.
template <typename T, int E, int W, bool Z, bool VL, bool CL>
__global__ void __launch_bounds__(gated_threads(W)) gated_scan_kernel(const GatedArgs p) {
  constexpr int kRows = W == 1 ? 4 : 1;
  __shared__ CarrySmem<W> sm;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (VL && blockIdx.x == 0) check_offsets(p.cu, p.S, p.L, p.err);
  const int split = CL ? p.split : 1, rank = CL ? int(cluster_rank()) : 0;
  const int64_t row = CL ? blockIdx.x / split : int64_t(blockIdx.x) * kRows + (W == 1 ? warp : 0);
  if (row >= int64_t(p.Bt) * p.D) return;
  const int bt = int(row / p.D), d = int(row % p.D);
  const int wr = (W == 1 ? 0 : warp) + rank * W;  // the warp's place among those of the row
  const T* x = static_cast<const T*>(p.x) + bt * p.x_sb + d * p.x_sd;
  const T* r = static_cast<const T*>(p.r) + bt * p.r_sb + d * p.r_sd;
  const T* i = static_cast<const T*>(p.i) + bt * p.i_sb + d * p.i_sd;
  const T* z = Z ? static_cast<const T*>(p.z) + bt * p.z_sb + d * p.z_sd : nullptr;
  T* out = static_cast<T*>(p.out) + bt * p.o_sb + d * p.o_sd;
  // windows start on 16-byte boundaries when every tensor's row is equally far from one
  const unsigned mis = misalign(x);
  const bool vec = misalign(r) == mis && misalign(i) == mis && misalign(out) == mis && (!Z || misalign(z) == mis);
  const int off = vec ? int(mis / sizeof(T)) : 0;
  float h = 0.0f;
  if (!VL && p.h0) h = p.h0[bt * p.h0_sb + d * p.h0_sd];
  SeqWalk walk;
  if (VL) {
    walk.start(p.cu, p.S, lane);
    if (p.last)
      for (int j = wr * 32 + lane; j < p.S; j += 32 * W * split)
        if (p.cu[j] >= p.cu[j + 1])
          p.last[j * p.ls_sb + d * p.ls_sd] = p.h0 ? p.h0[j * p.h0_sb + d * p.h0_sd] : 0.0f;
  }
  int flip = 0;
  const int tile = 32 * W * E * split;
  int wt = wr * 32 * E - off;
  GatedIn<T, E, Z> nx;
  auto fetch = [&](int t) {
    nx.x = win_load<T, E>(x, t, p.L, vec);
    nx.r = win_load<T, E>(r, t, p.L, vec);
    nx.i = win_load<T, E>(i, t, p.L, vec);
    if (Z) nx.z = win_load<T, E>(z, t, p.L, vec);
  };
  fetch(wt + lane * E);
  const GatedRow w = gated_row(p, d);
  if (CL) cluster_barrier();  // every CTA's shared memory is there
  for (int base = -off; base < p.L; base += tile, wt += tile) {
    const int t0 = wt + lane * E;
    f2_t xv[E / 2], rv[E / 2], iv[E / 2], zv[E / 2];
    SeqMask m{(1u << E) - 1u, 0u, 0u, 0u, 0, false};
    bool whole = wt >= 0 && wt + 32 * E <= p.L;
    if (VL) whole = walk.enter(wt, 32 * E, lane) && whole;
    if (!whole) {
      if (VL) m = walk.template masks<E>(wt, t0, p.L, lane);
      else m.valid = row_mask<E>(t0, p.L);
    }
    float h0_first = 0.0f;  // of the window's first sequence start, asked for early
    if (VL && m.first && p.h0) h0_first = p.h0[int64_t(walk.seq(m, t0, __ffs(m.first) - 1)) * p.h0_sb + d * p.h0_sd];
    auto unpack = [&] {
      win_get(nx.x, xv);
      win_get(nx.r, rv);
      win_get(nx.i, iv);
      if (Z) win_get(nx.z, zv);
      if (!whole) {  // steps outside count as zeros, whatever the tensors hold there
        blank<E>(xv, m.valid);
        blank<E>(rv, m.valid);
        blank<E>(iv, m.valid);
        if (Z) blank<E>(zv, m.valid);
      }
    };
    unpack();
    if (base + tile < p.L) fetch(t0 + tile);
    float av[E], bv[E];
    float A = 1.0f, B = 0.0f;
    if (w.slow) {
      steps<Z, true, E>(xv, rv, iv, zv, w, av, bv);
    } else if (!(steps<Z, false, E>(xv, rv, iv, zv, w, av, bv) < kGateMost)) {
      fetch(t0);
      unpack();
      if (base + tile < p.L) fetch(t0 + tile);
      steps<Z, true, E>(xv, rv, iv, zv, w, av, bv);
    }
    if (whole) {
#pragma unroll
      for (int k = 0; k < E; ++k) {
        B = fmaf(av[k], B, bv[k]);
        A *= av[k];
      }
    } else {
#pragma unroll
      for (int k = 0; k < E; ++k) {
        if (!(m.valid >> k & 1u)) av[k] = 1.0f, bv[k] = 0.0f;
        if (VL && (m.first >> k & 1u)) {
          if (p.h0) {
            const bool early = (m.first & ((1u << k) - 1u)) == 0u;
            bv[k] = fmaf(av[k], early ? h0_first : p.h0[int64_t(walk.seq(m, t0, k)) * p.h0_sb + d * p.h0_sd], bv[k]);
          }
          av[k] = kResetA;
        }
        float ca = av[k], cb = bv[k];
        compose<VL>(ca, cb, A, B);
        A = ca;
        B = cb;
      }
    }
    float hk = tile_carry<VL, false, W, CL>(A, B, h, sm, flip, W == 1 ? 0 : warp, lane, rank, split);
    f2_t ov[E / 2];
    if (!VL || whole) {
#pragma unroll
      for (int k = 0; k < E / 2; ++k) {
        const float h0 = fmaf(av[2 * k], hk, bv[2 * k]);
        hk = fmaf(av[2 * k + 1], h0, bv[2 * k + 1]);
        ov[k] = Z ? mul2(f2(h0, hk), zv[k]) : f2(h0, hk);
      }
    } else {
#pragma unroll
      for (int k = 0; k < E / 2; ++k) {
        float o[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int e = 2 * k + q;
          hk = apply<VL>(av[e], bv[e], hk);
          if ((m.last >> e & 1u) && p.last) p.last[int64_t(walk.seq(m, t0, e)) * p.ls_sb + d * p.ls_sd] = hk;
          o[q] = hk;
        }
        ov[k] = Z ? mul2(f2(o[0], o[1]), zv[k]) : f2(o[0], o[1]);
      }
    }
    win_store<T, E>(out, t0, m.valid, vec, ov);
  }
  if (!VL && p.last && lane == 0 && wr == 0) p.last[bt * p.ls_sb + d * p.ls_sd] = h;
}

// ---------------------------------------------------------------- backward

// dout -> gradients.  With q_t = dout_t silu(z_t), s_t = dLoss/dh_t obeys
//   s_t = q_t + c_(t+1),  c_t = a_t s_t                  (c: what flows into h_(t-1))
// and, with y = rate r = -log a, rho = a y / beta (0 where y = 0):
//   w_t = s_t a (i x rho - y h_(t-1))                    dLoss/d log(rate) of the step
//   dr_raw = (1 - r) w, dlam = sigmoid(lam) / softplus(lam) * sum_t w_t
//   di_raw = s beta x i (1 - i), dx = s beta i, dz = dout h silu'(z)
// (d beta / d y = a^2 / beta; written with y inside, nothing is singular at y = 0).
// The row is swept forward once, keeping the state before every tile, then backwards tile by tile,
// recomputing the states inside the tile: the second read finds the row in L2.  A row of one tile is
// read once.
template <typename T, int E, int W, bool Z, bool VL, bool CL>
__global__ void __launch_bounds__(gated_threads(W)) gated_bwd_kernel(const GatedArgs p) {
  constexpr int kRows = W == 1 ? 4 : 1;
  __shared__ CarrySmem<W> sm;
  __shared__ float s_red[3][W];
  __shared__ float s_sum[3][kMaxSplit];
  extern __shared__ float s_ckpt[];  // [kRows][ntiles]
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (VL && blockIdx.x == 0) check_offsets(p.cu, p.S, p.L, p.err);
  const int split = CL ? p.split : 1, rank = CL ? int(cluster_rank()) : 0;
  const int64_t row = CL ? blockIdx.x / split : int64_t(blockIdx.x) * kRows + (W == 1 ? warp : 0);
  if (row >= int64_t(p.Bt) * p.D) return;
  const int bt = int(row / p.D), d = int(row % p.D);
  const int wc = W == 1 ? 0 : warp, wr = wc + rank * W;
  float* ckpt = s_ckpt + (W == 1 ? warp * p.ntiles : 0);
  const T* x = static_cast<const T*>(p.x) + bt * p.x_sb + d * p.x_sd;
  const T* r = static_cast<const T*>(p.r) + bt * p.r_sb + d * p.r_sd;
  const T* i = static_cast<const T*>(p.i) + bt * p.i_sb + d * p.i_sd;
  const T* z = Z ? static_cast<const T*>(p.z) + bt * p.z_sb + d * p.z_sd : nullptr;
  const T* gy = static_cast<const T*>(p.dout) + bt * p.g_sb + d * p.g_sd;
  T* dx = static_cast<T*>(p.dx) + bt * p.dx_sb + d * p.dx_sd;
  T* dr = static_cast<T*>(p.dr) + bt * p.dr_sb + d * p.dr_sd;
  T* di = static_cast<T*>(p.di) + bt * p.di_sb + d * p.di_sd;
  T* dz = Z ? static_cast<T*>(p.dz) + bt * p.dz_sb + d * p.dz_sd : nullptr;
  const unsigned mis = misalign(x);
  const bool vec = misalign(r) == mis && misalign(i) == mis && misalign(gy) == mis && misalign(dx) == mis &&
                   misalign(dr) == mis && misalign(di) == mis && (!Z || (misalign(z) == mis && misalign(dz) == mis));
  const int off = vec ? int(mis / sizeof(T)) : 0;
  SeqWalk walk;
  if (VL) {
    walk.start(p.cu, p.S, lane);
    if (p.dh0)
      for (int j = wr * 32 + lane; j < p.S; j += 32 * W * split)
        if (p.cu[j] >= p.cu[j + 1])
          p.dh0[j * p.dh_sb + d * p.dh_sd] = p.dlast ? p.dlast[j * p.dl_sb + d * p.dl_sd] : 0.0f;
  }
  const int tile = 32 * W * E * split;
  const int ntiles = (p.L + off + tile - 1) / tile;
  const int lane0 = wr * 32 * E - off;  // the warp's first step in the first tile
  int flip = 0;

  GatedRow w;
  // forward sweep: the state before every tile
  float h = !VL && p.h0 ? p.h0[bt * p.h0_sb + d * p.h0_sd] : 0.0f;
  {
    GatedIn<T, E, false> nx;
    auto fetch = [&](int t) {
      nx.x = win_load<T, E>(x, t, p.L, vec);
      nx.r = win_load<T, E>(r, t, p.L, vec);
      nx.i = win_load<T, E>(i, t, p.L, vec);
    };
    if (ntiles > 1) fetch(lane0 + lane * E);
    w = gated_row(p, d);
    if (CL) cluster_barrier();  // every CTA's shared memory is there
    for (int tl = 0; tl + 1 < ntiles; ++tl) {
      if (lane == 0 && wc == 0) ckpt[tl] = h;
      const int wt = lane0 + tl * tile, t0 = wt + lane * E;
      f2_t xv[E / 2], rv[E / 2], iv[E / 2];
      SeqMask m{(1u << E) - 1u, 0u, 0u, 0u, 0, false};
      bool whole = wt >= 0;  // only the last tile reaches the row's end
      if (VL) whole = walk.enter(wt, 32 * E, lane) && whole;
      if (!whole) {
        if (VL) m = walk.template masks<E>(wt, t0, p.L, lane);
        else m.valid = row_mask<E>(t0, p.L);
      }
      float h0_first = 0.0f;
      if (VL && m.first && p.h0) h0_first = p.h0[int64_t(walk.seq(m, t0, __ffs(m.first) - 1)) * p.h0_sb + d * p.h0_sd];
      auto unpack = [&] {
        win_get(nx.x, xv);
        win_get(nx.r, rv);
        win_get(nx.i, iv);
        if (!whole) {
          blank<E>(xv, m.valid);
          blank<E>(rv, m.valid);
          blank<E>(iv, m.valid);
        }
      };
      unpack();
      if (tl + 2 < ntiles) fetch(t0 + tile);
      float av[E], bv[E];
      float A = 1.0f, B = 0.0f;
      f2_t none[E / 2];
      if (w.slow) {
        steps<false, true, E>(xv, rv, iv, none, w, av, bv);
      } else if (!(steps<false, false, E>(xv, rv, iv, none, w, av, bv) < kGateMost)) {
        fetch(t0);
        unpack();
        if (tl + 2 < ntiles) fetch(t0 + tile);
        steps<false, true, E>(xv, rv, iv, none, w, av, bv);
      }
      if (whole) {
#pragma unroll
        for (int k = 0; k < E; ++k) {
          B = fmaf(av[k], B, bv[k]);
          A *= av[k];
        }
      } else {
#pragma unroll
        for (int k = 0; k < E; ++k) {
          if (!(m.valid >> k & 1u)) av[k] = 1.0f, bv[k] = 0.0f;
          if (VL && (m.first >> k & 1u)) {
            if (p.h0) {
            const bool early = (m.first & ((1u << k) - 1u)) == 0u;
            bv[k] = fmaf(av[k], early ? h0_first : p.h0[int64_t(walk.seq(m, t0, k)) * p.h0_sb + d * p.h0_sd], bv[k]);
          }
            av[k] = kResetA;
          }
          float ca = av[k], cb = bv[k];
          compose<VL>(ca, cb, A, B);
          A = ca;
          B = cb;
        }
      }
      tile_carry<VL, false, W, CL>(A, B, h, sm, flip, wc, lane, rank, split);
    }
    if (lane == 0 && wc == 0 && ntiles > 0) ckpt[ntiles - 1] = h;
  }
  if (W == 1) __syncwarp();
  else __syncthreads();

  // backward sweep
  float sum_w = 0.0f, sum_r = 0.0f, sum_i = 0.0f;
  float c = !VL && p.dlast ? p.dlast[bt * p.dl_sb + d * p.dl_sd] : 0.0f;
  GatedIn<T, E, Z> nx;
  Win<T, E> ng;
  auto fetch = [&](int t) {
    nx.x = win_load<T, E>(x, t, p.L, vec);
    nx.r = win_load<T, E>(r, t, p.L, vec);
    nx.i = win_load<T, E>(i, t, p.L, vec);
    ng = win_load<T, E>(gy, t, p.L, vec);
    if (Z) nx.z = win_load<T, E>(z, t, p.L, vec);
  };
  if (ntiles > 0) fetch(lane0 + (ntiles - 1) * tile + lane * E);
  for (int tl = ntiles - 1; tl >= 0; --tl) {
    const int wt = lane0 + tl * tile, t0 = wt + lane * E;
    f2_t xv[E / 2], rv[E / 2], iv[E / 2], zv[E / 2], gv[E / 2];
    SeqMask m{(1u << E) - 1u, 0u, 0u, 0u, 0, false};
    bool whole = wt >= 0 && wt + 32 * E <= p.L;
    if (VL) whole = walk.enter(wt, 32 * E, lane) && whole;
    if (!whole) {
      if (VL) m = walk.template masks<E>(wt, t0, p.L, lane);
      else m.valid = row_mask<E>(t0, p.L);
    }
    float h0_first = 0.0f;  // of the window's first sequence start, asked for early
    if (VL && m.first && p.h0) h0_first = p.h0[int64_t(walk.seq(m, t0, __ffs(m.first) - 1)) * p.h0_sb + d * p.h0_sd];
    auto unpack = [&] {
      win_get(nx.x, xv);
      win_get(nx.r, rv);
      win_get(nx.i, iv);
      win_get(ng, gv);
      if (Z) win_get(nx.z, zv);
      if (!whole) {  // steps outside count as zeros, whatever the tensors hold there
        blank<E>(xv, m.valid);
        blank<E>(rv, m.valid);
        blank<E>(iv, m.valid);
        blank<E>(gv, m.valid);
        if (Z) blank<E>(zv, m.valid);
      }
    };
    float dl_last = 0.0f;  // of the window's last sequence end
    if (VL && m.last && p.dlast) dl_last = p.dlast[int64_t(walk.seq(m, t0, 31 - __clz(m.last))) * p.dl_sb + d * p.dl_sd];
    unpack();
    if (tl > 0) fetch(t0 - tile);
    float av[E], bv[E];
    f2_t pv[E / 2], cv[E / 2];
    float A = 1.0f, B = 0.0f;
    if (w.slow) {
      steps_grad<Z, true, E>(xv, rv, iv, zv, gv, w, whole, m.valid, av, bv, pv, cv);
    } else if (!(steps_grad<Z, false, E>(xv, rv, iv, zv, gv, w, whole, m.valid, av, bv, pv, cv) < kGateMost)) {
      fetch(t0);
      unpack();
      if (tl > 0) fetch(t0 - tile);
        steps_grad<Z, true, E>(xv, rv, iv, zv, gv, w, whole, m.valid, av, bv, pv, cv);
    }
    float hk;
    if (!VL || whole) {
#pragma unroll
      for (int k = 0; k < E; ++k) {
        B = fmaf(av[k], B, bv[k]);
        A *= av[k];
      }
      float hin = ckpt[tl];
      hk = tile_carry<VL, false, W, CL>(A, B, hin, sm, flip, wc, lane, rank, split);
      // w / s = a (i x rho - y h_before), the outputs' gradients, and the adjoint's map of the window
#pragma unroll
      for (int k = 0; k < E / 2; ++k) {
        const float h0 = fmaf(av[2 * k], hk, bv[2 * k]), h1 = fmaf(av[2 * k + 1], h0, bv[2 * k + 1]);
        const f2_t y = xv[k];
        xv[k] = mul2(f2(av[2 * k], av[2 * k + 1]), fma2(mul2(y, f2s(-1.0f)), f2(hk, h0), iv[k]));
        if (Z) zv[k] = mul2(zv[k], f2(h0, h1));
        hk = h1;
      }
      A = 1.0f;
      B = 0.0f;
#pragma unroll
      for (int k = E - 1; k >= 0; --k) {
        const float g = k & 1 ? f2hi(gv[k / 2]) : f2lo(gv[k / 2]);
        B = av[k] * (g + B);
        A *= av[k];
      }
    } else {
      float hb[E];
#pragma unroll
      for (int k = 0; k < E; ++k) {
        hb[k] = 0.0f;
        float ca = av[k], cb = bv[k];
        if (m.first >> k & 1u) {
          if (p.h0) {
            const bool early = (m.first & ((1u << k) - 1u)) == 0u;
            hb[k] = early ? h0_first : p.h0[int64_t(walk.seq(m, t0, k)) * p.h0_sb + d * p.h0_sd];
          }
          cb = fmaf(ca, hb[k], cb);
          ca = kResetA;
        }
        compose<VL>(ca, cb, A, B);
        A = ca;
        B = cb;
      }
      float hin = ckpt[tl];
      hk = tile_carry<VL, false, W, CL>(A, B, hin, sm, flip, wc, lane, rank, split);
#pragma unroll
      for (int k = 0; k < E; ++k) {
        if (!(m.first >> k & 1u)) hb[k] = hk;
        hk = fmaf(av[k], hb[k], bv[k]);
        if (!(m.valid >> k & 1u)) hk = hb[k] = 0.0f;  // outside every sequence
        bv[k] = hk;
      }
#pragma unroll
      for (int k = 0; k < E / 2; ++k) {
        xv[k] = mul2(f2(av[2 * k], av[2 * k + 1]), fma2(mul2(xv[k], f2s(-1.0f)), f2(hb[2 * k], hb[2 * k + 1]), iv[k]));
        if (Z) zv[k] = mul2(zv[k], f2(bv[2 * k], bv[2 * k + 1]));
      }
      A = 1.0f;
      B = 0.0f;
#pragma unroll
      for (int k = E - 1; k >= 0; --k) {
        float g = k & 1 ? f2hi(gv[k / 2]) : f2lo(gv[k / 2]);
        const bool end = m.last >> k & 1u;
        if (end && p.dlast) {
          const bool early = (m.last >> k) == 1u;
          g += early ? dl_last : p.dlast[int64_t(walk.seq(m, t0, k)) * p.dl_sb + d * p.dl_sd];
          gv[k / 2] = k & 1 ? f2(f2lo(gv[k / 2]), g) : f2(g, f2hi(gv[k / 2]));
        }
        float ca = end ? kResetA : av[k], cb = av[k] * g;
        compose<VL>(ca, cb, A, B);
        A = ca;
        B = cb;
      }
    }
    float ck = tile_carry<VL, true, W, CL>(A, B, c, sm, flip, wc, lane, rank, split);
    float sv[E];
#pragma unroll
    for (int k = E - 1; k >= 0; --k) {
      const float g = k & 1 ? f2hi(gv[k / 2]) : f2lo(gv[k / 2]);
      sv[k] = VL && (m.last >> k & 1u) ? g : g + ck;
      ck = av[k] * sv[k];
      if (VL && (m.first >> k & 1u) && p.dh0)
        p.dh0[int64_t(walk.seq(m, t0, k)) * p.dh_sb + d * p.dh_sd] = ck;
      if (VL && !whole && !(m.valid >> k & 1u)) sv[k] = 0.0f;  // what flows past the steps outside stays out of the sums
    }
    f2_t acc_w = 0, acc_r = 0, acc_i = 0;
#pragma unroll
    for (int k = 0; k < E / 2; ++k) {
      const f2_t s = f2(sv[2 * k], sv[2 * k + 1]);
      const f2_t ww = mul2(s, xv[k]);
      const f2_t gr = mul2(rv[k], ww);
      const f2_t gx = mul2(s, pv[k]);
      const f2_t gi = mul2(s, cv[k]);
      acc_w = add2(acc_w, ww);
      acc_r = add2(acc_r, gr);
      acc_i = add2(acc_i, gi);
      rv[k] = gr;
      xv[k] = gx;
      cv[k] = gi;
    }
    win_store<T, E>(dx, t0, m.valid, vec, xv);
    win_store<T, E>(dr, t0, m.valid, vec, rv);
    if (Z) win_store<T, E>(dz, t0, m.valid, vec, zv);
    win_store<T, E>(di, t0, m.valid, vec, cv);
    sum_w += f2lo(acc_w) + f2hi(acc_w);
    sum_r += f2lo(acc_r) + f2hi(acc_r);
    sum_i += f2lo(acc_i) + f2hi(acc_i);
  }
  if (!VL && p.dh0 && lane == 0 && wr == 0) p.dh0[bt * p.dh_sb + d * p.dh_sd] = c;

  // the row's sums, in a fixed order
#pragma unroll
  for (int k = 16; k > 0; k /= 2) {
    sum_w += __shfl_down_sync(~0u, sum_w, k);
    sum_r += __shfl_down_sync(~0u, sum_r, k);
    sum_i += __shfl_down_sync(~0u, sum_i, k);
  }
  if constexpr (W > 1) {
    if (lane == 0) {
      s_red[0][warp] = sum_w;
      s_red[1][warp] = sum_r;
      s_red[2][warp] = sum_i;
    }
    __syncthreads();
    if (threadIdx.x < 3) {
      float v = 0.0f;
      for (int k = 0; k < W; ++k) v += s_red[threadIdx.x][k];
      s_red[threadIdx.x][0] = v;
    }
    __syncthreads();
    sum_w = s_red[0][0];
    sum_r = s_red[1][0];
    sum_i = s_red[2][0];
    if constexpr (CL) {
      if (threadIdx.x == 0)
        for (int k = 0; k < 3; ++k)
          cluster_put1(&s_sum[k][rank], 0, s_red[k][0]);
      cluster_barrier();
      if (rank == 0 && threadIdx.x == 0) {
        sum_w = sum_r = sum_i = 0.0f;
        for (int k = 0; k < split; ++k) {
          sum_w += s_sum[0][k];
          sum_r += s_sum[1][k];
          sum_i += s_sum[2][k];
        }
      }
    }
  }
  if (lane == 0 && wr == 0) {
    if (p.part) {
      const int64_t n = int64_t(p.Bt) * p.D;
      p.part[row] = sum_w;
      p.part[n + row] = sum_r;
      p.part[2 * n + row] = sum_i;
    } else {
      const float lam = p.lam[d * p.lam_s], sp = softplus_exact(lam);
      p.dlam[d] = sum_w * (sp > 0.0f ? logistic_exact(lam) / sp : 1.0f);
      if (p.drb) p.drb[d] = sum_r;
      if (p.dib) p.dib[d] = sum_i;
    }
  }
}

// ---------------------------------------------------------------- decode step

template <typename T, bool Z>
__global__ void __launch_bounds__(256) gated_step_kernel(const GatedStepArgs p) {
  const int64_t at = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (at >= int64_t(p.Bt) * p.D) return;
  const int bt = int(at / p.D), d = int(at % p.D);
  const GatedRow w = gated_row(p, d);
  float* st = p.state + bt * p.st_sb + d * p.st_sd;
  const float xv = Elem<T>::load(static_cast<const T*>(p.x) + bt * p.x_sb + d * p.x_sd);
  const float rv = Elem<T>::load(static_cast<const T*>(p.r) + bt * p.r_sb + d * p.r_sd);
  const float iv = Elem<T>::load(static_cast<const T*>(p.i) + bt * p.i_sb + d * p.i_sd);
  const float zv = Z ? Elem<T>::load(static_cast<const T*>(p.z) + bt * p.z_sb + d * p.z_sd) : 0.0f;
  const f2_t x2[1] = {f2s(xv)}, r2[1] = {f2s(rv)}, i2[1] = {f2s(iv)};
  f2_t z2[1] = {f2s(zv)};
  float a[2], b[2];
  steps<Z, true, 2>(x2, r2, i2, z2, w, a, b);  // a gate each: the step waits for memory, not for the SFU
  const float h = fmaf(a[0], *st, b[0]);
  *st = h;
  const float y = Z ? h * f2lo(z2[0]) : h;
  T* o = static_cast<T*>(p.out) + bt * p.o_sb + d * p.o_sd;
  if constexpr (sizeof(T) == 2) *o = f_to_bf16(y);
  else *o = y;
}

// ---------------------------------------------------------------- launch

template <typename K>
cudaError_t gated_launch(K kernel, const GatedArgs& a, int warps, size_t smem, cudaStream_t s) {
  const int64_t rows = int64_t(a.Bt) * a.D;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(unsigned(warps == 1 ? (rows + 3) / 4 : rows * a.split));
  c.blockDim = dim3(unsigned(gated_threads(warps)));
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(a.split);
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = a.split > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&c, kernel, a);
}

}  // namespace mssm
