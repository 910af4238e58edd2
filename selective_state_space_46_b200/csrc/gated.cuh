// The real-gated linear recurrence: forward scan, backward scan and decode step (sm_100a).
//
//   r = sigmoid(r_raw + r_bias), i = sigmoid(i_raw + i_bias), rate = c softplus(lam)
//   a_t = exp(-rate r_t), beta_t = sqrt(1 - a_t^2), h_t = a_t h_(t-1) + beta_t i_t x_t
//   out_t = h_t silu(z_t)                                               (z optional)
//
// One state per channel, so unlike the 16-state selective scan the path is a stream: 8 bytes of
// bf16 I/O per element (10 with z) against three (four) SFU results and some 40 instructions.  A row's
// steps run along the lanes: every thread holds kGs consecutive steps (one 16-byte vector of bf16), reduces
// them to the affine map h -> A h + B, and the maps are composed by warp shuffles, across warps through
// shared memory, and from tile to tile by a carry in registers; the next tile's loads are in flight meanwhile.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "device_common.cuh"
#include "seq_walk.cuh"

namespace mssm {

constexpr int kStepThreads = 128;  // of a CTA of the decode step
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
  float rate;          // c softplus(lam)
  float cr, ci;        // -log2(e) times the biases
  bool slow;           // some gate may take y = rate r to 1/8: CARE
  // Polynomials of y on [0, 1/8] as polynomials of r, near-minimax fits with relative errors below 2^-24.9.
  // (A decay of 0.9 to 0.999 at r = 1, the usual start, has a rate of 0.001 to 0.105.)
  float a1, a2, a3, a4;  // exp(-y) = 1 + a1 r + ...: a fit of (1 - exp(-y)) / y
  float p0, p1, p2, p3;  // sqrt(2 rate) P(y), P = sqrt((1 - exp(-2y)) / (2y))
};

constexpr float kFastEnd = 0.125f;
constexpr float kSeriesEnd = 0.25f;

// A larger rate is put into the gate's exponent instead: 2^40 / (1 + e 2^40 / rate) is rate / (1 + e) to 2^-33 wherever
// that is below 128, and above, a is 0 and beta 1 in any case.  So y, y h and y / beta stay finite, for an infinite rate too.
constexpr float kMostRate = 1099511627776.0f;  // 2^40

template <typename Args>
__device__ __forceinline__ GatedRow gated_row(const Args& p, int d) {
  GatedRow w;
  float q = p.c * softplus_exact(p.lam[d * p.lam_s]);
  w.cr = p.rb ? -kLog2e * p.rb[d * p.rb_s] : 0.0f;
  if (q > kMostRate) {
    w.cr -= log2f(q * (1.0f / kMostRate));
    q = kMostRate;
  }
  const float q2 = q * q;
  w.rate = q;
  w.ci = p.ib ? -kLog2e * p.ib[d * p.ib_s] : 0.0f;
  w.slow = !(q < kFastEnd);
  w.a1 = -q;
  w.a2 = 0.499997109f * q2;
  w.a3 = -0.166526049f * q2 * q;
  w.a4 = 0.0397158563f * q2 * q2;
  const float root = sqrtf(2.0f * q);
  w.p0 = root;
  w.p1 = -0.499995232f * root * q;
  w.p2 = 0.208102137f * root * q2;
  w.p3 = -0.0592916161f * root * q2 * q;
  return w;
}

// sigmoid(v) = 1 / p, p = 1 + e, e = 2^(-log2(e) v).
//
// The usual path (CARE = false) takes one reciprocal root for all gates of a step,
//   u = 1 / (sqrt(pr) pi pz),  s = sqrt(r) = u pi pz,  sqrt(r) i = u pz,  1 / pz = (u pi)(pr s),
// and none for sqrt(1 - a^2) = sqrt(2 rate) sqrt(r) P(y), y = rate r < 1/8.  3 SFU results a step, 4 with z, and
// about 18 (25) packed instructions for two steps; what bounds the scan is the issue of instructions, so
// the polynomials take r and have the row's rate in their coefficients, and products with 1 + e are
// single fused instructions.
//
// `most` adds up pr pi^2 pz^2, which has to stay below 2^125 for this; where it does not, or is a NaN, the
// window is computed once more with CARE: a reciprocal for each gate, so every gate falls to the smallest
// normal number before it is zero, and a NaN stays with its own gate.  Rows whose rate reaches 1/8 take
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
__device__ __forceinline__ bool in_range(f2_t most) { return f2lo(most) + f2hi(most) < kGateMost; }

// CARE: a sigmoid and its complement, which is 1 long before e / (1 + e) overflows
__device__ __forceinline__ void sigmoid_both(f2_t v, f2_t& s, f2_t& c) {
  const f2_t e = ex2_2(v);
  s = rcp_2(one_plus(e));
  const f2_t q = mul2(e, s);
  c = f2(f2lo(e) < 1.0e18f ? f2lo(q) : 1.0f, f2hi(e) < 1.0e18f ? f2hi(q) : 1.0f);
}

// exp(-y) for y < 1/8 by its polynomial, rounded once: a relative error e of a slow decay compounds over its
// memory to e / y, and the SFU exponential's 2^-22 would be felt.
__device__ __forceinline__ f2_t decay(f2_t r, const GatedRow& w) {
  f2_t q = fma2(r, f2s(w.a4), f2s(w.a3));
  q = fma2(r, q, f2s(w.a2));
  q = fma2(r, q, f2s(w.a1));
  return fma2(r, q, f2s(1.0f));
}
__device__ __forceinline__ f2_t root_series(f2_t r, const GatedRow& w) {  // sqrt(2 rate) P
  f2_t q = fma2(r, f2s(w.p3), f2s(w.p2));
  q = fma2(r, q, f2s(w.p1));
  return fma2(r, q, f2s(w.p0));
}
// sqrt(rate / 2) / P(y); -y
__device__ __forceinline__ f2_t root_inverse(f2_t ny, float half_root) {
  f2_t q = fma2(ny, f2s(0.0211378392f), f2s(0.0416868366f));
  q = fma2(ny, q, f2s(-0.499999613f));
  return mul2(fma2(ny, q, f2s(1.0f)), f2s(half_root));
}
__device__ __forceinline__ f2_t decay_loss(f2_t y) {  // 1 - exp(-y), y < 1/4
  f2_t q = fma2(y, f2s(0.00753015606f), f2s(-0.0415001251f));
  q = fma2(y, q, f2s(0.166652888f));
  q = fma2(y, q, f2s(-0.499999642f));
  return mul2(y, fma2(y, q, f2s(1.0f)));
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

// CARE: two steps' a, driven terms b = sqrt(1 - a^2) i x and, with Z, silu(z), from the gates' exponents
template <bool Z>
__device__ __forceinline__ void step_care(f2_t x, f2_t ur, f2_t ui, f2_t zz, f2_t rate, f2_t& a, f2_t& b, f2_t& g) {
  f2_t beta, unused;
  decay_care(mul2(rcp_2(one_plus(ex2_2(ur))), rate), a, beta, unused);
  b = mul2(mul2(beta, rcp_2(one_plus(ex2_2(ui)))), x);
  if (Z) g = mul2(zz, rcp_2(one_plus(ex2_2(mul2(zz, f2s(-kLog2e))))));
}

// Two steps' a, driven terms b = sqrt(1 - a^2) i x and, with Z, silu(z).
template <bool Z, bool CARE>
__device__ __forceinline__ void step_pair(f2_t x, f2_t rr, f2_t ii, f2_t zz, const GatedRow& w, f2_t& a, f2_t& b, f2_t& g,
                                          f2_t& most) {
  const f2_t ur = fma2(rr, f2s(-kLog2e), f2s(w.cr)), ui = fma2(ii, f2s(-kLog2e), f2s(w.ci));
  if constexpr (CARE) {
    step_care<Z>(x, ur, ui, zz, f2s(w.rate), a, b, g);
  } else {
    const f2_t er = ex2_2(ur), ei = ex2_2(ui), ez = Z ? ex2_2(mul2(zz, f2s(-kLog2e))) : 0, pi = one_plus(ei);
    const f2_t t = Z ? fma2(pi, ez, pi) : pi, tt = mul2(t, t), all = fma2(tt, er, tt);
    most = add2(most, all);
    const f2_t u = rsqrt_2(all), s = mul2(u, t), r = mul2(s, s);
    a = decay(r, w);
    b = mul2(mul2(Z ? fma2(u, ez, u) : u, root_series(r, w)), x);
    if (Z) g = mul2(mul2(fma2(u, ei, u), fma2(er, s, s)), zz);
  }
}

// The same for the backward pass.  In: x, r, i, z, dout.  Out: -y (x), 1 - r (r), i x rho (i), dout silu'(z)
// (z), dout silu(z) (g), sqrt(1 - a^2) i (pv), b (1 - i) (cv), a and b.
template <bool Z, bool CARE>
__device__ __forceinline__ void step_pair_grad(f2_t& x, f2_t& rr, f2_t& ii, f2_t& zz, f2_t& gg, const GatedRow& w,
                                               f2_t& a, f2_t& b, f2_t& pv, f2_t& cv, f2_t& most) {
  const f2_t ur = fma2(rr, f2s(-kLog2e), f2s(w.cr)), ui = fma2(ii, f2s(-kLog2e), f2s(w.ci));
  const f2_t uz = Z ? mul2(zz, f2s(-kLog2e)) : 0;
  f2_t ic, sz = 0, szc = 0;
  if constexpr (CARE) {
    f2_t r, i, beta, y_beta;
    sigmoid_both(ur, r, rr);
    sigmoid_both(ui, i, ic);
    if (Z) sigmoid_both(uz, sz, szc);
    const f2_t y = mul2(r, f2s(w.rate));
    decay_care(y, a, beta, y_beta);
    pv = mul2(beta, i);
    ii = mul2(mul2(i, x), mul2(a, y_beta));
    b = mul2(pv, x);
    x = mul2(y, f2s(-1.0f));
  } else {
    const f2_t er = ex2_2(ur), ei = ex2_2(ui), ez = Z ? ex2_2(uz) : 0, pi = one_plus(ei);
    const f2_t t = Z ? fma2(pi, ez, pi) : pi, tt = mul2(t, t), all = fma2(tt, er, tt);
    most = add2(most, all);
    const f2_t u = rsqrt_2(all), s = mul2(u, t), sp = fma2(er, s, s);  // sp = 1 / s
    const f2_t si = Z ? fma2(u, ez, u) : u;                            // sqrt(r) i
    const f2_t r = mul2(s, s);
    ic = mul2(ei, mul2(si, sp));
    if (Z) {
      sz = mul2(fma2(u, ei, u), sp);
      szc = mul2(ez, sz);
    }
    rr = mul2(er, r);
    const f2_t ny = mul2(r, f2s(w.a1));
    a = decay(r, w);
    pv = mul2(si, root_series(r, w));
    ii = mul2(mul2(si, x), mul2(a, root_inverse(ny, 0.5f * w.p0)));
    b = mul2(pv, x);
    x = ny;
  }
  cv = mul2(b, ic);
  if (Z) {
    const f2_t ds = mul2(gg, sz);
    gg = mul2(ds, zz);
    zz = mul2(ds, fma2(zz, szc, f2s(1.0f)));
  }
}

// ---------------------------------------------------------------- a thread's window of a row

// A thread's kGs = 8 consecutive steps are 4 pairs of steps k and k + 4: two chains of 4 that the recurrence runs
// through together and joins once.
constexpr int kH = kGs / 2;

__device__ __forceinline__ float of(const f2_t (&f)[kH], int e) { return e < kH ? f2lo(f[e]) : f2hi(f[e - kH]); }
// 1 for the steps of `mask` and 0 for the others
__device__ __forceinline__ f2_t ones(unsigned mask, int k) {
  return f2(mask >> k & 1u ? 1.0f : 0.0f, mask >> (k + kH) & 1u ? 1.0f : 0.0f);
}
// zeros the steps of a window that `valid` leaves out
__device__ __forceinline__ void blank(f2_t (&v)[kH], unsigned valid) {
#pragma unroll
  for (int k = 0; k < kH; ++k)
    v[k] = f2(valid >> k & 1u ? f2lo(v[k]) : 0.0f, valid >> (k + kH) & 1u ? f2hi(v[k]) : 0.0f);
}

// the steps as stored
template <typename T>
struct Win {
  static constexpr int kVecs = kGs * int(sizeof(T)) / 16;
  uint4 v[kVecs];
};

template <typename T>
__device__ __forceinline__ void win_get(const Win<T>& w, f2_t (&f)[kH]) {
  if constexpr (sizeof(T) == 2) {
    f[0] = f2(bf16lo(w.v[0].x), bf16lo(w.v[0].z));
    f[1] = f2(bf16hi(w.v[0].x), bf16hi(w.v[0].z));
    f[2] = f2(bf16lo(w.v[0].y), bf16lo(w.v[0].w));
    f[3] = f2(bf16hi(w.v[0].y), bf16hi(w.v[0].w));
  } else {
    f[0] = f2(__uint_as_float(w.v[0].x), __uint_as_float(w.v[1].x));
    f[1] = f2(__uint_as_float(w.v[0].y), __uint_as_float(w.v[1].y));
    f[2] = f2(__uint_as_float(w.v[0].z), __uint_as_float(w.v[1].z));
    f[3] = f2(__uint_as_float(w.v[0].w), __uint_as_float(w.v[1].w));
  }
}

// The thread's steps of the warp's window [wt, wt + 32 kGs) of a row of L steps.  inner: the window lies inside the
// row and on a 16-byte boundary.  Steps outside the row are not read and come back as zero.
template <typename T>
__device__ __forceinline__ Win<T> win_load(const T* row, int wt, int lane, int L, bool inner) {
  Win<T> w;
  if (inner) {
    const uint4* p = reinterpret_cast<const uint4*>(row + wt) + lane * Win<T>::kVecs;
#pragma unroll
    for (int k = 0; k < Win<T>::kVecs; ++k) w.v[k] = __ldg(p + k);
    return w;
  }
  uint32_t u[4 * Win<T>::kVecs];
#pragma unroll
  for (int k = 0; k < 4 * Win<T>::kVecs; ++k) u[k] = 0u;
#pragma unroll
  for (int j = 0; j < kGs; ++j) {
    const int t = wt + lane * kGs + j;
    if (t < 0 || t >= L) continue;
    if constexpr (sizeof(T) == 2) {
      u[j / 2] |= uint32_t(row[t]) << (16 * (j & 1));
    } else {
      u[j] = __float_as_uint(row[t]);
    }
  }
#pragma unroll
  for (int k = 0; k < Win<T>::kVecs; ++k) w.v[k] = make_uint4(u[4 * k], u[4 * k + 1], u[4 * k + 2], u[4 * k + 3]);
  return w;
}

// Stores the steps of `mask` (bit j: the thread's step j, which lies inside the row).
template <typename T>
__device__ __forceinline__ void win_store(T* row, int wt, int lane, unsigned mask, bool inner, const f2_t (&f)[kH]) {
  if (inner && mask == (1u << kGs) - 1u) {
    uint4* p = reinterpret_cast<uint4*>(row + wt) + lane * Win<T>::kVecs;
    if constexpr (sizeof(T) == 2) {
      *p = make_uint4(pack_bf16x2(f2lo(f[0]), f2lo(f[1])), pack_bf16x2(f2lo(f[2]), f2lo(f[3])),
                      pack_bf16x2(f2hi(f[0]), f2hi(f[1])), pack_bf16x2(f2hi(f[2]), f2hi(f[3])));
    } else {
      p[0] = make_uint4(__float_as_uint(f2lo(f[0])), __float_as_uint(f2lo(f[1])), __float_as_uint(f2lo(f[2])),
                        __float_as_uint(f2lo(f[3])));
      p[1] = make_uint4(__float_as_uint(f2hi(f[0])), __float_as_uint(f2hi(f[1])), __float_as_uint(f2hi(f[2])),
                        __float_as_uint(f2hi(f[3])));
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < kGs; ++j) {
    if (!(mask >> j & 1u)) continue;
    const float v = of(f, j);
    T* to = row + wt + lane * kGs + j;
    if constexpr (sizeof(T) == 2) {
      *to = f_to_bf16(v);
    } else {
      *to = v;
    }
  }
}

template <typename T>
__device__ __forceinline__ unsigned misalign(const T* p) {
  return unsigned(reinterpret_cast<uintptr_t>(p) & 15u);
}

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
// after it.  a, b: the thread's map; whole: the warp's maps hold no reset.  Returns the value before the thread's own
// steps.
template <bool VL, bool REV, int W, bool CL>
__device__ __forceinline__ float tile_carry(float a, float b, float& h, CarrySmem<W>& sm, int& flip, int warp, int lane,
                                            int rank, int split, bool whole) {
  if (!VL || whole) warp_compose<false, REV>(a, b, lane);
  else warp_compose<true, REV>(a, b, lane);
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

// Warps of an SM for which registers are set aside: 80 registers a thread forward, 128 backward.  Measured
// for 20 / 24 / 28 / 32 warps forward, 1x2048x131072 bf16: 535 / 522 / 563 / 557 us; for 12 / 16 / 20 backward,
// 8x5120x4096 bf16: 901 / 819 / 901 us (fewer registers spill, fewer warps leave the issue slots idle).
constexpr int kScanWarps = 24, kBwdWarps = 16;
constexpr int gated_threads(int W) { return W == 1 ? 128 : 32 * W; }

// Where a CTA's warp works: W warps of a CTA share a row, with CL the CTAs of a cluster do; with W == 1 every
// warp has its own.
template <int W, bool CL>
struct GatedPlace {
  int warp, lane, split, rank;
  int wc, wr;      // the warp's place among those of the row in the CTA, and among all
  int64_t row;
  __device__ __forceinline__ GatedPlace(const GatedArgs& p) {
    warp = __shfl_sync(~0u, int(threadIdx.x) / 32, 0);
    lane = threadIdx.x % 32;
    split = CL ? p.split : 1;
    rank = CL ? int(cluster_rank()) : 0;
    wc = W == 1 ? 0 : warp;
    wr = wc + rank * W;
    row = CL ? blockIdx.x / split : W == 1 ? int64_t(blockIdx.x) * 4 + warp : int64_t(blockIdx.x);
  }
};

// A window in which no thread has more than one first and one last step: selected step by step, without a branch.
// The warp at a boundary holds up the other warps of its row, so what counts here is the way through.
__device__ __forceinline__ bool on_bit(unsigned mask, int e) { return mask >> e & 1u; }

// The map (A, B); the steps outside the sequences become the identity, and the first step's b takes h0.
__device__ __forceinline__ float2 edge_map(f2_t (&a)[kH], f2_t (&b)[kH], const SeqMask& m, float h0) {
  float av[kGs], bv[kGs], A = 1.0f, B = 0.0f;
#pragma unroll
  for (int k = 0; k < kH; ++k) {
    f2split(a[k], av[k], av[k + kH]);
    f2split(b[k], bv[k], bv[k + kH]);
  }
#pragma unroll
  for (int e = 0; e < kGs; ++e) {
    if (!on_bit(m.valid, e)) av[e] = 1.0f, bv[e] = 0.0f;
    if (on_bit(m.first, e)) bv[e] = fmaf(av[e], h0, bv[e]);
    const float through = fmaf(av[e], B, bv[e]);
    B = on_bit(m.first, e) ? bv[e] : through;
    A *= av[e];
  }
#pragma unroll
  for (int k = 0; k < kH; ++k) {
    a[k] = f2(av[k], av[k + kH]);
    b[k] = f2(bv[k], bv[k + kH]);
  }
  return make_float2(m.first ? kResetA : A, B);
}
// The states after every step (in b) and, with BEFORE, before it; returns that of the last step.
template <bool BEFORE>
__device__ __forceinline__ float edge_states(const f2_t (&a)[kH], f2_t (&b)[kH], const SeqMask& m, float h, float h0,
                                             f2_t (&before)[kH]) {
  float out[kGs], pre[kGs], last = 0.0f;
#pragma unroll
  for (int e = 0; e < kGs; ++e) {
    if (BEFORE) pre[e] = !on_bit(m.valid, e) ? 0.0f : on_bit(m.first, e) ? h0 : h;
    const float through = fmaf(of(a, e), h, of(b, e));
    h = on_bit(m.first, e) ? of(b, e) : through;
    if (on_bit(m.last, e)) last = h;
    out[e] = BEFORE && !on_bit(m.valid, e) ? 0.0f : h;
  }
#pragma unroll
  for (int k = 0; k < kH; ++k) {
    b[k] = f2(out[k], out[k + kH]);
    if (BEFORE) before[k] = f2(pre[k], pre[k + kH]);
  }
  return last;
}
// The adjoint's map; the last step's g takes dlast.
__device__ __forceinline__ float2 edge_adjoint_map(const f2_t (&a)[kH], f2_t (&g)[kH], const SeqMask& m, float dlast) {
  float gv[kGs], A = 1.0f, B = 0.0f;
#pragma unroll
  for (int e = kGs - 1; e >= 0; --e) {
    gv[e] = of(g, e);
    if (on_bit(m.last, e)) gv[e] += dlast;
    B = of(a, e) * (on_bit(m.last, e) ? gv[e] : gv[e] + B);
    A *= of(a, e);
  }
#pragma unroll
  for (int k = 0; k < kH; ++k) g[k] = f2(gv[k], gv[k + kH]);
  return make_float2(m.last ? kResetA : A, B);
}
// The adjoint at every step; returns what flows into the state before the first step.
__device__ __forceinline__ float edge_adjoint(const f2_t (&a)[kH], const f2_t (&g)[kH], const SeqMask& m, float c, f2_t (&s)[kH]) {
  float sv[kGs], first = 0.0f;
#pragma unroll
  for (int e = kGs - 1; e >= 0; --e) {
    const float se = on_bit(m.last, e) ? of(g, e) : of(g, e) + c;
    c = of(a, e) * se;
    if (on_bit(m.first, e)) first = c;
    sv[e] = on_bit(m.valid, e) ? se : 0.0f;  // what flows past the steps outside stays out of the sums
  }
#pragma unroll
  for (int k = 0; k < kH; ++k) s[k] = f2(sv[k], sv[k + kH]);
  return first;
}

__device__ __forceinline__ bool several(const SeqMask& m) {
  return (m.first & (m.first - 1u)) != 0u || (m.last & (m.last - 1u)) != 0u;
}

// A window with more boundaries than that, a thread's steps in local memory: sequences of a few steps.
struct BoundWin {
  float a[kGs], b[kGs];         // the steps' maps; b becomes the states
  float before[kGs], g[kGs];    // backward: the state before each step; dout silu(z), which becomes the adjoint
  SeqMask m;
  SeqWalk walk;
  int t0;
  // a state per sequence, at step e, where the one at `early` is known
  __device__ float state(const float* p, int64_t sb, int e, int early, float known) const {
    return !p ? 0.0f : e == early ? known : p[int64_t(walk.seq(m, t0, e)) * sb];
  }
  __device__ __forceinline__ void take(const f2_t (&av)[kH], const f2_t (&bv)[kH], const SeqMask& m_, const SeqWalk& walk_, int t) {
    m = m_;
    walk = walk_;
    t0 = t;
#pragma unroll
    for (int k = 0; k < kH; ++k) {
      f2split(av[k], a[k], a[k + kH]);
      f2split(bv[k], b[k], b[k + kH]);
    }
  }
};

// Forward: the window's map.  h0: of this channel.
static __device__ __noinline__ float2 bound_map(BoundWin& w, const float* h0, int64_t sb, float h0_first) {
  float A = 1.0f, B = 0.0f;
  const int early = __ffs(w.m.first) - 1;
#pragma unroll 1
  for (int e = 0; e < kGs; ++e) {
    float a = w.a[e], b = w.b[e];
    w.before[e] = 0.0f;
    if (!(w.m.valid >> e & 1u)) a = 1.0f, b = 0.0f;
    if (w.m.first >> e & 1u) {
      w.before[e] = w.state(h0, sb, e, early, h0_first);
      b = fmaf(a, w.before[e], b);
      a = kResetA;
    }
    compose<true>(a, b, A, B);
    A = a;
    B = b;
  }
  return make_float2(A, B);
}

// The states from the one before the window; `last`: of this channel, written at the sequences' ends.
static __device__ __noinline__ void bound_states(BoundWin& w, float h, float* last, int64_t sb) {
#pragma unroll 1
  for (int e = 0; e < kGs; ++e) {
    const bool valid = w.m.valid >> e & 1u;
    if (!(w.m.first >> e & 1u)) w.before[e] = h;
    if (valid) h = fmaf(w.a[e], w.before[e], w.b[e]);
    if (!valid) w.before[e] = 0.0f;  // outside every sequence
    w.b[e] = valid ? h : 0.0f;
    if ((w.m.last >> e & 1u) && last) last[int64_t(w.walk.seq(w.m, w.t0, e)) * sb] = h;
  }
}

// Backward: the adjoint's map, dlast added to g at the sequences' ends.
static __device__ __noinline__ float2 bound_adjoint_map(BoundWin& w, const float* dlast, int64_t sb, float dl_last) {
  float A = 1.0f, B = 0.0f;
  const int early = 31 - __clz(w.m.last);
#pragma unroll 1
  for (int e = kGs - 1; e >= 0; --e) {
    const bool end = w.m.last >> e & 1u;
    if (end) w.g[e] += w.state(dlast, sb, e, early, dl_last);
    float a = end ? kResetA : w.a[e], b = w.a[e] * w.g[e];
    compose<true>(a, b, A, B);
    A = a;
    B = b;
  }
  return make_float2(A, B);
}

// The adjoint from what flows into the window's end.
static __device__ __noinline__ void bound_adjoint(BoundWin& w, float c, float* dh0, int64_t sb) {
#pragma unroll 1
  for (int e = kGs - 1; e >= 0; --e) {
    const float s = w.m.last >> e & 1u ? w.g[e] : w.g[e] + c;
    c = w.a[e] * s;
    if ((w.m.first >> e & 1u) && dh0) dh0[int64_t(w.walk.seq(w.m, w.t0, e)) * sb] = c;
    w.g[e] = w.m.valid >> e & 1u ? s : 0.0f;  // what flows past the steps outside stays out of the sums
  }
}

// The map of a window whose steps all count: of its halves, and of all (A, B).
struct WinMap {
  float a_lo, b_lo, a_hi, b_hi;
  float A, B;
};
__device__ __forceinline__ WinMap win_map(const f2_t (&a)[kH], const f2_t (&b)[kH]) {
  f2_t aa = a[0], bb = b[0];
#pragma unroll
  for (int k = 1; k < kH; ++k) {
    bb = fma2(a[k], bb, b[k]);
    aa = mul2(aa, a[k]);
  }
  WinMap m;
  f2split(aa, m.a_lo, m.a_hi);
  f2split(bb, m.b_lo, m.b_hi);
  m.A = m.a_lo * m.a_hi;
  m.B = fmaf(m.a_hi, m.b_lo, m.b_hi);
  return m;
}

// 1x2048x131072 bf16 with z: 518 us from a cold L2 (5.2 TB/s, issue 70%), 542 to 580 back to back, at the clock under
// that load; 1536x27048 packed without z: 128 us, 88 unpacked; 2x1536x2048 18.4 us a call.  Rates from 1/8 on:
// 8x2048x4096 with z 152 us, 129 below.
template <typename T, int W, bool Z, bool VL, bool CL>
__global__ void __launch_bounds__(gated_threads(W), kScanWarps * 32 / gated_threads(W)) gated_scan_kernel(const GatedArgs p) {
  __shared__ CarrySmem<W> sm;
  if (VL && blockIdx.x == 0) check_offsets(p.cu, p.S, p.L, p.err);
  const GatedPlace<W, CL> at(p);
  const int lane = at.lane;
  if (at.row >= int64_t(p.Bt) * p.D) return;
  const int bt = int(unsigned(at.row) / unsigned(p.D)), d = int(unsigned(at.row) % unsigned(p.D));  // Bt D < 2^31
  const T* x = static_cast<const T*>(p.x) + bt * p.x_sb + d * p.x_sd;
  const T* r = static_cast<const T*>(p.r) + bt * p.r_sb + d * p.r_sd;
  const T* i = static_cast<const T*>(p.i) + bt * p.i_sb + d * p.i_sd;
  const T* z = Z ? static_cast<const T*>(p.z) + bt * p.z_sb + d * p.z_sd : nullptr;
  T* out = static_cast<T*>(p.out) + bt * p.o_sb + d * p.o_sd;
  // windows start on 16-byte boundaries when every tensor's row is equally far from one
  const unsigned mis = misalign(x);
  const bool vec = misalign(r) == mis && misalign(i) == mis && misalign(out) == mis && (!Z || misalign(z) == mis);
  const int off = vec ? int(mis / sizeof(T)) : 0;
  const int tile = 32 * W * kGs * at.split;
  int wt = at.wr * 32 * kGs - off;
  struct { Win<T> x, r, i, z; } nx;
  auto fetch = [&](int t) {
    const bool inner = vec && t >= 0 && t + 32 * kGs <= p.L;
    nx.x = win_load<T>(x, t, lane, p.L, inner);
    nx.r = win_load<T>(r, t, lane, p.L, inner);
    nx.i = win_load<T>(i, t, lane, p.L, inner);
    if (Z) nx.z = win_load<T>(z, t, lane, p.L, inner);
  };
  fetch(wt);
  float h = 0.0f;
  if (!VL && p.h0) h = p.h0[bt * p.h0_sb + d * p.h0_sd];
  SeqWalk walk;
  if (VL) {
    walk.start(p.cu, p.S, p.L, lane);
    if (p.last)
      for (int j = at.wr * 32 + lane; j < p.S; j += 32 * W * at.split)
        if (p.cu[j] >= p.cu[j + 1])
          p.last[j * p.ls_sb + d * p.ls_sd] = p.h0 ? p.h0[j * p.h0_sb + d * p.h0_sd] : 0.0f;
  }
  const GatedRow w = gated_row(p, d);
  if (CL) cluster_barrier();  // every CTA's shared memory is there
  int flip = 0;
  for (int base = -off; base < p.L; base += tile, wt += tile) {
    const int t0 = wt + lane * kGs;
    const bool inner = wt >= 0 && wt + 32 * kGs <= p.L;
    SeqMask m{(1u << kGs) - 1u, 0u, 0u, 0u, 0, false};
    bool whole = inner;
    if (VL) whole = walk.enter(wt, 32 * kGs, lane) && whole;
    if (!whole) {
      if (VL) m = walk.masks(wt, t0, lane);
      else m.valid = steps_inside(t0, 0, p.L);
    }
    float h0_first = 0.0f;  // of the window's first sequence start, asked for early
    if (VL && m.first && p.h0) h0_first = p.h0[int64_t(walk.seq(m, t0, __ffs(m.first) - 1)) * p.h0_sb + d * p.h0_sd];
    f2_t xv[kH], rv[kH], iv[kH], zv[kH], a[kH], b[kH];
    auto unpack = [&] {
      win_get(nx.x, xv);
      win_get(nx.r, rv);
      win_get(nx.i, iv);
      if (Z) win_get(nx.z, zv);
      if (!whole) {  // steps outside count as zeros, whatever the tensors hold there
        blank(xv, m.valid);
        blank(rv, m.valid);
        blank(iv, m.valid);
        if (Z) blank(zv, m.valid);
      }
    };
    unpack();
    if (base + tile < p.L) fetch(wt + tile);
    f2_t most = 0;
    bool care = w.slow;
    if (!care) {
#pragma unroll
      for (int k = 0; k < kH; ++k) step_pair<Z, false>(xv[k], rv[k], iv[k], zv[k], w, a[k], b[k], zv[k], most);
      care = __any_sync(~0u, !in_range(most));
      if (care) {
        fetch(wt);
        unpack();
        if (base + tile < p.L) fetch(wt + tile);
      }
    }
    if (care) {
#pragma unroll
      for (int k = 0; k < kH; ++k) step_pair<Z, true>(xv[k], rv[k], iv[k], zv[k], w, a[k], b[k], zv[k], most);
    }
    f2_t o[kH];
    if (!VL || whole) {
      if (!VL && !whole) {
#pragma unroll
        for (int k = 0; k < kH; ++k) {  // the identity outside the row
          const f2_t on = ones(m.valid, k);
          b[k] = mul2(b[k], on);
          a[k] = fma2(a[k], on, fma2(on, f2s(-1.0f), f2s(1.0f)));
        }
      }
      const WinMap wm = win_map(a, b);
      const float in = tile_carry<VL, false, W, CL>(wm.A, wm.B, h, sm, flip, at.wc, lane, at.rank, at.split, whole);
      f2_t hh = f2(in, fmaf(wm.a_lo, in, wm.b_lo));
#pragma unroll
      for (int k = 0; k < kH; ++k) {
        hh = fma2(a[k], hh, b[k]);
        o[k] = Z ? mul2(hh, zv[k]) : hh;
      }
    } else {
      const bool few = !__any_sync(~0u, several(m));
      BoundWin bw;
      float2 map;
      if (few) {
        map = edge_map(a, b, m, h0_first);
      } else {
        bw.take(a, b, m, walk, t0);
        map = bound_map(bw, p.h0 ? p.h0 + d * p.h0_sd : nullptr, p.h0_sb, h0_first);
      }
      const float in = tile_carry<VL, false, W, CL>(map.x, map.y, h, sm, flip, at.wc, lane, at.rank, at.split, whole);
      if (few) {
        const float last = edge_states<false>(a, b, m, in, h0_first, b);
        if (m.last && p.last) p.last[int64_t(walk.seq(m, t0, 31 - __clz(m.last))) * p.ls_sb + d * p.ls_sd] = last;
      } else {
        bound_states(bw, in, p.last ? p.last + d * p.ls_sd : nullptr, p.ls_sb);
#pragma unroll
        for (int k = 0; k < kH; ++k) b[k] = f2(bw.b[k], bw.b[k + kH]);
      }
#pragma unroll
      for (int k = 0; k < kH; ++k) o[k] = Z ? mul2(b[k], zv[k]) : b[k];
    }
    win_store(out, wt, lane, m.valid, vec && inner, o);
  }
  if (!VL && p.last && lane == 0 && at.wr == 0) p.last[bt * p.ls_sb + d * p.ls_sd] = h;
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
// 8x5120x4096 bf16 with z: 774 us from a cold L2 (3.9 TB/s, issue 64%), 774 to 837 back to back (845 to 880 with rates
// from 1/8 on); 2x1536x2048 41 us a call.
template <typename T, int W, bool Z, bool VL, bool CL>
__global__ void __launch_bounds__(gated_threads(W), kBwdWarps * 32 / gated_threads(W)) gated_bwd_kernel(const GatedArgs p) {
  __shared__ CarrySmem<W> sm;
  __shared__ float s_red[3][W];
  __shared__ float s_sum[3][kMaxSplit];
  extern __shared__ float s_ckpt[];  // [rows of the CTA][ntiles]
  if (VL && blockIdx.x == 0) check_offsets(p.cu, p.S, p.L, p.err);
  const GatedPlace<W, CL> at(p);
  const int lane = at.lane, warp = at.warp, wc = at.wc, wr = at.wr, split = at.split, rank = at.rank;
  const int64_t row = at.row;
  if (row >= int64_t(p.Bt) * p.D) return;
  const int bt = int(unsigned(row) / unsigned(p.D)), d = int(unsigned(row) % unsigned(p.D));  // Bt D < 2^31
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
  const int tile = 32 * W * kGs * split;
  const int ntiles = (p.L + off + tile - 1) / tile;
  const int lane0 = wr * 32 * kGs - off;  // the warp's first step in the first tile
  struct { Win<T> x, r, i; } nx;
  Win<T> nz, ng;
  auto inner_at = [&](int t) { return t >= 0 && t + 32 * kGs <= p.L; };
  auto fetch = [&](int t) {
    const bool inner = vec && inner_at(t);
    nx.x = win_load<T>(x, t, lane, p.L, inner);
    nx.r = win_load<T>(r, t, lane, p.L, inner);
    nx.i = win_load<T>(i, t, lane, p.L, inner);
  };
  auto fetch_all = [&](int t) {
    const bool inner = vec && inner_at(t);
    fetch(t);
    ng = win_load<T>(gy, t, lane, p.L, inner);
    if (Z) nz = win_load<T>(z, t, lane, p.L, inner);
  };
  if (ntiles > 1) fetch(lane0);
  else if (ntiles > 0) fetch_all(lane0);
  SeqWalk walk;
  if (VL) {
    walk.start(p.cu, p.S, p.L, lane);
    if (p.dh0)
      for (int j = wr * 32 + lane; j < p.S; j += 32 * W * split)
        if (p.cu[j] >= p.cu[j + 1])
          p.dh0[j * p.dh_sb + d * p.dh_sd] = p.dlast ? p.dlast[j * p.dl_sb + d * p.dl_sd] : 0.0f;
  }
  const GatedRow w = gated_row(p, d);
  if (CL) cluster_barrier();  // every CTA's shared memory is there
  int flip = 0;
  SeqMask m;
  bool whole;
  float h0_first;  // of the window's first sequence start, asked for early
  auto enter = [&](int wt) {
    m = SeqMask{(1u << kGs) - 1u, 0u, 0u, 0u, 0, false};
    whole = inner_at(wt);
    if (VL) whole = walk.enter(wt, 32 * kGs, lane) && whole;
    if (!whole) {
      if (VL) m = walk.masks(wt, wt + lane * kGs, lane);
      else m.valid = steps_inside(wt + lane * kGs, 0, p.L);
    }
    h0_first = 0.0f;
    if (VL && m.first && p.h0)
      h0_first = p.h0[int64_t(walk.seq(m, wt + lane * kGs, __ffs(m.first) - 1)) * p.h0_sb + d * p.h0_sd];
  };
  f2_t xv[kH], rv[kH], iv[kH], zv[kH], gv[kH], a[kH], b[kH];
  // steps outside count as zeros, whatever the tensors hold there
  auto unpack = [&] {
    win_get(nx.x, xv);
    win_get(nx.r, rv);
    win_get(nx.i, iv);
    if (!whole) {
      blank(xv, m.valid);
      blank(rv, m.valid);
      blank(iv, m.valid);
    }
  };
  auto unpack_all = [&] {
    unpack();
    win_get(ng, gv);
    if (Z) win_get(nz, zv);
    if (!whole) {
      blank(gv, m.valid);
      if (Z) blank(zv, m.valid);
    }
  };

  // the identity outside: y = 0, a = 1 (b is 0 with x)
  auto identity_outside = [&] {
#pragma unroll
    for (int k = 0; k < kH; ++k) {
      const f2_t on = ones(m.valid, k);
      xv[k] = mul2(xv[k], on);
      a[k] = fma2(a[k], on, fma2(on, f2s(-1.0f), f2s(1.0f)));
    }
  };

  // forward sweep: the state before every tile
  float h = !VL && p.h0 ? p.h0[bt * p.h0_sb + d * p.h0_sd] : 0.0f;
  for (int tl = 0; tl + 1 < ntiles; ++tl) {
    if (lane == 0 && wc == 0) ckpt[tl] = h;
    const int wt = lane0 + tl * tile, t0 = wt + lane * kGs;
    enter(wt);
    unpack();
    if (tl + 2 < ntiles) fetch(wt + tile);
    else fetch_all(wt + tile);
    f2_t most = 0, none;
    bool care = w.slow;
    if (!care) {
#pragma unroll
      for (int k = 0; k < kH; ++k) step_pair<false, false>(xv[k], rv[k], iv[k], 0, w, a[k], b[k], none, most);
      care = __any_sync(~0u, !in_range(most));
      if (care) {
        fetch(wt);
        unpack();
        if (tl + 2 < ntiles) fetch(wt + tile);
        else fetch_all(wt + tile);
      }
    }
    if (care) {
#pragma unroll
      for (int k = 0; k < kH; ++k) step_pair<false, true>(xv[k], rv[k], iv[k], 0, w, a[k], b[k], none, most);
    }
    float A, B;
    if (!VL || whole) {
      if (!VL && !whole) identity_outside();
      const WinMap wm = win_map(a, b);
      A = wm.A;
      B = wm.B;
    } else {
      float2 map;
      if (!__any_sync(~0u, several(m))) {
        map = edge_map(a, b, m, h0_first);
      } else {
        BoundWin bw;
        bw.take(a, b, m, walk, t0);
        map = bound_map(bw, p.h0 ? p.h0 + d * p.h0_sd : nullptr, p.h0_sb, h0_first);
      }
      A = map.x;
      B = map.y;
    }
    tile_carry<VL, false, W, CL>(A, B, h, sm, flip, wc, lane, rank, split, whole);
  }
  if (lane == 0 && wc == 0 && ntiles > 0) ckpt[ntiles - 1] = h;
  if (W == 1) __syncwarp();
  else __syncthreads();

  // backward sweep
  f2_t acc_w = 0, acc_r = 0, acc_i = 0;
  float c = !VL && p.dlast ? p.dlast[bt * p.dl_sb + d * p.dl_sd] : 0.0f;
  for (int tl = ntiles - 1; tl >= 0; --tl) {
    const int wt = lane0 + tl * tile, t0 = wt + lane * kGs;
    const bool inner = vec && inner_at(wt);
    enter(wt);
    float dl_last = 0.0f;  // of the window's last sequence end
    if (VL && m.last && p.dlast) dl_last = p.dlast[int64_t(walk.seq(m, t0, 31 - __clz(m.last))) * p.dl_sb + d * p.dl_sd];
    unpack_all();
    if (tl > 0) fetch_all(wt - tile);
    f2_t pv[kH], cv[kH], most = 0;
    bool care = w.slow;
    if (!care) {
#pragma unroll
      for (int k = 0; k < kH; ++k)
        step_pair_grad<Z, false>(xv[k], rv[k], iv[k], zv[k], gv[k], w, a[k], b[k], pv[k], cv[k], most);
      care = __any_sync(~0u, !in_range(most));
      if (care) {
        fetch_all(wt);
        unpack_all();
        if (tl > 0) fetch_all(wt - tile);
      }
    }
    if (care) {
#pragma unroll
      for (int k = 0; k < kH; ++k)
        step_pair_grad<Z, true>(xv[k], rv[k], iv[k], zv[k], gv[k], w, a[k], b[k], pv[k], cv[k], most);
    }
    if (!whole) identity_outside();
    // now xv: -y, rv: 1 - r, iv: i x rho, zv: dout silu'(z), gv: dout silu(z)
    f2_t s[kH];
    float hin = ckpt[tl];
    if (!VL || whole) {
      const WinMap wm = win_map(a, b);
      const float in = tile_carry<VL, false, W, CL>(wm.A, wm.B, hin, sm, flip, wc, lane, rank, split, whole);
      // w / s = a (i x rho - y h_before), dz, and what flows back out of the halves
      f2_t hh = f2(in, fmaf(wm.a_lo, in, wm.b_lo));
#pragma unroll
      for (int k = 0; k < kH; ++k) {
        xv[k] = mul2(a[k], fma2(xv[k], hh, iv[k]));
        hh = fma2(a[k], hh, b[k]);
        if (Z) zv[k] = mul2(zv[k], hh);
      }
      f2_t back = mul2(a[kH - 1], gv[kH - 1]);
#pragma unroll
      for (int k = kH - 2; k >= 0; --k) back = mul2(a[k], add2(gv[k], back));
      float c_lo, c_hi;
      f2split(back, c_lo, c_hi);
      if (Z) win_store(dz, wt, lane, m.valid, inner, zv);
      const float cin = tile_carry<VL, true, W, CL>(wm.A, fmaf(wm.a_lo, c_hi, c_lo), c, sm, flip, wc, lane, rank, split, whole);
      f2_t cc = f2(fmaf(wm.a_hi, cin, c_hi), cin);
#pragma unroll
      for (int k = kH - 1; k >= 0; --k) {
        s[k] = add2(gv[k], cc);
        cc = mul2(a[k], s[k]);
      }
    } else {
      const bool few = !__any_sync(~0u, several(m));
      BoundWin bw;
      f2_t before[kH];
      float2 map;
      if (few) {
        map = edge_map(a, b, m, h0_first);
      } else {
        bw.take(a, b, m, walk, t0);
        map = bound_map(bw, p.h0 ? p.h0 + d * p.h0_sd : nullptr, p.h0_sb, h0_first);
      }
      const float in = tile_carry<VL, false, W, CL>(map.x, map.y, hin, sm, flip, wc, lane, rank, split, whole);
      if (few) {
        edge_states<true>(a, b, m, in, h0_first, before);
      } else {
        bound_states(bw, in, nullptr, 0);
#pragma unroll
        for (int k = 0; k < kH; ++k) {
          before[k] = f2(bw.before[k], bw.before[k + kH]);
          b[k] = f2(bw.b[k], bw.b[k + kH]);
        }
      }
#pragma unroll
      for (int k = 0; k < kH; ++k) {
        xv[k] = mul2(a[k], fma2(xv[k], before[k], iv[k]));
        if (Z) zv[k] = mul2(zv[k], b[k]);
      }
      if (Z) win_store(dz, wt, lane, m.valid, inner, zv);
      if (few) {
        map = edge_adjoint_map(a, gv, m, dl_last);
      } else {
#pragma unroll
        for (int k = 0; k < kH; ++k) f2split(gv[k], bw.g[k], bw.g[k + kH]);
        map = bound_adjoint_map(bw, p.dlast ? p.dlast + d * p.dl_sd : nullptr, p.dl_sb, dl_last);
      }
      const float cin = tile_carry<VL, true, W, CL>(map.x, map.y, c, sm, flip, wc, lane, rank, split, whole);
      if (few) {
        const float first = edge_adjoint(a, gv, m, cin, s);
        if (m.first && p.dh0) p.dh0[int64_t(walk.seq(m, t0, __ffs(m.first) - 1)) * p.dh_sb + d * p.dh_sd] = first;
      } else {
        bound_adjoint(bw, cin, p.dh0 ? p.dh0 + d * p.dh_sd : nullptr, p.dh_sb);
#pragma unroll
        for (int k = 0; k < kH; ++k) s[k] = f2(bw.g[k], bw.g[k + kH]);
      }
    }
#pragma unroll
    for (int k = 0; k < kH; ++k) {
      const f2_t ww = mul2(s[k], xv[k]);
      rv[k] = mul2(rv[k], ww);
      xv[k] = mul2(s[k], pv[k]);
      cv[k] = mul2(s[k], cv[k]);
      acc_w = add2(acc_w, ww);
      acc_r = add2(acc_r, rv[k]);
      acc_i = add2(acc_i, cv[k]);
    }
    win_store(dx, wt, lane, m.valid, inner, xv);
    win_store(dr, wt, lane, m.valid, inner, rv);
    win_store(di, wt, lane, m.valid, inner, cv);
  }
  float sum_w = f2lo(acc_w) + f2hi(acc_w), sum_r = f2lo(acc_r) + f2hi(acc_r), sum_i = f2lo(acc_i) + f2hi(acc_i);
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

// A thread takes V neighbouring channels of R batch rows: the channels' constants (a softplus each) once, then
// all R rows' loads before the first is used.  V = 4 when every row and vector starts on a boundary of 4 elements
// and channels are next to each other, V = 1 otherwise.  Two rows a thread where that
// still fills the GPU (256x4096 fp32 10.2 us with the launch, 12.3 with one and with four).
template <typename T, int V>
__device__ __forceinline__ void step_load(const T* at, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = Elem<T>::load(at);
  } else if constexpr (sizeof(T) == 2) {
    const uint2 u = *reinterpret_cast<const uint2*>(at);
    v[0] = bf16lo(u.x); v[1] = bf16hi(u.x); v[2] = bf16lo(u.y); v[3] = bf16hi(u.y);
  } else {
    const float4 u = *reinterpret_cast<const float4*>(at);
    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
  }
}
template <typename T, int V>
__device__ __forceinline__ void step_store(T* at, const float (&v)[V]) {
  if constexpr (V == 1) {
    if constexpr (sizeof(T) == 2) *at = f_to_bf16(v[0]);
    else *at = v[0];
  } else if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint2*>(at) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  } else {
    *reinterpret_cast<float4*>(at) = make_float4(v[0], v[1], v[2], v[3]);
  }
}

template <typename T, int V, int R, bool Z>
__global__ void __launch_bounds__(kStepThreads) gated_step_kernel(const GatedStepArgs p) {
  const int per = (p.D + V - 1) / V;  // threads along the channels
  const unsigned at = blockIdx.x * unsigned(kStepThreads) + threadIdx.x;
  const int d = int(at % unsigned(per)) * V, b0 = int(at / unsigned(per)) * R;
  if (b0 >= p.Bt) return;
  float st[R][V], xv[R][V], rv[R][V], iv[R][V], zv[R][V];
  const int64_t b64 = b0;
  float* state = p.state + b64 * p.st_sb + d * p.st_sd;
#pragma unroll
  for (int k = 0; k < R; ++k) {
    if (b0 + k >= p.Bt) break;
    const int64_t b = b64 + k;
    step_load<float, V>(state + k * p.st_sb, st[k]);
    step_load<T, V>(static_cast<const T*>(p.x) + b * p.x_sb + d * p.x_sd, xv[k]);
    step_load<T, V>(static_cast<const T*>(p.r) + b * p.r_sb + d * p.r_sd, rv[k]);
    step_load<T, V>(static_cast<const T*>(p.i) + b * p.i_sb + d * p.i_sd, iv[k]);
    if (Z) step_load<T, V>(static_cast<const T*>(p.z) + b * p.z_sb + d * p.z_sd, zv[k]);
  }
  float lam[V], rb[V] = {}, ib[V] = {};
  step_load<float, V>(p.lam + d * p.lam_s, lam);
  if (p.rb) step_load<float, V>(p.rb + d * p.rb_s, rb);
  if (p.ib) step_load<float, V>(p.ib + d * p.ib_s, ib);
  f2_t rate[(V + 1) / 2], cr[(V + 1) / 2], ci[(V + 1) / 2];
#pragma unroll
  for (int v = 0; v < V; v += 2) {
    constexpr int n = V > 1 ? 1 : 0;
    const float q = p.c * softplus_exact(lam[v]);
    rate[v / 2] = f2(q, V > 1 ? p.c * softplus_exact(lam[v + n]) : q);
    cr[v / 2] = mul2(f2s(-kLog2e), f2(rb[v], rb[v + n]));
    ci[v / 2] = mul2(f2s(-kLog2e), f2(ib[v], ib[v + n]));
  }
#pragma unroll
  for (int k = 0; k < R; ++k) {
    if (b0 + k >= p.Bt) break;
    const int64_t b = b64 + k;
    float h[V], y[V];
#pragma unroll
    for (int v = 0; v < V; v += 2) {
      constexpr int n = V > 1 ? 1 : 0;
      const f2_t zz = Z ? f2(zv[k][v], zv[k][v + n]) : 0;
      f2_t a, bb, g = 0;
      step_care<Z>(f2(xv[k][v], xv[k][v + n]), fma2(f2(rv[k][v], rv[k][v + n]), f2s(-kLog2e), cr[v / 2]),
                   fma2(f2(iv[k][v], iv[k][v + n]), f2s(-kLog2e), ci[v / 2]), zz, rate[v / 2], a, bb, g);
      const f2_t hh = fma2(a, f2(st[k][v], st[k][v + n]), bb), yy = Z ? mul2(hh, g) : hh;
      h[v] = f2lo(hh);
      y[v] = f2lo(yy);
      if (V > 1) h[v + n] = f2hi(hh), y[v + n] = f2hi(yy);
    }
    step_store<float, V>(state + k * p.st_sb, h);
    step_store<T, V>(static_cast<T*>(p.out) + b * p.o_sb + d * p.o_sd, y);
  }
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
