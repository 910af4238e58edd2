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

#include "device_common.cuh"

namespace mssm {

constexpr int kGs = 8;             // steps per thread
constexpr int kGatedWarps = 4;     // warps per CTA
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
  int ntiles;                      // tiles of a row (backward: checkpoints in shared memory)
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

// ---------------------------------------------------------------- scalar pieces

__device__ __forceinline__ float sqrt_approx(float x) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// softplus and the logistic function of a per-channel parameter, once per row: the accurate
// library functions (the rate's relative error multiplies every decay's logarithm).
__device__ __forceinline__ float softplus_exact(float v) { return fmaxf(v, 0.0f) + log1pf(expf(-fabsf(v))); }
__device__ __forceinline__ float logistic_exact(float v) {
  const float e = expf(-fabsf(v));
  return (v >= 0.0f ? 1.0f : e) / (1.0f + e);
}

// per-channel constants of a row
struct GatedRow {
  float rate;       // c softplus(lam)
  float rb, ib;
};

template <typename Args>
__device__ __forceinline__ GatedRow gated_row(const Args& p, int d) {
  GatedRow w;
  const float sp = softplus_exact(p.lam[d * p.lam_s]);
  w.rate = p.c * sp;
  w.rb = p.rb ? p.rb[d * p.rb_s] : 0.0f;
  w.ib = p.ib ? p.ib[d * p.ib_s] : 0.0f;
  return w;
}

// The decay a = exp(-y), y = rate r >= 0, and 1 - a^2.  Below y = 1/4, 1 - a is the Taylor series
// y (1 - y/2 + ... - y^5/720) (first omitted term y^6/5040 < 5e-8 of it), so a is rounded once: a
// relative error e of a slow decay compounds over its memory to e / y, and the SFU's 2^-22 would be
// felt.  1 - a^2 = (1 - a)(1 + a) keeps the series' relative accuracy.  Above 1/4, 1 - a >= 0.22
// and the SFU exponential serves both.
struct Decay {
  float a, v;  // v = 1 - a^2
};

__device__ __forceinline__ Decay decay(float y) {
  float q = fmaf(y, -1.0f / 720.0f, 1.0f / 120.0f);
  q = fmaf(y, q, -1.0f / 24.0f);
  q = fmaf(y, q, 1.0f / 6.0f);
  q = fmaf(y, q, -0.5f);
  q = fmaf(y, q, 1.0f);
  const float e = ex2f(-kLog2e * y);
  const bool small = y < 0.25f;
  const float m = small ? y * q : 1.0f - e;
  Decay d;
  d.a = small ? 1.0f - m : e;
  d.v = fmaf(-m, m, m + m);
  return d;
}

// The logistic function as e^-|v| / (1 + e^-|v|) or 1 / (1 + e^-|v|): every denominator lies in
// [1, 2], so several share one reciprocal of their product without overflow.
struct Gates {
  float r, i, sz;     // sz: sigmoid(z) with Z
  float r1, i1, sz1;  // their complements, without the cancellation of 1 - r
};

template <bool Z, bool COMP = false>
__device__ __forceinline__ Gates gates(float vr, float vi, float z) {
  const float er = ex2f(-kLog2e * fabsf(vr)), ei = ex2f(-kLog2e * fabsf(vi));
  const float nr = vr >= 0.0f ? 1.0f : er, ni = vi >= 0.0f ? 1.0f : ei;
  const float pr = 1.0f + er, pi = 1.0f + ei;
  Gates g;
  if constexpr (Z) {
    const float ez = ex2f(-kLog2e * fabsf(z));
    const float nz = z >= 0.0f ? 1.0f : ez, pz = 1.0f + ez;
    const float ri = pr * pi;
    const float q = rcpf(ri * pz);
    const float qz = q * pz;
    const float fr = pi * qz, fi = pr * qz, fz = ri * q;  // the reciprocals of pr, pi, pz
    g.r = nr * fr;
    g.i = ni * fi;
    g.sz = nz * fz;
    if (COMP) {
      g.r1 = (vr >= 0.0f ? er : 1.0f) * fr;
      g.i1 = (vi >= 0.0f ? ei : 1.0f) * fi;
      g.sz1 = (z >= 0.0f ? ez : 1.0f) * fz;
    }
  } else {
    const float q = rcpf(pr * pi);
    const float fr = pi * q, fi = pr * q;
    g.r = nr * fr;
    g.i = ni * fi;
    g.sz = 1.0f;
    if (COMP) {
      g.r1 = (vr >= 0.0f ? er : 1.0f) * fr;
      g.i1 = (vi >= 0.0f ? ei : 1.0f) * fi;
      g.sz1 = 0.0f;
    }
  }
  return g;
}

// ---------------------------------------------------------------- a thread's window of a row

// kGs consecutive elements as stored: 16 bytes of bf16 or 32 of fp32
template <typename T>
struct Win {
  static constexpr int kVecs = kGs * int(sizeof(T)) / 16;
  uint4 v[kVecs];
};

template <typename T>
__device__ __forceinline__ void win_get(const Win<T>& w, float (&f)[kGs]) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t u[4] = {w.v[0].x, w.v[0].y, w.v[0].z, w.v[0].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = bf16lo(u[k]);
      f[2 * k + 1] = bf16hi(u[k]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      f[4 * k] = __uint_as_float(w.v[k].x);
      f[4 * k + 1] = __uint_as_float(w.v[k].y);
      f[4 * k + 2] = __uint_as_float(w.v[k].z);
      f[4 * k + 3] = __uint_as_float(w.v[k].w);
    }
  }
}

// Steps [t0, t0 + kGs) of a row of L steps.  vec: the window's address is 16-byte aligned.  Steps
// outside the row are not read and come back as zero.
template <typename T>
__device__ __forceinline__ Win<T> win_load(const T* row, int t0, int L, bool vec) {
  Win<T> w;
  if (vec && t0 >= 0 && t0 + kGs <= L) {
    const uint4* p = reinterpret_cast<const uint4*>(row + t0);
#pragma unroll
    for (int k = 0; k < Win<T>::kVecs; ++k) w.v[k] = __ldg(p + k);
    return w;
  }
  uint32_t u[4 * Win<T>::kVecs];
#pragma unroll
  for (int k = 0; k < 4 * Win<T>::kVecs; ++k) u[k] = 0u;
#pragma unroll
  for (int j = 0; j < kGs; ++j) {
    const int t = t0 + j;
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

// Stores the steps of `mask` (bit j: step t0 + j, which lies inside the row).
template <typename T>
__device__ __forceinline__ void win_store(T* row, int t0, unsigned mask, bool vec, const float (&f)[kGs]) {
  if (vec && mask == (1u << kGs) - 1u) {
    uint4* p = reinterpret_cast<uint4*>(row + t0);
    if constexpr (sizeof(T) == 2) {
      p[0] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                        pack_bf16x2(f[6], f[7]));
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        p[k] = make_uint4(__float_as_uint(f[4 * k]), __float_as_uint(f[4 * k + 1]), __float_as_uint(f[4 * k + 2]),
                          __float_as_uint(f[4 * k + 3]));
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < kGs; ++j) {
    if (!(mask >> j & 1u)) continue;
    if constexpr (sizeof(T) == 2) {
      row[t0 + j] = f_to_bf16(f[j]);
    } else {
      row[t0 + j] = f[j];
    }
  }
}

template <typename T>
__device__ __forceinline__ unsigned misalign(const T* p) {
  return unsigned(reinterpret_cast<uintptr_t>(p) & 15u);
}

// ---------------------------------------------------------------- packed sequences

// What a window holds of the packed sequences: bit j for step t0 + j.
struct SeqMask {
  unsigned valid, first, last;  // inside a sequence; its first step; its last step
  int seq;                      // the sequence of the first valid step (or an index before it)
};

// The last offset at or before t: the largest j in [lo, S] with cu[j] <= t, lo - 1 if there is none
// at or after lo.  Whatever the offsets hold, the answer stays in [lo - 1, S].
__device__ __forceinline__ int seq_find(const int* cu, int S, int t, int lo) {
  int hi = S + 1;
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (__ldg(cu + mid) <= t) lo = mid + 1;
    else hi = mid;
  }
  return lo - 1;
}

__device__ __forceinline__ SeqMask seq_mask(const int* cu, int S, int t0, int L, int& hint) {
  SeqMask m{0u, 0u, 0u, 0};
  const int tb = t0 < 0 ? 0 : t0, te = t0 + kGs < L ? t0 + kGs : L;
  if (tb >= te) return m;
  int j = seq_find(cu, S, tb, hint);
  hint = j < 0 ? 0 : j;
  m.seq = j;
  int start = j >= 0 ? __ldg(cu + j) : -1;
  int next = j < S ? __ldg(cu + j + 1) : 0x7fffffff;
  for (int t = tb; t < te; ++t) {
    while (next <= t) {  // t enters sequence j (empty ones are passed over)
      ++j;
      start = next;
      next = j < S ? __ldg(cu + j + 1) : 0x7fffffff;
    }
    if (j < 0 || j >= S) continue;
    const unsigned bit = 1u << (t - t0);
    m.valid |= bit;
    if (t == start) m.first |= bit;
    if (t + 1 == next) m.last |= bit;
  }
  return m;
}

// The sequence of step t, searching from the window's index; an index in [0, S) whatever the
// offsets hold.
__device__ __forceinline__ int seq_of(const int* cu, int S, int t, int from) {
  const int j = seq_find(cu, S, t, from < 0 ? 0 : from);
  return j < 0 ? 0 : j < S ? j : S - 1;
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

// Carries `h` across a tile of W warps: in, the value before the tile; out, after it.  a, b: the
// thread's map.  Returns the value before the thread's own steps.  buf: 2 * W pairs of shared memory
// (two sets, used in turn, so one barrier per tile is enough).
template <bool VL, bool REV, int W>
__device__ __forceinline__ float tile_carry(float a, float b, float& h, float2* buf, int& flip, int warp, int lane) {
  warp_compose<VL, REV>(a, b, lane);
  float ea = REV ? __shfl_down_sync(~0u, a, 1) : __shfl_up_sync(~0u, a, 1);
  float eb = REV ? __shfl_down_sync(~0u, b, 1) : __shfl_up_sync(~0u, b, 1);
  if (lane == (REV ? 31 : 0)) ea = 1.0f, eb = 0.0f;
  const int edge = REV ? 0 : 31;
  if constexpr (W == 1) {
    const float ta = __shfl_sync(~0u, a, edge), tb = __shfl_sync(~0u, b, edge);
    const float mine = apply<VL>(ea, eb, h);
    h = apply<VL>(ta, tb, h);
    return mine;
  } else {
    float2* s = buf + flip * W;
    flip ^= 1;
    if (lane == edge) s[warp] = make_float2(a, b);
    __syncthreads();
    float in = h;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const int w = REV ? W - 1 - k : k;
      if (w == warp) in = h;
      const float2 m = s[w];
      h = apply<VL>(m.x, m.y, h);
    }
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

template <typename T, bool Z>
struct GatedIn {
  Win<T> x, r, i, z;
};

// W warps of a CTA share a row; with W == 1 every warp has its own.
template <typename T, int W, bool Z, bool VL>
__global__ void __launch_bounds__(32 * kGatedWarps) gated_scan_kernel(const GatedArgs p) {
  constexpr int kRows = kGatedWarps / W;
  __shared__ float2 s_buf[2 * kGatedWarps];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (VL && blockIdx.x == 0) check_offsets(p.cu, p.S, p.L, p.err);
  const int64_t row = int64_t(blockIdx.x) * kRows + (W == 1 ? warp : 0);
  if (row >= int64_t(p.Bt) * p.D) return;
  const int bt = int(row / p.D), d = int(row % p.D);
  const int wr = W == 1 ? 0 : warp;
  const T* x = static_cast<const T*>(p.x) + bt * p.x_sb + d * p.x_sd;
  const T* r = static_cast<const T*>(p.r) + bt * p.r_sb + d * p.r_sd;
  const T* i = static_cast<const T*>(p.i) + bt * p.i_sb + d * p.i_sd;
  const T* z = Z ? static_cast<const T*>(p.z) + bt * p.z_sb + d * p.z_sd : nullptr;
  T* out = static_cast<T*>(p.out) + bt * p.o_sb + d * p.o_sd;
  const GatedRow w = gated_row(p, d);
  // windows start on 16-byte boundaries when every tensor's row is equally far from one
  const unsigned mis = misalign(x);
  const bool vec = misalign(r) == mis && misalign(i) == mis && misalign(out) == mis && (!Z || misalign(z) == mis);
  const int off = vec ? int(mis / sizeof(T)) : 0;
  float h = 0.0f;
  if (!VL && p.h0) h = p.h0[bt * p.h0_sb + d * p.h0_sd];
  if (VL && p.last) {
    for (int j = wr * 32 + lane; j < p.S; j += 32 * W)
      if (p.cu[j] >= p.cu[j + 1])
        p.last[j * p.ls_sb + d * p.ls_sd] = p.h0 ? p.h0[j * p.h0_sb + d * p.h0_sd] : 0.0f;
  }
  int flip = 0, hint = 0;
  const int tile = 32 * W * kGs;
  int t0 = (wr * 32 + lane) * kGs - off;
  GatedIn<T, Z> nx;
  auto fetch = [&](int t) {
    nx.x = win_load(x, t, p.L, vec);
    nx.r = win_load(r, t, p.L, vec);
    nx.i = win_load(i, t, p.L, vec);
    if (Z) nx.z = win_load(z, t, p.L, vec);
  };
  fetch(t0);
  for (int base = -off; base < p.L; base += tile, t0 += tile) {
    float xv[kGs], rv[kGs], iv[kGs], zv[kGs], av[kGs], bv[kGs];
    win_get(nx.x, xv);
    win_get(nx.r, rv);
    win_get(nx.i, iv);
    if (Z) win_get(nx.z, zv);
    if (base + tile < p.L) fetch(t0 + tile);
    SeqMask m;
    if (VL) {
      m = seq_mask(p.cu, p.S, t0, p.L, hint);
    } else {
      const int lo = t0 < 0 ? -t0 : 0, n = p.L - t0 < kGs ? p.L - t0 : kGs;  // steps [lo, n) of the window
      m.valid = n > lo ? ((1u << n) - 1u) & ~((1u << lo) - 1u) : 0u;
    }
    float A = 1.0f, B = 0.0f;
#pragma unroll
    for (int k = 0; k < kGs; ++k) {
      const Gates g = gates<Z>(rv[k] + w.rb, iv[k] + w.ib, Z ? zv[k] : 0.0f);
      const Decay dc = decay(w.rate * g.r);
      const float a = dc.a, beta = sqrt_approx(dc.v);
      if (Z) zv[k] *= g.sz;
      const bool ok = m.valid >> k & 1u;
      av[k] = ok ? a : 1.0f;
      bv[k] = ok ? beta * (g.i * xv[k]) : 0.0f;
      if (VL && (m.first >> k & 1u)) {
        if (p.h0) bv[k] = fmaf(a, p.h0[int64_t(seq_of(p.cu, p.S, t0 + k, m.seq)) * p.h0_sb + d * p.h0_sd], bv[k]);
        av[k] = kResetA;
      }
      float ca = av[k], cb = bv[k];
      compose<VL>(ca, cb, A, B);
      A = ca;
      B = cb;
    }
    float hk = tile_carry<VL, false, W>(A, B, h, s_buf, flip, wr, lane);
    float ov[kGs];
#pragma unroll
    for (int k = 0; k < kGs; ++k) {
      hk = apply<VL>(av[k], bv[k], hk);
      if (VL && (m.last >> k & 1u) && p.last)
        p.last[int64_t(seq_of(p.cu, p.S, t0 + k, m.seq)) * p.ls_sb + d * p.ls_sd] = hk;
      ov[k] = Z ? hk * zv[k] : hk;
    }
    win_store(out, t0, m.valid, vec, ov);
  }
  if (!VL && p.last && lane == 0 && wr == 0) p.last[bt * p.ls_sb + d * p.ls_sd] = h;
}

// ---------------------------------------------------------------- backward

// dout -> gradients.  With q_t = dout_t silu(z_t), s_t = dLoss/dh_t obeys
//   s_t = q_t + c_(t+1),  c_t = a_t s_t                  (c: what flows into h_(t-1))
// and, with la = log a = -rate r, rho = -la / beta (0 where la = 0):
//   w_t = s_t (la a h_(t-1) + a^2 i x rho)               dLoss/d log(rate) of the step
//   dr_raw = (1 - r) w, dlam = sigmoid(lam) / softplus(lam) * sum_t w_t
//   di_raw = s beta x i (1 - i), dx = s beta i, dz = dout h silu'(z)
// (d beta / d la = -a^2 / beta; written with la inside, nothing is singular at la = 0).
// The row is swept forward once, keeping the state before every tile, then backwards tile by tile,
// recomputing the states inside the tile: the second read finds the row in L2.
template <typename T, int W, bool Z, bool VL>
__global__ void __launch_bounds__(32 * kGatedWarps) gated_bwd_kernel(const GatedArgs p) {
  constexpr int kRows = kGatedWarps / W;
  __shared__ float2 s_buf[2 * kGatedWarps];
  __shared__ float s_red[3 * kGatedWarps];
  extern __shared__ float s_ckpt[];  // [kRows][ntiles]
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (VL && blockIdx.x == 0) check_offsets(p.cu, p.S, p.L, p.err);
  const int64_t row = int64_t(blockIdx.x) * kRows + (W == 1 ? warp : 0);
  if (row >= int64_t(p.Bt) * p.D) return;
  const int bt = int(row / p.D), d = int(row % p.D);
  const int wr = W == 1 ? 0 : warp;
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
  const GatedRow w = gated_row(p, d);
  const unsigned mis = misalign(x);
  const bool vec = misalign(r) == mis && misalign(i) == mis && misalign(gy) == mis && misalign(dx) == mis &&
                   misalign(dr) == mis && misalign(di) == mis && (!Z || (misalign(z) == mis && misalign(dz) == mis));
  const int off = vec ? int(mis / sizeof(T)) : 0;
  if (VL && p.dh0) {
    for (int j = wr * 32 + lane; j < p.S; j += 32 * W)
      if (p.cu[j] >= p.cu[j + 1])
        p.dh0[j * p.dh_sb + d * p.dh_sd] = p.dlast ? p.dlast[j * p.dl_sb + d * p.dl_sd] : 0.0f;
  }
  const int tile = 32 * W * kGs;
  const int ntiles = (p.L + off + tile - 1) / tile;
  int flip = 0;
  float av[kGs], bv[kGs], hp[kGs];

  // a, the driven term and the masks of the window at t0
  auto masks = [&](int t0, int& hint) {
    SeqMask m{0u, 0u, 0u, 0};
    if (VL) {
      m = seq_mask(p.cu, p.S, t0, p.L, hint);
    } else {
      const int lo = t0 < 0 ? -t0 : 0, n = p.L - t0 < kGs ? p.L - t0 : kGs;
      m.valid = n > lo ? ((1u << n) - 1u) & ~((1u << lo) - 1u) : 0u;
      if (p.L - 1 >= t0 && p.L - 1 < t0 + kGs) m.last = 1u << (p.L - 1 - t0);
    }
    return m;
  };

  // forward sweep: the state before every tile
  {
    float h = !VL && p.h0 ? p.h0[bt * p.h0_sb + d * p.h0_sd] : 0.0f;
    int hint = 0;
    for (int tl = 0; tl < ntiles; ++tl) {
      if (lane == 0 && wr == 0) ckpt[tl] = h;
      if (tl + 1 == ntiles) break;
      const int t0 = tl * tile + (wr * 32 + lane) * kGs - off;
      float xv[kGs], rv[kGs], iv[kGs];
      win_get(win_load(x, t0, p.L, vec), xv);
      win_get(win_load(r, t0, p.L, vec), rv);
      win_get(win_load(i, t0, p.L, vec), iv);
      const SeqMask m = masks(t0, hint);
      float A = 1.0f, B = 0.0f;
#pragma unroll
      for (int k = 0; k < kGs; ++k) {
        const Gates g = gates<false>(rv[k] + w.rb, iv[k] + w.ib, 0.0f);
        const Decay dc = decay(w.rate * g.r);
        const float a = dc.a, beta = sqrt_approx(dc.v);
        const bool ok = m.valid >> k & 1u;
        float ca = ok ? a : 1.0f, cb = ok ? beta * (g.i * xv[k]) : 0.0f;
        if (VL && (m.first >> k & 1u)) {
          if (p.h0) cb = fmaf(a, p.h0[int64_t(seq_of(p.cu, p.S, t0 + k, m.seq)) * p.h0_sb + d * p.h0_sd], cb);
          ca = kResetA;
        }
        compose<VL>(ca, cb, A, B);
        A = ca;
        B = cb;
      }
      tile_carry<VL, false, W>(A, B, h, s_buf, flip, wr, lane);
    }
  }
  if (W == 1) __syncwarp();
  else __syncthreads();

  // backward sweep
  float sum_w = 0.0f, sum_r = 0.0f, sum_i = 0.0f;
  float c = 0.0f;
  for (int tl = ntiles - 1; tl >= 0; --tl) {
    const int t0 = tl * tile + (wr * 32 + lane) * kGs - off;
    float xv[kGs], rv[kGs], iv[kGs], zv[kGs], gv[kGs], bet[kGs], rho[kGs], yv[kGs], i1[kGs];
    win_get(win_load(x, t0, p.L, vec), xv);
    win_get(win_load(r, t0, p.L, vec), rv);
    win_get(win_load(i, t0, p.L, vec), iv);
    win_get(win_load(gy, t0, p.L, vec), gv);
    if (Z) win_get(win_load(z, t0, p.L, vec), zv);
    int hint = 0;
    const SeqMask m = masks(t0, hint);
    float A = 1.0f, B = 0.0f;
#pragma unroll
    for (int k = 0; k < kGs; ++k) {
      const Gates g = gates<Z, true>(rv[k] + w.rb, iv[k] + w.ib, Z ? zv[k] : 0.0f);
      const float y = w.rate * g.r;
      const Decay dc = decay(y);
      const float a = dc.a;
      const float q = dc.v > 0.0f ? rsqrt_approx(dc.v) : 0.0f;
      bet[k] = dc.v * q;
      rho[k] = a * y * q;  // a rho
      yv[k] = y;
      rv[k] = g.r1;
      iv[k] = g.i;
      i1[k] = g.i1;
      if (Z) {
        // zv: dout silu'(z) (then times h); gv: dout silu(z)
        const float dy = gv[k];
        gv[k] = dy * zv[k] * g.sz;
        zv[k] = dy * g.sz * fmaf(zv[k], g.sz1, 1.0f);
      }
      const bool ok = m.valid >> k & 1u;
      av[k] = ok ? a : 1.0f;
      bv[k] = ok ? bet[k] * (g.i * xv[k]) : 0.0f;
      hp[k] = 0.0f;
      if (VL && (m.first >> k & 1u) && p.h0)
        hp[k] = p.h0[int64_t(seq_of(p.cu, p.S, t0 + k, m.seq)) * p.h0_sb + d * p.h0_sd];
      float ca = av[k], cb = bv[k];
      if (VL && (m.first >> k & 1u)) {
        cb = fmaf(a, hp[k], cb);
        ca = kResetA;
      }
      compose<VL>(ca, cb, A, B);
      A = ca;
      B = cb;
    }
    float hin = ckpt[tl];
    float hk = tile_carry<VL, false, W>(A, B, hin, s_buf, flip, wr, lane);
    // states before every step, and the adjoint's map of the window
#pragma unroll
    for (int k = 0; k < kGs; ++k) {
      if (!(VL && (m.first >> k & 1u))) hp[k] = hk;
      hk = fmaf(av[k], hp[k], bv[k]);
      if (Z) zv[k] *= hk;
    }
    A = 1.0f;
    B = 0.0f;
#pragma unroll
    for (int k = kGs - 1; k >= 0; --k) {
      if (!(m.valid >> k & 1u)) gv[k] = 0.0f;
      if ((m.last >> k & 1u) && p.dlast) {
        const int64_t sq = VL ? seq_of(p.cu, p.S, t0 + k, m.seq) : bt;
        gv[k] += p.dlast[sq * p.dl_sb + d * p.dl_sd];
      }
      float ca = av[k], cb = av[k] * gv[k];
      if (VL && (m.last >> k & 1u)) ca = kResetA;
      compose<VL>(ca, cb, A, B);
      A = ca;
      B = cb;
    }
    float ck = tile_carry<VL, true, W>(A, B, c, s_buf, flip, wr, lane);
#pragma unroll
    for (int k = kGs - 1; k >= 0; --k) {
      const float s = (VL && (m.last >> k & 1u)) ? gv[k] : gv[k] + ck;
      const float a = av[k];
      ck = a * s;
      if (VL && (m.first >> k & 1u) && p.dh0)
        p.dh0[int64_t(seq_of(p.cu, p.S, t0 + k, m.seq)) * p.dh_sb + d * p.dh_sd] = ck;
      const float ix = iv[k] * xv[k];
      const float ww = s * a * fmaf(ix, rho[k], -yv[k] * hp[k]);
      const float sb = s * bet[k];
      const float gr = rv[k] * ww;
      const float gi = sb * ix * i1[k];
      if (m.valid >> k & 1u) {
        sum_w += ww;
        sum_r += gr;
        sum_i += gi;
      }
      xv[k] = sb * iv[k];
      rv[k] = gr;
      iv[k] = gi;
    }
    win_store(dx, t0, m.valid, vec, xv);
    win_store(dr, t0, m.valid, vec, rv);
    win_store(di, t0, m.valid, vec, iv);
    if (Z) win_store(dz, t0, m.valid, vec, zv);
  }
  if (!VL && p.dh0 && lane == 0 && wr == 0)
    p.dh0[bt * p.dh_sb + d * p.dh_sd] = ntiles ? c : (p.dlast ? p.dlast[bt * p.dl_sb + d * p.dl_sd] : 0.0f);

  // the row's sums, in a fixed order
#pragma unroll
  for (int k = 16; k > 0; k /= 2) {
    sum_w += __shfl_down_sync(~0u, sum_w, k);
    sum_r += __shfl_down_sync(~0u, sum_r, k);
    sum_i += __shfl_down_sync(~0u, sum_i, k);
  }
  if constexpr (W > 1) {
    if (lane == 0) {
      s_red[warp] = sum_w;
      s_red[W + warp] = sum_r;
      s_red[2 * W + warp] = sum_i;
    }
    __syncthreads();
    if (warp == 0 && lane == 0)
      for (int k = 1; k < W; ++k) {
        sum_w += s_red[k];
        sum_r += s_red[W + k];
        sum_i += s_red[2 * W + k];
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
  const Gates g = gates<Z>(rv + w.rb, iv + w.ib, zv);
  const Decay dc = decay(w.rate * g.r);
  const float h = fmaf(dc.a, *st, sqrt_approx(dc.v) * (g.i * xv));
  *st = h;
  const float y = Z ? h * (zv * g.sz) : h;
  T* o = static_cast<T*>(p.out) + bt * p.o_sb + d * p.o_sd;
  if constexpr (sizeof(T) == 2) *o = f_to_bf16(y);
  else *o = y;
}

}  // namespace mssm
