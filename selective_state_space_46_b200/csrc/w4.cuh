// Linear map with 4-bit weights and group scales for a few tokens (sm_100a).
//
//   y[m, n] = sum_k x[m, k] scale[n, k / group] (code[n, k] - zero[n, k / group]) + bias[n]
//
// At a few tokens the product is the stream of its weights.  The weight is laid out once in the order
// in which a warp's lanes consume it: for every 16 outputs and 64 inputs one 512-byte block, 16 bytes
// per lane, which unpack into the A fragments of four m16n8k16 products (outputs as rows, tokens as
// columns).  Lane 4 g + c holds outputs g and g + 8 and the inputs [8c, 8c + 8) of both halves of the
// 64 (the order of the summed index is free as long as x takes the same one), so its x is contiguous
// too.  A code becomes the bf16 number 128 + code by or-ing it into the mantissa; subtracting
// 128 + zero is exact, the products of bf16 pairs are exact, and every group's sum is scaled in fp32.
// fp32 activations are three bf16 numbers whose sum is exact.
#pragma once

#include <cstdint>

#include "device_common.cuh"

namespace mssm {

constexpr int kW4Rows = 16;    // outputs per tile
constexpr int kW4K = 64;       // inputs per block
constexpr int kW4Warps = 8;    // warps per CTA; they split the inputs

struct W4Args {
  const void* x;               // [M, K], k stride 1
  int64_t x_sm;
  const uint4* q;              // [tiles][blocks][32 lanes]
  const void* scale;           // [tiles][groups][8][2]: outputs g and g + 8
  const uint8_t* zero;         // the same, or null: 8
  const float* bias;           // [N] or null
  int64_t bias_s;
  void* out;                   // [M, N]
  int64_t o_sm, o_sn;
  int M, N, K;
  int blocks, groups, group;   // blocks of 64 inputs; groups stored per tile; inputs per group
  bool vec_x;                  // rows of x start on 16-byte boundaries
};

struct W4PackArgs {
  const uint8_t* codes;        // [N, (K + 1) / 2]: even inputs in the low nibble
  int64_t c_sn, c_sk;
  const void* scale;           // [N, G]
  int64_t s_sn, s_sg;
  const uint8_t* zero;         // [N, G] or null
  int64_t z_sn, z_sg;
  uint32_t* q;
  void* q_scale;
  uint8_t* q_zero;
  int N, K, G, group;
  int tiles, blocks, groups;
};

// one thread per packed word (8 codes) and, in the same grid, per packed scale
template <typename S>
__global__ void __launch_bounds__(256) w4_pack_kernel(const W4PackArgs p) {
  const int64_t words = int64_t(p.tiles) * p.blocks * 128, scales = int64_t(p.tiles) * p.groups * kW4Rows;
  for (int64_t at = int64_t(blockIdx.x) * 256 + threadIdx.x; at < words + scales; at += int64_t(gridDim.x) * 256) {
    if (at >= words) {
      const int64_t e = at - words;
      const int half = int(e & 1), g = int(e >> 1 & 7);
      const int64_t tg = e >> 4;
      const int grp = int(tg % p.groups);
      const int64_t n = tg / p.groups * kW4Rows + g + 8 * half;
      const bool in = n < p.N && grp < p.G;
      static_cast<S*>(p.q_scale)[e] = in ? static_cast<const S*>(p.scale)[n * p.s_sn + grp * p.s_sg] : S(0);
      if (p.q_zero) p.q_zero[e] = in ? (p.zero[n * p.z_sn + grp * p.z_sg] & 15) : 8;
      continue;
    }
    const int w = int(at & 3), lane = int(at >> 2 & 31);
    const int64_t tb = at >> 7;
    const int64_t n = tb / p.blocks * kW4Rows + lane / 4 + 8 * (w / 2);
    const int64_t k0 = tb % p.blocks * kW4K + 32 * (w % 2) + 8 * (lane % 4);
    uint32_t v = 0;
    for (int j = 0; j < 8; ++j) {
      const int64_t k = k0 + j;
      uint32_t code = 8;
      if (n < p.N && k < p.K) {
        code = p.codes[n * p.c_sn + k / 2 * p.c_sk] >> (4 * (k & 1)) & 15u;
      } else if (p.zero && n < p.N && k / p.group < p.G) {
        code = p.zero[n * p.z_sn + k / p.group * p.z_sg] & 15u;  // behind the last input: the weight 0
      }
      v |= code << (4 * (j / 2) + 16 * (j & 1));
    }
    p.q[at] = v;
  }
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// pair j of a word as bf16 (128 + code) - zero
__device__ __forceinline__ uint32_t w4_pair(uint32_t w, int j, uint32_t zero) {
  return sub_bf16x2((w >> (4 * j) & 0x000f000fu) | 0x43004300u, zero);
}

// 8 consecutive inputs of a token as bf16 pairs, in `P` parts whose sum is the input (1 for bf16, 3 for fp32)
template <typename T>
struct XFrag {
  static constexpr int kParts = sizeof(T) == 2 ? 1 : 3;
  uint32_t v[kParts][4];
};

// fp32 as three bf16 numbers: the upper 16 bits, those of the rest, and what is left, all exact.
// Truncation keeps finite values finite; an infinity or NaN stays in the first part alone.
__device__ __forceinline__ void split3(float x, uint32_t& a, uint32_t& b, uint32_t& c) {
  const uint32_t u = __float_as_uint(x);
  const bool fin = (u & 0x7f800000u) != 0x7f800000u;
  const uint32_t h = fin ? u & 0xffff0000u : (u & 0x007fffffu ? 0x7fc00000u : u);
  const float r1 = fin ? x - __uint_as_float(h) : 0.0f;
  const uint32_t m = __float_as_uint(r1) & 0xffff0000u;
  const float r2 = r1 - __uint_as_float(m);
  a = h >> 16;
  b = m >> 16;
  c = __float_as_uint(r2) >> 16;
}

template <typename T>
__device__ __forceinline__ XFrag<T> x_load(const T* x, int k, int K, bool on, bool vec) {
  XFrag<T> f;
  if constexpr (sizeof(T) == 2) {
    if (on && vec && k + 8 <= K) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(x + k));
      f.v[0][0] = u.x; f.v[0][1] = u.y; f.v[0][2] = u.z; f.v[0][3] = u.w;
      return f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = on && k + 2 * j < K ? x[k + 2 * j] : 0u, hi = on && k + 2 * j + 1 < K ? x[k + 2 * j + 1] : 0u;
      f.v[0][j] = lo | hi << 16;
    }
  } else {
    float e[8];
    if (on && vec && k + 8 <= K) {
      const float4 u = __ldg(reinterpret_cast<const float4*>(x + k)), v = __ldg(reinterpret_cast<const float4*>(x + k) + 1);
      e[0] = u.x; e[1] = u.y; e[2] = u.z; e[3] = u.w; e[4] = v.x; e[5] = v.y; e[6] = v.z; e[7] = v.w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = on && k + j < K ? x[k + j] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t a0, b0, c0, a1, b1, c1;
      split3(e[2 * j], a0, b0, c0);
      split3(e[2 * j + 1], a1, b1, c1);
      f.v[0][j] = a0 | a1 << 16;
      f.v[1][j] = b0 | b1 << 16;
      f.v[2][j] = c0 | c1 << 16;
    }
  }
  return f;
}

__device__ __forceinline__ float2 load_scale2(const float* s, int64_t at) {
  return __ldg(reinterpret_cast<const float2*>(s) + at);
}
__device__ __forceinline__ float2 load_scale2(const uint16_t* s, int64_t at) {
  const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(s) + at);
  return make_float2(bf16lo(u), bf16hi(u));
}

// One CTA per 16 outputs and 8 * NT tokens; its warps take every kW4Warps-th block of 64 inputs and add up
// in shared memory, in order.  HALF: the group is an odd multiple of 32, so both halves of a block have
// their own scale.
template <typename T, typename S, int NT, bool HALF, bool ZERO>
__global__ void __launch_bounds__(32 * kW4Warps) w4_linear_kernel(const W4Args p) {
  __shared__ float s_acc[kW4Warps][NT * 8][kW4Rows + 1];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, c = lane % 4;
  const int tile = blockIdx.x, m0 = blockIdx.y * (8 * NT);
  const uint4* q = p.q + int64_t(tile) * p.blocks * 32 + lane;
  const S* scale = static_cast<const S*>(p.scale);
  const int64_t sbase = int64_t(tile) * p.groups * 8 + g;
  const T* xr[NT];
  bool on[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int m = m0 + 8 * n + g;
    on[n] = m < p.M;
    xr[n] = static_cast<const T*>(p.x) + (on[n] ? m : 0) * p.x_sm;
  }
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[n][k] = 0.0f;

  for (int kb = warp; kb < p.blocks; kb += kW4Warps) {
    const uint4 w = __ldg(q + int64_t(kb) * 32);
    const uint32_t wlo[2] = {w.x, w.y}, whi[2] = {w.z, w.w};
    float part[NT][4];
    float2 sc;
    uint32_t z0 = 0x43084308u, z1 = 0x43084308u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 0 || HALF) {
        const int grp = (kb * kW4K + 32 * h) / p.group;
        sc = load_scale2(scale, sbase + int64_t(grp) * 8);
        if (ZERO) {
          const uint32_t zz = __ldg(reinterpret_cast<const uint16_t*>(p.zero) + sbase + int64_t(grp) * 8);
          z0 = (zz & 0xffu) * 0x10001u | 0x43004300u;
          z1 = (zz >> 8) * 0x10001u | 0x43004300u;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) part[n][k] = 0.0f;
      }
      XFrag<T> xf[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) xf[n] = x_load(xr[n], kb * kW4K + 32 * h + 8 * c, p.K, on[n], p.vec_x);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint32_t a[4] = {w4_pair(wlo[h], 2 * s, z0), w4_pair(whi[h], 2 * s, z1), w4_pair(wlo[h], 2 * s + 1, z0),
                               w4_pair(whi[h], 2 * s + 1, z1)};
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int t = 0; t < XFrag<T>::kParts; ++t) mma_bf16(part[n], a, xf[n].v[t][2 * s], xf[n].v[t][2 * s + 1]);
      }
      if (h == 1 || HALF) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          acc[n][0] = fmaf(sc.x, part[n][0], acc[n][0]);
          acc[n][1] = fmaf(sc.x, part[n][1], acc[n][1]);
          acc[n][2] = fmaf(sc.y, part[n][2], acc[n][2]);
          acc[n][3] = fmaf(sc.y, part[n][3], acc[n][3]);
        }
      }
    }
  }
  // accumulator element: rows g (0, 1) and g + 8 (2, 3), tokens 2c and 2c + 1
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int k = 0; k < 4; ++k) s_acc[warp][8 * n + 2 * c + (k & 1)][g + 8 * (k >> 1)] = acc[n][k];
  __syncthreads();
  for (int e = threadIdx.x; e < 8 * NT * kW4Rows; e += 32 * kW4Warps) {
    const int m = e / kW4Rows, r = e % kW4Rows;
    const int n = tile * kW4Rows + r;
    if (m0 + m >= p.M || n >= p.N) continue;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < kW4Warps; ++k) v += s_acc[k][m][r];
    if (p.bias) v += p.bias[n * p.bias_s];
    T* o = static_cast<T*>(p.out) + (m0 + m) * p.o_sm + n * p.o_sn;
    if constexpr (sizeof(T) == 2) *o = f_to_bf16(v);
    else *o = v;
  }
}

}  // namespace mssm
