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
  int tiles, blocks, groups, group;   // tiles of 16 outputs; blocks of 64 inputs; groups stored per tile; inputs per group
  int group_shift;             // log2(group / 32), or -1 when the group is no power of two
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

// the 8 inputs of a lane, from its places in shared memory (512 bytes apart) in pieces of 16 bytes
template <typename T>
__device__ __forceinline__ XFrag<T> x_frag(const char* at) {
  XFrag<T> f;
  const uint4 u = *reinterpret_cast<const uint4*>(at);
  if constexpr (sizeof(T) == 2) {
    f.v[0][0] = u.x; f.v[0][1] = u.y; f.v[0][2] = u.z; f.v[0][3] = u.w;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(at + 512);
    const float e[8] = {__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w),
                        __uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w)};
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

// The scales of outputs g and g + 8 are a pair of 4 or 8 bytes, read as fp32.
__device__ __forceinline__ float2 scale_pair(const float* s) { return *reinterpret_cast<const float2*>(s); }
__device__ __forceinline__ float2 scale_pair(const uint16_t* s) {
  const uint32_t u = *reinterpret_cast<const uint32_t*>(s);
  return make_float2(bf16lo(u), bf16hi(u));
}

// Asks for 8 inputs of a token, from k on.  inner: all of them exist and start on a 16-byte boundary; otherwise
// zeros stand behind the last one, fp32 comes by the element and bf16 through registers.
template <typename T>
__device__ __forceinline__ void x_ask(unsigned to, const T* x, int k, int K, bool inner) {
  if (inner) {
#pragma unroll
    for (int v = 0; v < int(sizeof(T)) / 2; ++v)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(to + v * 512), "l"(x + v * (16 / sizeof(T))) : "memory");
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool in = k + j < K;
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to + j / 4 * 512 + 4 * (j % 4)), "l"(x - k + (in ? k + j : 0)),
                   "r"(in ? 4 : 0)
                   : "memory");
    }
  } else {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      u[j] = (k + 2 * j < K ? uint32_t(x[2 * j]) : 0u) | (k + 2 * j + 1 < K ? uint32_t(x[2 * j + 1]) << 16 : 0u);
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]) : "memory");
  }
}

// One CTA per TT tiles of 16 outputs and 8 * NT tokens; its W warps take every W-th block of 64 inputs and add up
// in shared memory, in order.  HALF: the group is an odd multiple of 32, so both halves of a block have
// their own scale.  Every lane has its 16 bytes of the next blocks, their scales and its x on the way into its
// own places of shared memory (no other lane reads them, so the copies' own order is all the
// synchronisation).  One token is bound by the instructions that unpack the codes as much as by the stream
// of weights: 60 a block of 1024 codes, beside those of the loop and of x, which two tiles share.  Warp-level
// products of 16 x 8 x 16 suit 8 to 32 tokens; a tile of 128 rows in tensor memory would stay mostly empty.
// 1x5120x20480 bf16: 22.6 us a call (2.4 TB/s, ALU pipe 63%); 32x5120x20480: 53 us with the launch.
template <typename T, typename S, int NT, int TT, bool HALF, bool ZERO>
struct W4Ring {
  static constexpr int kSets = HALF ? 2 : 1;
  static constexpr int kPair = 2 * int(sizeof(S));
  static constexpr int kXPart = 32 * 8 * int(sizeof(T));  // of half a block and 8 tokens
  // places in a slot: weights, x, scales, zero points
  static constexpr int kX = 512 * TT, kScale = kX + 2 * NT * kXPart, kZero = kScale + 32 * kPair * kSets * TT;
  static constexpr int kSlot = kZero + (ZERO ? 32 * 4 * kSets * TT : 0);
  // about 7 KB of a warp, so that 32 warps of an SM have 48 KB of weights on the way
  static constexpr int kSlots = 7168 / kSlot > 6 ? 6 : 7168 / kSlot < 2 ? 2 : 7168 / kSlot;
  static constexpr int kWarp = kSlot * kSlots;
};

template <typename T, typename S, int NT, int TT, int W, bool HALF, bool ZERO>
__global__ void __launch_bounds__(32 * W) w4_linear_kernel(const W4Args p) {
  using Ring = W4Ring<T, S, NT, TT, HALF, ZERO>;
  constexpr int kSlots = Ring::kSlots, kSets = Ring::kSets;
  extern __shared__ __align__(16) char s_mem[];  // the warps' rings, then their sums
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, c = lane % 4;
  const int tile0 = blockIdx.x * TT, m0 = blockIdx.y * (8 * NT);
  // a last CTA without a second tile computes its first one twice
  const int64_t next_q = TT > 1 && tile0 + 1 < p.tiles ? int64_t(p.blocks) * 32 : 0;
  const int64_t next_s = TT > 1 && tile0 + 1 < p.tiles ? int64_t(p.groups) * 16 : 0;
  const uint4* q = p.q + (int64_t(tile0) * p.blocks + warp) * 32 + lane;
  const S* scale = static_cast<const S*>(p.scale) + (int64_t(tile0) * p.groups * 8 + g) * 2;
  const uint8_t* zero = ZERO ? p.zero + (int64_t(tile0) * p.groups * 8 + (g & ~1)) * 2 : nullptr;  // 4 bytes: g and g ^ 1
  const T* xr[NT];
  bool on[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int m = m0 + 8 * n + g;
    on[n] = m < p.M;
    xr[n] = static_cast<const T*>(p.x) + (on[n] ? m : 0) * p.x_sm + warp * kW4K + 8 * c;
  }
  // tokens behind the last one are zeros, which nothing overwrites
#pragma unroll
  for (int n = 0; n < NT; ++n)
    if (!on[n])
      for (int k = 0; k < kSlots; ++k)
        for (int e = 0; e < 2 * int(Ring::kXPart / 512); ++e)
          *reinterpret_cast<uint4*>(s_mem + warp * Ring::kWarp + k * Ring::kSlot + Ring::kX + 2 * n * Ring::kXPart + e * 512 + lane * 16) =
              make_uint4(0u, 0u, 0u, 0u);
  const unsigned ring = unsigned(__cvta_generic_to_shared(s_mem)) + warp * Ring::kWarp, ring_end = ring + Ring::kWarp;
  // the pointers are those of the block that is asked for next
  int asked = warp;
  unsigned to = ring;
  auto ask = [&] {
    if (asked < p.blocks) {
#pragma unroll
      for (int t = 0; t < TT; ++t)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + t * 512 + lane * 16), "l"(q + t * next_q) : "memory");
      const int k = asked * kW4K + 8 * c;
      const bool inner = p.vec_x && (asked + 1) * kW4K <= p.K;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (on[n])
#pragma unroll
          for (int h = 0; h < 2; ++h)
            x_ask(to + Ring::kX + (2 * n + h) * Ring::kXPart + lane * 16, xr[n] + 32 * h, k + 32 * h, p.K, inner);
#pragma unroll
      for (int h = 0; h < kSets; ++h) {
        const unsigned u = unsigned(2 * asked + h);  // in units of 32 inputs
        const unsigned grp = p.group_shift >= 0 ? u >> p.group_shift : u / unsigned(p.group / 32);
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to + Ring::kScale + (32 * (kSets * t + h) + lane) * Ring::kPair),
                       "l"(scale + size_t(grp) * 16 + t * next_s), "n"(Ring::kPair)
                       : "memory");
          if (ZERO)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + Ring::kZero + (32 * (kSets * t + h) + lane) * 4),
                         "l"(zero + size_t(grp) * 16 + t * next_s)
                         : "memory");
        }
      }
      q += 32 * W;
#pragma unroll
      for (int n = 0; n < NT; ++n) xr[n] += W * kW4K;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    asked += W;
    to += Ring::kSlot;
    if (to == ring_end) to = ring;
  };
#pragma unroll
  for (int j = 0; j < kSlots - 1; ++j) ask();

  float acc[TT][NT][4];
#pragma unroll
  for (int e = 0; e < TT * NT * 4; ++e) (&acc[0][0][0])[e] = 0.0f;
  const char* at = s_mem + warp * Ring::kWarp;
  for (int kb = warp; kb < p.blocks; kb += W) {
    ask();
    asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 1) : "memory");
    uint32_t wlo[TT][2], whi[TT][2];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const uint4 w = *reinterpret_cast<const uint4*>(at + t * 512 + lane * 16);
      wlo[t][0] = w.x; wlo[t][1] = w.y; whi[t][0] = w.z; whi[t][1] = w.w;
    }
    float part[TT][NT][4];
    uint32_t z0[TT], z1[TT];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int set = HALF ? h : 0;
      if (h == 0 || HALF) {
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          z0[t] = z1[t] = 0x43084308u;
          if (ZERO) {
            const uint32_t zz = *reinterpret_cast<const uint32_t*>(at + Ring::kZero + (32 * (kSets * t + set) + lane) * 4) >> (16 * (g & 1));
            z0[t] = (zz & 0xffu) * 0x10001u | 0x43004300u;
            z1[t] = (zz >> 8 & 0xffu) * 0x10001u | 0x43004300u;
          }
        }
#pragma unroll
        for (int e = 0; e < TT * NT * 4; ++e) (&part[0][0][0])[e] = 0.0f;
      }
      uint32_t a[TT][2][4];
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          a[t][s][0] = w4_pair(wlo[t][h], 2 * s, z0[t]);
          a[t][s][1] = w4_pair(whi[t][h], 2 * s, z1[t]);
          a[t][s][2] = w4_pair(wlo[t][h], 2 * s + 1, z0[t]);
          a[t][s][3] = w4_pair(whi[t][h], 2 * s + 1, z1[t]);
        }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const XFrag<T> xf = x_frag<T>(at + Ring::kX + (2 * n + h) * Ring::kXPart + lane * 16);
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int e = 0; e < XFrag<T>::kParts; ++e) mma_bf16(part[t][n], a[t][s], xf.v[e][2 * s], xf.v[e][2 * s + 1]);
      }
      if (h == 1 || HALF) {
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const float2 sc = scale_pair(reinterpret_cast<const S*>(at + Ring::kScale + (32 * (kSets * t + set) + lane) * Ring::kPair));
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            acc[t][n][0] = fmaf(sc.x, part[t][n][0], acc[t][n][0]);
            acc[t][n][1] = fmaf(sc.x, part[t][n][1], acc[t][n][1]);
            acc[t][n][2] = fmaf(sc.y, part[t][n][2], acc[t][n][2]);
            acc[t][n][3] = fmaf(sc.y, part[t][n][3], acc[t][n][3]);
          }
        }
      }
    }
    at += Ring::kSlot;
    if (at == s_mem + (warp + 1) * Ring::kWarp) at -= Ring::kWarp;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  // accumulator element: rows g (0, 1) and g + 8 (2, 3), tokens 2c and 2c + 1
  float* s_acc = reinterpret_cast<float*>(s_mem);  // [W][8 NT][16 TT + 1]
  constexpr int kRow = kW4Rows * TT + 1;
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        s_acc[(warp * 8 * NT + 8 * n + 2 * c + (k & 1)) * kRow + kW4Rows * t + g + 8 * (k >> 1)] = acc[t][n][k];
  __syncthreads();
  for (int e = threadIdx.x; e < 8 * NT * kW4Rows * TT; e += 32 * W) {
    const int m = e / (kW4Rows * TT), r = e % (kW4Rows * TT);
    const int64_t n = int64_t(tile0) * kW4Rows + r;
    if (m0 + m >= p.M || n >= p.N) continue;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < W; ++k) v += s_acc[(k * 8 * NT + m) * kRow + r];
    if (p.bias) v += p.bias[n * p.bias_s];
    T* o = static_cast<T*>(p.out) + (m0 + m) * p.o_sm + n * p.o_sn;
    if constexpr (sizeof(T) == 2) *o = f_to_bf16(v);
    else *o = v;
  }
}

// shared memory of a CTA
template <typename T, typename S, int NT, int TT, int W, bool HALF, bool ZERO>
constexpr size_t w4_smem() {
  const size_t ring = size_t(W) * W4Ring<T, S, NT, TT, HALF, ZERO>::kWarp,
               sums = size_t(W) * 8 * NT * (kW4Rows * TT + 1) * 4;
  return ring > sums ? ring : sums;
}

}  // namespace mssm
