// Instantiation and launch of the 4-bit linear map's kernels.
#include "launch.h"

namespace mssm {

template <typename T, typename S, int NT, int W, bool HALF, bool ZERO>
static cudaError_t w4_run(const W4Args& a, cudaStream_t s) {
  constexpr size_t smem = w4_smem<T, S, NT, W, HALF, ZERO>();
  const auto kernel = w4_linear_kernel<T, S, NT, W, HALF, ZERO>;
  if (smem > 48 * 1024) {  // once for every device; the caller holds the library's lock
    static uint64_t allowed = 0;
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && !(dev < 64 && (allowed >> dev & 1u))) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
      if (e == cudaSuccess && dev < 64) allowed |= uint64_t(1) << dev;
    }
    if (e != cudaSuccess) return e;
  }
  const dim3 g(unsigned((a.N + kW4Rows - 1) / kW4Rows), unsigned((a.M + 8 * NT - 1) / (8 * NT)));
  kernel<<<g, 32 * W, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T, typename S, int NT, int W>
static cudaError_t w4_w(const W4Args& a, cudaStream_t s) {
  if (a.group % kW4K != 0) return a.zero ? w4_run<T, S, NT, W, true, true>(a, s) : w4_run<T, S, NT, W, true, false>(a, s);
  return a.zero ? w4_run<T, S, NT, W, false, true>(a, s) : w4_run<T, S, NT, W, false, false>(a, s);
}

template <typename T, typename S, int NT>
static cudaError_t w4_n(const W4Args& a, int warps, cudaStream_t s) {
  return warps == 4 ? w4_w<T, S, NT, 4>(a, s) : warps == 8 ? w4_w<T, S, NT, 8>(a, s) : w4_w<T, S, NT, 16>(a, s);
}

template <typename T, typename S>
static cudaError_t w4_s(const W4Args& a, int warps, cudaStream_t s) {
  if (a.M <= 8) return w4_n<T, S, 1>(a, warps, s);
  if constexpr (sizeof(T) == 2)
    if (a.M > 16) return w4_n<T, S, 4>(a, warps, s);
  return w4_n<T, S, 2>(a, warps, s);  // fp32: the ring of 32 tokens' x would not fit
}

cudaError_t launch_w4_linear(const W4Args& a, int warps, int dtype, int scale_dtype, cudaStream_t s) {
  if (dtype == 1) return scale_dtype == 1 ? w4_s<uint16_t, uint16_t>(a, warps, s) : w4_s<uint16_t, float>(a, warps, s);
  return scale_dtype == 1 ? w4_s<float, uint16_t>(a, warps, s) : w4_s<float, float>(a, warps, s);
}

cudaError_t launch_w4_pack(const W4PackArgs& a, int scale_dtype, cudaStream_t s) {
  const int64_t n = int64_t(a.tiles) * a.blocks * 128 + int64_t(a.tiles) * a.groups * kW4Rows;
  const int64_t want = (n + 255) / 256;
  const unsigned g = unsigned(want < 65536 ? want : 65536);
  if (scale_dtype == 1)
    w4_pack_kernel<uint16_t><<<g, 256, 0, s>>>(a);
  else
    w4_pack_kernel<float><<<g, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace mssm
