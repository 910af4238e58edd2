// Instantiation and launch of the 4-bit linear map's kernels.
#include "launch.h"

namespace mssm {

template <typename T, typename S, int NT>
static cudaError_t w4_n(const W4Args& a, cudaStream_t s) {
  const dim3 g(unsigned((a.N + kW4Rows - 1) / kW4Rows), unsigned((a.M + 8 * NT - 1) / (8 * NT)));
  const bool half = a.group % kW4K != 0;
  if (half) {
    if (a.zero) w4_linear_kernel<T, S, NT, true, true><<<g, 32 * kW4Warps, 0, s>>>(a);
    else w4_linear_kernel<T, S, NT, true, false><<<g, 32 * kW4Warps, 0, s>>>(a);
  } else {
    if (a.zero) w4_linear_kernel<T, S, NT, false, true><<<g, 32 * kW4Warps, 0, s>>>(a);
    else w4_linear_kernel<T, S, NT, false, false><<<g, 32 * kW4Warps, 0, s>>>(a);
  }
  return cudaGetLastError();
}

template <typename T, typename S>
static cudaError_t w4_s(const W4Args& a, cudaStream_t s) {
  if (a.M <= 8) return w4_n<T, S, 1>(a, s);
  return w4_n<T, S, 2>(a, s);
}

cudaError_t launch_w4_linear(const W4Args& a, int dtype, int scale_dtype, cudaStream_t s) {
  if (dtype == 1) return scale_dtype == 1 ? w4_s<uint16_t, uint16_t>(a, s) : w4_s<uint16_t, float>(a, s);
  return scale_dtype == 1 ? w4_s<float, uint16_t>(a, s) : w4_s<float, float>(a, s);
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
