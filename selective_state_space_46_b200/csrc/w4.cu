// Instantiation and launch of the 4-bit linear map's kernels.
#include "launch.h"

namespace mssm {

template <typename T, typename S, int NT, int TT, int W, bool HALF, bool ZERO>
static cudaError_t w4_run(const W4Args& a, cudaStream_t s) {
  constexpr size_t smem = w4_smem<T, S, NT, TT, W, HALF, ZERO>();
  const auto kernel = w4_linear_kernel<T, S, NT, TT, W, HALF, ZERO>;
  if (smem > 48 * 1024) {
    static int set_gen[64] = {};  // one record per kernel instantiation
    const cudaError_t e = opt_in_smem(kernel, int(smem), set_gen);
    if (e != cudaSuccess) return e;
  }
  const dim3 g(unsigned((a.tiles + TT - 1) / TT), unsigned((a.M + 8 * NT - 1) / (8 * NT)));
  kernel<<<g, 32 * W, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T, typename S, int NT, int TT, int W>
static cudaError_t w4_w(const W4Args& a, cudaStream_t s) {
  if (a.group % kW4K != 0)
    return a.zero ? w4_run<T, S, NT, TT, W, true, true>(a, s) : w4_run<T, S, NT, TT, W, true, false>(a, s);
  return a.zero ? w4_run<T, S, NT, TT, W, false, true>(a, s) : w4_run<T, S, NT, TT, W, false, false>(a, s);
}

template <typename T, typename S, int NT>
static cudaError_t w4_n(const W4Args& a, W4Plan plan, cudaStream_t s) {
  if (plan.tiles == 2) return w4_w<T, S, NT, 2, 8>(a, s);
  return plan.warps == 8 ? w4_w<T, S, NT, 1, 8>(a, s) : w4_w<T, S, NT, 1, 16>(a, s);
}

template <typename T, typename S>
static cudaError_t w4_s(const W4Args& a, W4Plan plan, cudaStream_t s) {
  if (a.M <= 8) return w4_n<T, S, 1>(a, plan, s);
  if constexpr (sizeof(T) == 2)
    if (a.M > 16) return w4_n<T, S, 4>(a, plan, s);
  return w4_n<T, S, 2>(a, plan, s);  // fp32: the ring of 32 tokens' x would not fit
}

cudaError_t launch_w4_linear(const W4Args& a, W4Plan plan, int dtype, int scale_dtype, cudaStream_t s) {
  if (dtype == 1) return scale_dtype == 1 ? w4_s<uint16_t, uint16_t>(a, plan, s) : w4_s<uint16_t, float>(a, plan, s);
  return scale_dtype == 1 ? w4_s<float, uint16_t>(a, plan, s) : w4_s<float, float>(a, plan, s);
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
