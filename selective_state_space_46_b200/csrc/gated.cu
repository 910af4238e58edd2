// Instantiation and launch of the gated linear recurrence's forward scan and decode step.
#include "launch.h"

namespace mssm {

template <typename T, int W, bool Z, bool CL>
static cudaError_t scan_v(const GatedArgs& a, cudaStream_t s) {
  if (a.cu) return gated_launch(gated_scan_kernel<T, W, Z, true, CL>, a, W, 0, s);
  return gated_launch(gated_scan_kernel<T, W, Z, false, CL>, a, W, 0, s);
}

template <typename T, int W, bool CL>
static cudaError_t scan_w(const GatedArgs& a, cudaStream_t s) {
  return a.z ? scan_v<T, W, true, CL>(a, s) : scan_v<T, W, false, CL>(a, s);
}

template <typename T>
static cudaError_t scan_t(const GatedArgs& a, int warps, cudaStream_t s) {
  if (a.split > 1) return scan_w<T, 8, true>(a, s);
  return warps == 1 ? scan_w<T, 1, false>(a, s)
         : warps == 2 ? scan_w<T, 2, false>(a, s)
         : warps == 4 ? scan_w<T, 4, false>(a, s) : scan_w<T, 8, false>(a, s);
}

cudaError_t launch_gated_scan(const GatedArgs& a, int warps, int dtype, cudaStream_t s) {
  return dtype == 1 ? scan_t<uint16_t>(a, warps, s) : scan_t<float>(a, warps, s);
}

template <typename T, int V, int R>
static cudaError_t step_r(const GatedStepArgs& a, cudaStream_t s) {
  const int64_t n = int64_t((a.D + V - 1) / V) * ((a.Bt + R - 1) / R);
  const unsigned g = unsigned((n + kStepThreads - 1) / kStepThreads);
  if (a.z)
    gated_step_kernel<T, V, R, true><<<g, kStepThreads, 0, s>>>(a);
  else
    gated_step_kernel<T, V, R, false><<<g, kStepThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
static cudaError_t step_t(const GatedStepArgs& a, bool vec, int rows, cudaStream_t s) {
  if (!vec) return rows > 1 ? step_r<T, 1, 2>(a, s) : step_r<T, 1, 1>(a, s);
  return rows > 1 ? step_r<T, 4, 2>(a, s) : step_r<T, 4, 1>(a, s);
}

cudaError_t launch_gated_step(const GatedStepArgs& a, bool vec, int rows, int dtype, cudaStream_t s) {
  return dtype == 1 ? step_t<uint16_t>(a, vec, rows, s) : step_t<float>(a, vec, rows, s);
}

}  // namespace mssm
