// Instantiation and launch of the gated linear recurrence's kernels.
#include "launch.h"

namespace mssm {

template <typename T, int W, bool Z>
static cudaError_t scan_v(const GatedArgs& a, cudaStream_t s) {
  const int64_t rows = int64_t(a.Bt) * a.D;
  const unsigned g = unsigned((rows + kGatedWarps / W - 1) / (kGatedWarps / W));
  if (a.cu)
    gated_scan_kernel<T, W, Z, true><<<g, 32 * kGatedWarps, 0, s>>>(a);
  else
    gated_scan_kernel<T, W, Z, false><<<g, 32 * kGatedWarps, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T, int W>
static cudaError_t scan_w(const GatedArgs& a, cudaStream_t s) {
  return a.z ? scan_v<T, W, true>(a, s) : scan_v<T, W, false>(a, s);
}

template <typename T>
static cudaError_t scan_t(const GatedArgs& a, int warps, cudaStream_t s) {
  return warps == 1 ? scan_w<T, 1>(a, s) : scan_w<T, kGatedWarps>(a, s);
}

cudaError_t launch_gated_scan(const GatedArgs& a, int warps, int dtype, cudaStream_t s) {
  return dtype == 1 ? scan_t<uint16_t>(a, warps, s) : scan_t<float>(a, warps, s);
}

// the batch's row sums, added in order
static __global__ void gated_param_grads_kernel(const GatedArgs p) {
  const int d = blockIdx.x * blockDim.x + threadIdx.x;
  if (d >= p.D) return;
  const int64_t n = int64_t(p.Bt) * p.D;
  float w = 0.0f, r = 0.0f, i = 0.0f;
  for (int b = 0; b < p.Bt; ++b) {
    const int64_t at = int64_t(b) * p.D + d;
    w += p.part[at];
    r += p.part[n + at];
    i += p.part[2 * n + at];
  }
  const float lam = p.lam[d * p.lam_s], sp = softplus_exact(lam);
  // softplus underflows together with the logistic function, whose ratio to it tends to 1
  p.dlam[d] = w * (sp > 0.0f ? logistic_exact(lam) / sp : 1.0f);
  if (p.drb) p.drb[d] = r;
  if (p.dib) p.dib[d] = i;
}

template <typename T, int W, bool Z>
static cudaError_t bwd_v(const GatedArgs& a, cudaStream_t s) {
  const int64_t rows = int64_t(a.Bt) * a.D;
  const int per = kGatedWarps / W;
  const unsigned g = unsigned((rows + per - 1) / per);
  const size_t smem = size_t(per) * size_t(a.ntiles) * 4;
  if (a.cu)
    gated_bwd_kernel<T, W, Z, true><<<g, 32 * kGatedWarps, smem, s>>>(a);
  else
    gated_bwd_kernel<T, W, Z, false><<<g, 32 * kGatedWarps, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T, int W>
static cudaError_t bwd_w(const GatedArgs& a, cudaStream_t s) {
  return a.z ? bwd_v<T, W, true>(a, s) : bwd_v<T, W, false>(a, s);
}

template <typename T>
static cudaError_t bwd_t(const GatedArgs& a, int warps, cudaStream_t s) {
  return warps == 1 ? bwd_w<T, 1>(a, s) : bwd_w<T, kGatedWarps>(a, s);
}

cudaError_t launch_gated_bwd(const GatedArgs& a, int warps, int dtype, cudaStream_t s) {
  cudaError_t e = dtype == 1 ? bwd_t<uint16_t>(a, warps, s) : bwd_t<float>(a, warps, s);
  if (e != cudaSuccess || !a.part) return e;
  gated_param_grads_kernel<<<unsigned((a.D + 127) / 128), 128, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
static cudaError_t step_t(const GatedStepArgs& a, cudaStream_t s) {
  const unsigned g = unsigned((int64_t(a.Bt) * a.D + 255) / 256);
  if (a.z)
    gated_step_kernel<T, true><<<g, 256, 0, s>>>(a);
  else
    gated_step_kernel<T, false><<<g, 256, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_gated_step(const GatedStepArgs& a, int dtype, cudaStream_t s) {
  return dtype == 1 ? step_t<uint16_t>(a, s) : step_t<float>(a, s);
}

}  // namespace mssm
