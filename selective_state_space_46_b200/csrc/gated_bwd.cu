// Instantiation and launch of the gated linear recurrence's backward scan.
#include "launch.h"

namespace mssm {

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

template <typename T, int W, bool Z, bool CL>
static cudaError_t bwd_v(const GatedArgs& a, size_t smem, cudaStream_t s) {
  if (a.cu) return gated_launch(gated_bwd_kernel<T, W, Z, true, CL>, a, W, smem, s);
  return gated_launch(gated_bwd_kernel<T, W, Z, false, CL>, a, W, smem, s);
}

template <typename T, int W, bool CL>
static cudaError_t bwd_w(const GatedArgs& a, size_t smem, cudaStream_t s) {
  return a.z ? bwd_v<T, W, true, CL>(a, smem, s) : bwd_v<T, W, false, CL>(a, smem, s);
}

template <typename T>
static cudaError_t bwd_t(const GatedArgs& a, int warps, size_t smem, cudaStream_t s) {
  if (a.split > 1) return bwd_w<T, 8, true>(a, smem, s);
  return warps == 1 ? bwd_w<T, 1, false>(a, smem, s)
         : warps == 2 ? bwd_w<T, 2, false>(a, smem, s)
         : warps == 4 ? bwd_w<T, 4, false>(a, smem, s) : bwd_w<T, 8, false>(a, smem, s);
}

cudaError_t launch_gated_bwd(const GatedArgs& a, int warps, int dtype, cudaStream_t s) {
  const size_t smem = size_t(warps == 1 ? 4 : 1) * size_t(a.ntiles) * 4;
  const cudaError_t e = dtype == 1 ? bwd_t<uint16_t>(a, warps, smem, s) : bwd_t<float>(a, warps, smem, s);
  if (e != cudaSuccess || !a.part) return e;
  gated_param_grads_kernel<<<unsigned((a.D + 127) / 128), 128, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace mssm
