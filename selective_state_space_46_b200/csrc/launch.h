// Internal host-side launch interface between the C ABI layer and the kernels.
#pragma once

#include <cuda_runtime.h>

#include "bwd.cuh"
#include "conv.cuh"
#include "decode.cuh"
#include "gated.cuh"
#include "scan.cuh"
#include "w4.cuh"

namespace mssm {

// dtype: 0 = fp32 storage, 1 = bf16 storage.  Return the launch error, if any.
// rows: channels per row tile (32, 64 or 128), rpt: rows per thread (1 or 2; 2 for bf16 only),
// so rows / rpt threads per CTA; the grid is (Bt * tiles_per_batch, nseg [- 1]).
cudaError_t launch_scan_chunk_state(const ScanArgs& a, int rows, int rpt, int dtype, bool softplus, cudaStream_t s);
cudaError_t launch_scan_out(const ScanArgs& a, int rows, int rpt, int dtype, bool has_z, bool softplus,
                            cudaStream_t s);
// Persistent chained forward kernel (row tiles of 32 * rpt channels), `grid` one-warp CTAs.
cudaError_t launch_scan_chained(const ScanArgs& a, int grid, int rpt, int dtype, bool has_z, bool softplus,
                                cudaStream_t s);
// Fused single-pass (look-back) kernel (row tiles of 32 * rpt channels), `grid` one-warp CTAs.
cudaError_t launch_scan_fused(const ScanArgs& a, int grid, int rpt, int dtype, bool has_z, bool softplus,
                              cudaStream_t s);
// Split-chunk kernel (row tiles of 32 * rpt channels), `grid` persistent CTAs of kSplitWarps
// warps; seg_len is kSplitWarps sub-segments.
cudaError_t launch_scan_split(const ScanArgs& a, int grid, int rpt, int dtype, bool has_z, bool softplus,
                              cudaStream_t s);
// Device address of this device's error word (cached per device).
cudaError_t device_error_word(unsigned int** out);
// Drops every cached device address of a module symbol (after this, the next call looks
// them up again: a device reset may load the module at another address).
void forget_device_addresses();
// Incremented by forget_device_addresses: caches of per-device setup compare against it.
int device_address_generation();

// Lets `kernel` use `bytes` of dynamic shared memory (above the 48 KB default), once per
// device, and again after mssm_shutdown (a device reset drops it).  set_gen: the caller's
// own per-device record for this kernel (the address generation it was set in, + 1).
template <typename K>
cudaError_t opt_in_smem(K kernel, int bytes, int (&set_gen)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  const int gen = device_address_generation() + 1;
  if (set_gen[dev] != gen) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    set_gen[dev] = gen;
  }
  return cudaSuccess;
}

// bulk: the state is one contiguous [rows][16] range (bulk-copy kernel), else one thread per row.
enum class DecodePath { kStream, kBulkTile, kPerRow };
cudaError_t launch_state_update(const DecodeArgs& a, int dtype, bool has_z, DecodePath path, cudaStream_t s);
// Causal conv1d + SiLU: grid (ceil(rows / kConvWarps), items); one decode step of it.
cudaError_t launch_causal_conv1d(const ConvArgs& a, int items, int dtype, bool silu, cudaStream_t s);
cudaError_t launch_causal_conv1d_update(const ConvUpdateArgs& a, int dtype, cudaStream_t s);
// Backward scan: pass A (chunk summaries both ways and their folds, when there is more than
// one chunk) and pass B (recompute and backward sweep per chunk).
cudaError_t launch_scan_bwd(const BwdArgs& a, int dtype, bool has_z, cudaStream_t s);
// Gated linear recurrence: `warps` (1, 2, 4 or 8) warps of a CTA per row, and a.split CTAs (above 1: 8 warps,
// and a cluster).  The backward pass is followed by the sum of the batch's row sums when a.part is given.
cudaError_t launch_gated_scan(const GatedArgs& a, int warps, int dtype, cudaStream_t s);
cudaError_t launch_gated_bwd(const GatedArgs& a, int warps, int dtype, cudaStream_t s);
// `vec`: 4 channels a thread (every pointer and row stride allows it); `rows`: batch rows a thread, 1 or 2.
cudaError_t launch_gated_step(const GatedStepArgs& a, bool vec, int rows, int dtype, cudaStream_t s);
// 4-bit linear map: the layout of a weight, and the product.
cudaError_t launch_w4_pack(const W4PackArgs& a, int scale_dtype, cudaStream_t s);
struct W4Plan {
  int tiles, warps;  // of a CTA: 2 tiles and 8 warps, or 1 tile and 8 or 16 warps
};
cudaError_t launch_w4_linear(const W4Args& a, W4Plan plan, int dtype, int scale_dtype, cudaStream_t s);
// Reads (and optionally clears) the current device's error word.
cudaError_t read_device_error(unsigned int* value, bool clear);

}  // namespace mssm
