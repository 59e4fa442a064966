// zt_host.h -- host helpers shared by the C ABI's translation units: the last
// CUDA error, launch status, occupancy and opt-in shared memory, and the TMA
// descriptor encoder.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace zt {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// last CUDA error seen by a library call on this host thread (diagnostics only)
extern thread_local cudaError_t g_last_cuda_error;

// Launch status: clear a stale non-sticky error left by an earlier, unrelated
// runtime call before launching (so it is not blamed on this launch), then
// read and clear the launch's own error.
inline void clear_stale_error() { (void)cudaGetLastError(); }
int launch_status();

// Resident CTAs per SM for (kernel, block, smem) on the current device, and
// the device's SM count; -1 if the kernel cannot run there.  On first use of a
// kernel on a device its dynamic shared memory limit is raised once to the
// device's opt-in maximum, so every later launch of any size fits.
int resident_ctas(const void *fn, int threads, size_t smem, int &sms);

// cuTensorMapEncodeTiled, looked up once through the runtime (no link to the
// driver library needed); null when it is unavailable.
PFN_cuTensorMapEncodeTiled_v12000 tma_encoder();

}  // namespace zt
