// Launchers of the 16-bit operators (layer norm, rotary positions, linear).
// The entry points beside them validate; these only launch.
#pragma once

#include "overlap.h"
#include "svdq_internal.h"

namespace svdq {

// Rotary frequencies as fractions of a turn (times 2^64) and each pair's
// axis; passed to the kernel by value.
struct alignas(16) RopeTurns {
  uint64_t turn[SVDQ_ROPE_MAX_PAIRS + 8];     // zeros past the pairs
  uint8_t axis[SVDQ_ROPE_MAX_PAIRS + 8];
  int pairs, axes;
};

inline bool is_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Rows of `ld` elements of `esize` bytes start on 16-byte boundaries.
inline bool rows_aligned16(const void* p, int ld, int esize) {
  return is_aligned16(p) && ((long long)ld * esize) % 16 == 0;
}

// Launch of a 16-bit operator's kernel: it may start while the kernel before
// it in the stream runs out (its blocks then set up their shared memory and
// wait), which hides the launch behind that kernel's last blocks.  Every such
// kernel calls grid_wait() in all its threads before it touches global
// memory, so that what it reads and overwrites is in order.  It reads with
// plain loads or copies: a non-coherent load (ld.global.nc) wants memory that
// nothing writes while the kernel is resident, and the kernel before it does.
template <typename... P, typename... A>
cudaError_t launch_op(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster,
                      cudaStream_t st, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// The status of a CUDA result.  The runtime keeps a failed call's error for the
// thread until it is read; it is read here, since the call answers with its
// status and the next check of a launch, the library's or its user's, would
// take the old error for its own.
inline svdq_status status_of(cudaError_t e) {
  if (e == cudaSuccess) return SVDQ_OK;
  (void)cudaGetLastError();
  return SVDQ_ERR_CUDA;
}

inline int dtype_size(int dtype) { return dtype == SVDQ_DTYPE_F32 ? 4 : 2; }

}  // namespace svdq
