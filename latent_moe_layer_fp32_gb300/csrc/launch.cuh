// Host-side launch helper of the paged-cache operators: a kernel launched with
// programmatic stream serialisation (its griddepcontrol.wait orders it behind
// the launch before it), named and counted like every launch of the library.
#pragma once
#include <utility>

#include "kernels.cuh"

namespace lmoe {

template <typename... KArgs, typename... Args>
int launch_pdl(const char* name, dim3 grid, dim3 block, size_t smem, cudaStream_t s, void (*kern)(KArgs...),
               Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  pre_launch(s, name);
  if (cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...) != cudaSuccess) return LMOE_ECUDA;
  launched();
  return LMOE_OK;
}

// Raises a kernel's dynamic shared memory limit, once per device.  `done` is
// the kernel's own bit set of devices.
template <typename Mask, typename... KArgs>
int allow_smem(Mask& done, void (*kern)(KArgs...), int bytes) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return LMOE_ECUDA;
  if (done.load() >> (dev & 63) & 1ull) return LMOE_OK;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return LMOE_ECUDA;
  done.fetch_or(1ull << (dev & 63));
  return LMOE_OK;
}

// The optional status workspace of calls that need no scratch: LMOE_OK with
// *st set (null without a workspace), after zeroing the status word.
int optional_status(void* ws, size_t ws_bytes, cudaStream_t s, Status** st);
// LMOE_OK, LMOE_EINVAL or LMOE_EUNSUPPORTED for a cache descriptor; with
// `memory` false only its head count and width are looked at
int check_cache(const lmoe_kv_cache* c, bool memory);
int check_cache_fp8(const lmoe_kv_cache_fp8* c, bool memory);
// Whether no two rows of a cache share an element: in the order of their strides, each dimension steps past all
// that the ones below it span.
bool rows_apart(int64_t block_stride, int64_t n_blocks, int64_t head_stride, int64_t kv_heads, int64_t slot_stride,
                int64_t block_size, int64_t head_dim);

}  // namespace lmoe
