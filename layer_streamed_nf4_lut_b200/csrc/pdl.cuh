// Programmatic dependent launch: a kernel is set up while the one before it on the stream ends, and touches
// memory only when that one's results are there.
#pragma once
#include <cuda_runtime.h>

#include <type_traits>

#include "internal.h"

namespace soup {

// In every thread, before the kernel's first access to memory that another kernel may have written, or may still
// read.  It waits for the whole kernel before, which has itself waited for the one before that.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel may be set up from here on (once every block of this one has come so far).
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

struct PdlLaunch {
  cudaLaunchConfig_t c{};
  cudaLaunchAttribute a{};
  PdlLaunch(unsigned grid, int threads, int smem, cudaStream_t st) {
    c.gridDim = dim3(grid);
    c.blockDim = dim3(static_cast<unsigned>(threads));
    c.dynamicSmemBytes = static_cast<size_t>(smem);
    c.stream = st;
    a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &a;
    c.numAttrs = 1;
    ++g_kernel_launches;
  }
};
template <typename... Params, typename... Args>
cudaError_t pdl_start(void (*kernel)(Params...), unsigned grid, int threads, int smem, cudaStream_t st, const Args&... args) {
  const PdlLaunch l(grid, threads, smem, st);
  return cudaLaunchKernelEx(&l.c, kernel, static_cast<Params>(args)...);
}
// The same for a kernel of one structure, which is not copied on the way (AdamW's has 28 KB).
template <typename P>
cudaError_t pdl_start_one(void (*kernel)(P), unsigned grid, int threads, int smem, cudaStream_t st,
                          const std::remove_const_t<P>& arg) {
  const PdlLaunch l(grid, threads, smem, st);
  void* args[1] = {const_cast<void*>(static_cast<const void*>(&arg))};
  return cudaLaunchKernelExC(&l.c, reinterpret_cast<const void*>(kernel), args);
}

}  // namespace soup
