// Shared helpers of libgptq: status handling, launch accounting, element loads.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>
#include <stdint.h>

#include "gptq.h"

namespace gptq {

void note_launch();  // counts every kernel launch issued by the library
void note_error(cudaError_t e, const char* where);  // remembers the last CUDA failure

inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

inline size_t align256(size_t b) { return (b + 255) & ~size_t(255); }

__device__ __forceinline__ void raise_status(int32_t* st, int bits) {
  if (st) atomicOr(st, bits);
}

__device__ __forceinline__ float load_f32(const void* p, int dt, int64_t idx) {
  if (dt == GPTQ_F32) return static_cast<const float*>(p)[idx];
  if (dt == GPTQ_F16) return __half2float(static_cast<const __half*>(p)[idx]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[idx]);
}

// An NVTX range around one ABI call, so that a profiler can select a call's
// kernels (e.g. ncu --nvtx --nvtx-include "gptq_prepare/"); without a tool
// attached the push and pop return at once.
struct CallRange {
  explicit CallRange(const char* name) { nvtxRangePushA(name); }
  ~CallRange() { nvtxRangePop(); }
  CallRange(const CallRange&) = delete;
  CallRange& operator=(const CallRange&) = delete;
};

// Programmatic dependent launch: a grid launched with the attribute may start while its
// predecessor in the stream drains, once every CTA of that one has called allow_successor() or
// exited; it sets itself up and waits for the predecessor's end, and for its writes, here.  All
// threads of such a grid call wait_for_predecessor() before they touch global memory or start
// a bounded wait, and they read what earlier kernels wrote with plain loads: a read-only
// (non-coherent) load may hit a line that the SM cached while the predecessor was running, so
// such kernels take no __restrict__ const pointers.  Calls in a row then hide their launches
// and set-up: a product of 333 tokens with 11008 x 4104 weights takes 16.1 us on the device
// instead of 20.3.
__device__ __forceinline__ void wait_for_predecessor() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void allow_successor() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// The attribute that lets a grid start early.
inline cudaLaunchAttribute may_start_early() {
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  return at;
}

template <typename... P, typename... A>
inline cudaError_t launch_early(void (*kernel)(P...), dim3 grid, dim3 block, cudaStream_t stream,
                                A... args) {
  cudaLaunchAttribute at = may_start_early();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Opt a kernel into more than 48 KB of dynamic shared memory (idempotent).
template <typename K>
inline cudaError_t allow_smem(K kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

}  // namespace gptq

// Launch a kernel, count it, and turn a launch error into GPTQ_ERR_CUDA.
#define GPTQ_LAUNCH(kernel, grid, block, smem, stream, ...)                 \
  do {                                                                      \
    kernel<<<(grid), (block), (smem), (stream)>>>(__VA_ARGS__);             \
    ::gptq::note_launch();                                                  \
    const cudaError_t e_ = cudaGetLastError();                              \
    if (e_ != cudaSuccess) {                                                \
      ::gptq::note_error(e_, #kernel);                                      \
      return GPTQ_ERR_CUDA;                                                 \
    }                                                                       \
  } while (0)

// Count a launch that `call` (cudaLaunchKernelEx) made, or turn its error into GPTQ_ERR_CUDA and
// clear it, so that the next launch is not blamed for it.
#define GPTQ_LAUNCHED(call, name)                                           \
  do {                                                                      \
    const cudaError_t e_ = (call);                                          \
    if (e_ != cudaSuccess) {                                                \
      (void)cudaGetLastError();                                             \
      ::gptq::note_error(e_, name);                                         \
      return GPTQ_ERR_CUDA;                                                 \
    }                                                                       \
    ::gptq::note_launch();                                                  \
  } while (0)

// A launch that may start early: of a kernel that calls wait_for_predecessor() (no dynamic
// shared memory).
#define GPTQ_LAUNCH_EARLY(kernel, grid, block, stream, ...) \
  GPTQ_LAUNCHED(::gptq::launch_early(kernel, grid, block, stream, __VA_ARGS__), #kernel)

#define GPTQ_CUDA(call)                                                     \
  do {                                                                      \
    const cudaError_t e_ = (call);                                          \
    if (e_ != cudaSuccess) {                                                \
      ::gptq::note_error(e_, #call);                                        \
      return GPTQ_ERR_CUDA;                                                 \
    }                                                                       \
  } while (0)

#define GPTQ_TRY(expr)                          \
  do {                                          \
    gptq_status s_ = (expr);                    \
    if (s_ != GPTQ_OK) return s_;               \
  } while (0)
