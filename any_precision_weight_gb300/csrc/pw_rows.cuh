// What the operators on rows share: element types, 16-byte loads, argument checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <nvtx3/nvToolsExt.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "pw_internal.h"

namespace pw {

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }

// The 16 / sizeof(T) elements of one 16-byte load, as fp32.
template <typename T>
__device__ __forceinline__ void unpack16(const uint4& raw, float (&v)[16 / sizeof(T)]) {
  const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
  for (int i = 0; i < static_cast<int>(16 / sizeof(T)); ++i) v[i] = to_f32<T>(e[i]);
}

// The larger of two numbers; NaN where either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

struct NvtxCall {
  explicit NvtxCall(const char* name) { nvtxRangePushA(name); }
  ~NvtxCall() { nvtxRangePop(); }
  NvtxCall(const NvtxCall&) = delete;
  NvtxCall& operator=(const NvtxCall&) = delete;
};

inline int failf(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline int failf(int code, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return set_error(code, buf);
}

inline int launch_status(cudaError_t e, const char* what) {
  return e == cudaSuccess ? PW_OK : failf(PW_ECUDA, "%s: launch: %s", what, cudaGetErrorString(e));
}

inline size_t dtype_bytes(int dtype) { return dtype == PW_F32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype == PW_F16 || dtype == PW_BF16 || dtype == PW_F32; }
inline bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Streaming multiprocessors of the current device (asked once per device).
int sm_count();

// A launch that may begin before the one ahead of it in the stream has left the GPU: its
// kernel calls after_those_before() before it touches memory.
template <typename... P, typename... A>
inline cudaError_t launch_close(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, int cluster, cudaStream_t s,
                                const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute a[2]{};
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  a[1].id = cudaLaunchAttributeClusterDimension;
  a[1].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
  cfg.attrs = a;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
// Everything before this kernel in its stream has ended, and its results can be read.
__device__ __forceinline__ void after_those_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel in the stream may begin (up to its own after_those_before()).  Called
// behind it, so that the next one begins after all that this one waited for; and not by
// kernels whose results may be router logits, which pw_moe_forward reads before it waits.
__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace pw
