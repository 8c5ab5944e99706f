// Shared by the language-model operators (route.cu, pages.cu,
// paged_attention.cu): errors of their C entry points, vectors of elements
// and their conversion to and from 32 bits.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "spmv.h"

namespace lbcsr {

// Records the calling thread's last error (spmv_last_error) and returns s.
spmv_status_t llm_fail(spmv_status_t s, const char *what, const char *detail = nullptr) noexcept;

inline spmv_status_t llm_bad(const char *what) noexcept { return llm_fail(SPMV_ERR_INVALID_ARG, what); }

inline spmv_status_t llm_launched(const char *what, cudaError_t e) noexcept {
    return e == cudaSuccess ? SPMV_OK : llm_fail(SPMV_ERR_CUDA, what, cudaGetErrorString(e));
}

inline bool elem_ok(int elem) { return elem == SPMV_ELEM_F32 || elem == SPMV_ELEM_BF16 || elem == SPMV_ELEM_F16; }
inline int elem_size(int elem) { return elem == SPMV_ELEM_F32 ? 4 : 2; }

inline bool aligned_to(const void *p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0; }

// The operators are chained: each kernel is launched while the one before it
// in the stream still runs, and waits for it (all of it, its writes visible)
// before it touches global memory; so a launch costs the stream about 2 us
// less.  after_previous() is every such kernel's first statement.  What the
// kernel before wrote is visible after it to ordinary loads only: a load
// through the read-only path is defined for data that nobody writes while the
// kernel lives, which begins before the wait, and may be moved above it.  So
// these kernels take no pointer as __restrict__ and use no __ldg; loads that
// are to be in flight together are written before the stores.
__device__ __forceinline__ void after_previous() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
// cluster: blocks in a cluster, 0: none.
template <typename... Params, typename... Args>
cudaError_t launch_chained(void (*kernel)(Params...), unsigned grid, unsigned block, size_t smem, unsigned cluster,
                           cudaStream_t stream, Args... args) {
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = cluster;
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3(grid);
    config.blockDim = dim3(block);
    config.dynamicSmemBytes = smem;
    config.stream = stream;
    config.attrs = attrs;
    config.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&config, kernel, static_cast<Params>(args)...);
}

// Division by a constant d, 1 <= d < 2^31 ("Division by Invariant Integers
// using Multiplication", Granlund and Montgomery, 1994, section 4): with
// 2^s >= d > 2^(s-1) and m = floor(2^32 (2^s - d) / d) + 1, t / d =
// (mulhi(m, t) + t) >> s for every t < 2^32; for t < 2^31 the sum fits 32 bits.
inline void set_divisor(uint32_t d, uint32_t *mul, uint32_t *shift) {
    uint32_t s = 0;
    while ((1ull << s) < d) ++s;
    *mul = (uint32_t)(((1ull << 32) * ((1ull << s) - d)) / d + 1);
    *shift = s;
}

// N consecutive elements, moved by one load or store of sizeof(Vec) bytes.
template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
    T v[N];
};

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

template <typename T>
__device__ __forceinline__ T zero_of() { return from_float<T>(0.0f); }

}  // namespace lbcsr
