// ops_common.cuh -- what the handle-free operators (rows.cu, norm.cu, w4.cu) share: element types,
// vector loads and stores with conversion to fp32, argument checks and launches.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"
#include "ptx.cuh"

namespace moe {

constexpr int kSms = 148;   // SMs of a B200; grids of persistent blocks are multiples of it

// ---- host side -----------------------------------------------------------------

inline bool op_aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// a required pointer: present and 16-byte aligned
inline bool op_ptr(const void *p) { return p && op_aligned16(p); }

inline bool op_overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + nb && y < x + na;
}

inline size_t dtype_size(int dtype) { return dtype == MOE_F32 ? 4 : 2; }
inline bool dtype_known(int dtype) { return dtype == MOE_BF16 || dtype == MOE_F16 || dtype == MOE_F32; }

// MOE_OK if the current device can run the library's sm_100a code
int op_device();

// launch with the attributes the operators use; pdl: the kernel may be scheduled while its
// predecessor on the stream ends and waits for it itself (griddep_wait)
template <class... P, class... A>
cudaError_t op_launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, bool pdl, int cluster,
                      A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
    if (e != cudaSuccess) cudaGetLastError();   // reported through the status, not left behind
    return e;
}

// ---- device side ---------------------------------------------------------------

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// N consecutive elements, held as they are in memory; moved in 16-byte pieces where N spans them
template <class T, int N>
struct alignas((N * sizeof(T) >= 16) ? 16 : N * sizeof(T)) Vec {
    T v[N];
};

// read once, not read again by this kernel: do not keep it in L1
template <class T, int N>
__device__ __forceinline__ Vec<T, N> ld_vec(const T *p)
{
    Vec<T, N> r;
    constexpr int B = N * sizeof(T);
    if constexpr (B >= 16) {
        uint4 *w = reinterpret_cast<uint4 *>(r.v);
#pragma unroll
        for (int i = 0; i < B / 16; ++i) w[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
    } else if constexpr (B == 8) {
        *reinterpret_cast<uint2 *>(r.v) = __ldg(reinterpret_cast<const uint2 *>(p));
    } else if constexpr (B == 4) {
        *reinterpret_cast<uint32_t *>(r.v) = __ldg(reinterpret_cast<const uint32_t *>(p));
    } else {
        *reinterpret_cast<uint16_t *>(r.v) = __ldg(reinterpret_cast<const uint16_t *>(p));
    }
    return r;
}

template <class T, int N>
__device__ __forceinline__ void st_vec(T *p, const Vec<T, N> &r)
{
    constexpr int B = N * sizeof(T);
    if constexpr (B >= 16) {
        const uint4 *w = reinterpret_cast<const uint4 *>(r.v);
#pragma unroll
        for (int i = 0; i < B / 16; ++i) reinterpret_cast<uint4 *>(p)[i] = w[i];
    } else if constexpr (B == 8) {
        *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(r.v);
    } else if constexpr (B == 4) {
        *reinterpret_cast<uint32_t *>(p) = *reinterpret_cast<const uint32_t *>(r.v);
    } else {
        *reinterpret_cast<uint16_t *>(p) = *reinterpret_cast<const uint16_t *>(r.v);
    }
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace moe
