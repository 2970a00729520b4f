// ops_common.cuh -- what the handle-free operators (rows.cu, norm.cu, w4.cu) share: element types,
// vector loads and stores with conversion to fp32, argument checks and launches.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cstring>
#include <type_traits>

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

// the status of a runtime call; a failure is reported through it and not left behind for the next call to report again
inline int op_status(cudaError_t e)
{
    if (e == cudaSuccess) return MOE_OK;
    cudaGetLastError();
    return MOE_ECUDA;
}

// MOE_OK if the current device can run the library's sm_100a code
int op_device();

// Launch with the attributes the operators use.  early: the kernel may be scheduled while its predecessor on the stream
// ends; it begins with op_begin(), which waits for that end.
template <class... P, class... A>
cudaError_t op_launch_when(bool early, void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, int cluster,
                           A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (early) {
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

template <class... P, class... A>
cudaError_t op_launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, int cluster, A... args)
{
    return op_launch_when(true, kernel, grid, block, smem, s, cluster, args...);
}

// ---- device side ---------------------------------------------------------------

// The first thing every thread does: wait until all earlier work on the stream has ended and its writes are visible,
// then let the next launch get its blocks ready behind this one's.  In this order, so that a launch never
// begins before the work two launches back has ended.  Saves the launch gap of 2 to 3 us between kernels.
__device__ __forceinline__ void op_begin()
{
    griddep_wait();
    griddep_launch_dependents();
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// two fp32 values as one word of a 16-bit type
template <class T> __device__ __forceinline__ uint32_t pack2(float a, float b)
{
    uint32_t w;
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(a, b);
        memcpy(&w, &h, 4);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        memcpy(&w, &h, 4);
    }
    return w;
}

// N consecutive elements as the words they are in memory (16-bit elements unpacked one by one would take
// a register each)
template <class T, int N>
struct Raw {
    static constexpr int B = N * static_cast<int>(sizeof(T)), NW = (B + 3) / 4;
    uint32_t w[NW];
    // through the read-only path: what is loaded must not be written by the same kernel
    __device__ __forceinline__ void load(const T *p)
    {
        if constexpr (B >= 16) {
#pragma unroll
            for (int i = 0; i < NW / 4; ++i) {
                const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p) + i);
                w[4 * i] = u.x;
                w[4 * i + 1] = u.y;
                w[4 * i + 2] = u.z;
                w[4 * i + 3] = u.w;
            }
        } else if constexpr (B == 8) {
            const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
            w[0] = u.x;
            w[1] = u.y;
        } else if constexpr (B == 4) {
            w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
        } else {
            w[0] = __ldg(reinterpret_cast<const uint16_t *>(p));
        }
    }
    __device__ __forceinline__ void store(T *p) const
    {
        if constexpr (B >= 16) {
#pragma unroll
            for (int i = 0; i < NW / 4; ++i)
                reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        } else if constexpr (B == 8) {
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        } else if constexpr (B == 4) {
            *reinterpret_cast<uint32_t *>(p) = w[0];
        } else {
            *reinterpret_cast<uint16_t *>(p) = static_cast<uint16_t>(w[0]);
        }
    }
    // element e (a constant after unrolling)
    __device__ __forceinline__ float get(int e) const
    {
        if constexpr (sizeof(T) == 4) {
            return __uint_as_float(w[e]);
        } else if constexpr (std::is_same<T, __half>::value) {
            __half2 h;
            memcpy(&h, &w[e / 2], 4);
            return e & 1 ? __high2float(h) : __low2float(h);
        } else {
            return __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
        }
    }
    // all elements, from f(e)
    template <class F> __device__ __forceinline__ void set(F &&f)
    {
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(f(i));
            else w[i] = pack2<T>(f(2 * i), N > 1 ? f(2 * i + 1) : 0.f);
        }
    }
};

// two fp32 values in one 64-bit register pair: sm_100 adds, multiplies and fuses both in one instruction
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float x, float y)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpack(F2 a)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

// elements 2 i and 2 i + 1 of 16 bytes of T as fp32, and the way back
template <class T> __device__ __forceinline__ F2 pair_of(const uint4 &u, int i);
__device__ __forceinline__ uint32_t word_of(const uint4 &u, int i) { return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w; }
template <> __device__ __forceinline__ F2 pair_of<float>(const uint4 &u, int i)
{
    return f2(__uint_as_float(word_of(u, 2 * i)), __uint_as_float(word_of(u, 2 * i + 1)));
}
template <> __device__ __forceinline__ F2 pair_of<__nv_bfloat16>(const uint4 &u, int i)
{
    const uint32_t w = word_of(u, i);
    return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <> __device__ __forceinline__ F2 pair_of<__half>(const uint4 &u, int i)
{
    const uint32_t w = word_of(u, i);
    __half2 h;
    memcpy(&h, &w, 4);
    const float2 f = __half22float2(h);
    return f2(f.x, f.y);
}
// pair i of 16 bytes of T
template <class T> __device__ __forceinline__ void set_pair(uint32_t (&w)[4], int i, F2 a)
{
    const float2 f = unpack(a);
    if constexpr (sizeof(T) == 4) {
        w[2 * i] = __float_as_uint(f.x);
        w[2 * i + 1] = __float_as_uint(f.y);
    } else {
        w[i] = pack2<T>(f.x, f.y);
    }
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace moe
