// ops_common.cuh -- device helpers of the operators around the experts: rows of bf16, fp16 or fp32
// values moved 16 bytes at a time and computed on in fp32.
#pragma once

#include "../../include/moe.h"
#include "common.cuh"
#include "ops.h"

namespace moe {

template <typename T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
    static __device__ __forceinline__ void unpack(uint32_t w, float& a, float& b) {
        a = __uint_as_float(w << 16);
        b = __uint_as_float(w & 0xFFFF0000u);
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
};
template <> struct Elem<__half> {
    static __device__ __forceinline__ void unpack(uint32_t w, float& a, float& b) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        a = f.x;
        b = f.y;
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
};

// N consecutive values as 16-byte words (N * sizeof(T) a multiple of 16): loaded raw, so a thread
// can have many loads in flight, and widened to fp32 where they are used.
template <typename T, int N> struct Vec {
    static constexpr int kWords = N * (int)sizeof(T) / 16;
    uint4 w[kWords];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void store(T* p) const {
#pragma unroll
        for (int i = 0; i < kWords; ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
    }
    __device__ __forceinline__ void get(float (&v)[N]) const {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(T) == 4) v[4 * i + j] = __uint_as_float(u[j]);
                else Elem<T>::unpack(u[j], v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
            }
        }
    }
    __device__ __forceinline__ void set(const float (&v)[N]) {   // rounded to nearest, ties to even
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            uint32_t u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(T) == 4) u[j] = __float_as_uint(v[4 * i + j]);
                else u[j] = Elem<T>::pack(v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
            }
            w[i] = make_uint4(u[0], u[1], u[2], u[3]);
        }
    }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Device errors of these operators (MOE_STATUS_* bits): one word per source file and device, taken
// (read and cleared) by moe_ops_status.  `taken` receives the word on the device first, so a bit
// raised meanwhile by a kernel in another stream stays for the next call.
static __device__ uint32_t g_ops_status[2];
static __global__ void take_status_kernel() { g_ops_status[1] = atomicExch(&g_ops_status[0], 0u); }
static inline cudaError_t take_status(uint32_t* host, cudaStream_t st) {
    take_status_kernel<<<1, 1, 0, st>>>();
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess)
        e = cudaMemcpyFromSymbolAsync(host, g_ops_status, sizeof(uint32_t), sizeof(uint32_t), cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    return e;
}

// Calls F with a value of the element type that `dtype` names.
template <typename F> cudaError_t with_dtype(int dtype, F f) {
    switch (dtype) {
        case MOE_DTYPE_BF16: return f(__nv_bfloat16());
        case MOE_DTYPE_FP16: return f(__half());
        case MOE_DTYPE_FP32: return f(float());
    }
    return cudaErrorInvalidValue;
}

}  // namespace moe
