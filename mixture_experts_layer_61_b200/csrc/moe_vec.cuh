// moe_vec.cuh -- 16-byte vectors of the activation dtype as fp32 values.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace moe {

template <typename T>
struct Vec16 {
    static constexpr int N = 16 / sizeof(T);
};

__device__ __forceinline__ void unpack(const int4& v, float* f, const __nv_bfloat16*) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = __bfloat1622float2(h[i]);
        f[2 * i] = x.x;
        f[2 * i + 1] = x.y;
    }
}
__device__ __forceinline__ void unpack(const int4& v, float* f, const float*) {
    const float* x = reinterpret_cast<const float*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = x[i];
}
__device__ __forceinline__ int4 pack(const float* f, const __nv_bfloat16*) {
    int4 v;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    return v;
}
__device__ __forceinline__ int4 pack(const float* f, const float*) {
    int4 v;
    float* x = reinterpret_cast<float*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = f[i];
    return v;
}

}  // namespace moe
