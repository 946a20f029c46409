// elem.cuh -- element types of the operators around the decoder blocks: loads
// that widen to binary32 (exact) and stores that round once, one element or
// four neighbours at a time.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace repro {

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v)
{
    return __bfloat162float(v);
}

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v)
{
    return __float2bfloat16_rn(v);
}

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p)
{
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                       __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
}

// the same for data that is read once and that no thread writes during the kernel
__device__ __forceinline__ float4 stream4(const float* p) { return ld_stream(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 stream4(const __nv_bfloat16* p)
{
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                       __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
}

__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v)
{
    uint2 o;
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    o.x = *reinterpret_cast<const unsigned*>(&a);
    o.y = *reinterpret_cast<const unsigned*>(&b);
    *reinterpret_cast<uint2*>(p) = o;
}

// 16 bytes: four binary32 or eight bf16 neighbours, widened
__device__ __forceinline__ void load16(const float* p, float* x)
{
    const float4 v = load4(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float* x)
{
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ void store16(float* p, const float* x) { store4(p, make_float4(x[0], x[1], x[2], x[3])); }
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float* x)
{
    unsigned w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const unsigned*>(&v);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// index i of a list of int32 (bytes 4) or int64 (bytes 8)
__device__ __forceinline__ int64_t load_index(const void* p, int bytes, int64_t i)
{
    return bytes == 8 ? __ldg(static_cast<const long long*>(p) + i)
                      : (int64_t)__ldg(static_cast<const int*>(p) + i);
}

// whether rows of T starting at p, `ld` elements apart, begin on 4-element boundaries
template <typename T> inline bool rows4(const void* p, int64_t ld)
{
    return (reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T))) == 0 && ld % 4 == 0;
}

} // namespace repro
