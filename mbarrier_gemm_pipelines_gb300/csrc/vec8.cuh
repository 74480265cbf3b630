// vec8.cuh -- eight neighbouring elements at a time, as fp32 in registers.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

namespace gbr {

__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(x[i] << 16);
        v[2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        x[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(x[0], x[1], x[2], x[3]);
}

// The first `count` (below 8: the rest zero) of eight elements at any address.
__device__ __forceinline__ uint4 load8_raw(const __nv_bfloat16* p, int32_t count) {
    uint32_t x[4] = {};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < count) x[j / 2] |= uint32_t(__bfloat16_as_ushort(p[j])) << (16 * (j % 2));
    return make_uint4(x[0], x[1], x[2], x[3]);
}

// 16-byte aligned addresses.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    unpack8(*reinterpret_cast<const uint4*>(p), v);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) = pack8(v);
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

}  // namespace gbr
