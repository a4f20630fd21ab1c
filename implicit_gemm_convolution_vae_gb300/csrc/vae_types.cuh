// Element types of the token operators: f32, f16 and bf16 loads and stores,
// eight elements (16 bytes of a 16-bit type) or one at a time, always through
// f32 registers with one rounding to nearest even on the way out.
#pragma once

#include <cuda_bf16.h>

#include "vae_common.cuh"

namespace vae {

inline bool type_ok(int t) { return t == VAE_F32 || t == VAE_F16 || t == VAE_BF16; }
inline size_t type_size(int t) { return t == VAE_F32 ? 4u : 2u; }

template <int T>
struct Elem;
template <>
struct Elem<VAE_F32> {
    using type = float;
};
template <>
struct Elem<VAE_F16> {
    using type = __half;
};
template <>
struct Elem<VAE_BF16> {
    using type = __nv_bfloat16;
};

template <int T>
__device__ __forceinline__ float to_f32(typename Elem<T>::type v) {
    if constexpr (T == VAE_F32) return v;
    else if constexpr (T == VAE_F16) return __half2float(v);
    else return __bfloat162float(v);
}
template <int T>
__device__ __forceinline__ typename Elem<T>::type from_f32(float v) {
    if constexpr (T == VAE_F32) return v;
    else if constexpr (T == VAE_F16) return __float2half_rn(v);
    else return __float2bfloat16_rn(v);
}

// Two f32 packed to 16 bits each (a in the low half).
template <int T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    static_assert(T != VAE_F32, "16-bit types");
    if constexpr (T == VAE_F16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}
template <int T>
__device__ __forceinline__ float2 unpack2(uint32_t u) {
    if constexpr (T == VAE_F16) return __half22float2(*reinterpret_cast<const __half2*>(&u));
    else return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
}

// Pairs of f32 in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

// Eight consecutive elements at a 16-byte aligned address.
template <int T>
__device__ __forceinline__ void load8(const void* p, float (&v)[8]) {
    if constexpr (T == VAE_F32) {
        const float4 a = *static_cast<const float4*>(p), b = *(static_cast<const float4*>(p) + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 a = *static_cast<const uint4*>(p);
        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2<T>(u[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}
template <int T>
__device__ __forceinline__ void store8(void* p, const float (&v)[8]) {
    if constexpr (T == VAE_F32) {
        *static_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *(static_cast<float4*>(p) + 1) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *static_cast<uint4*>(p) = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]),
                                             pack2<T>(v[6], v[7]));
    }
}

}  // namespace vae
