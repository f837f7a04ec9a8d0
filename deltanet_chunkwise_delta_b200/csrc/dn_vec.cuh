// Element access shared by the operators around the delta-rule kernels: bf16 and fp32
// values in registers as fp32, alone or V at a time.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace dn {

template <typename E>
__device__ __forceinline__ float ld_elem(const E* p) {
    if constexpr (sizeof(E) == 2) return __bfloat162float(*p);
    else return *p;
}
template <typename E>
__device__ __forceinline__ void st_elem(E* p, float x) {
    if constexpr (sizeof(E) == 2) *p = __float2bfloat16_rn(x);
    else *p = x;
}

// Four consecutive elements (8-byte aligned bf16, 16-byte aligned fp32).
template <typename E>
__device__ __forceinline__ float4 ld_elem4(const E* p) {
    if constexpr (sizeof(E) == 2) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                           __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
    } else {
        return *reinterpret_cast<const float4*>(p);
    }
}
template <typename E>
__device__ __forceinline__ void st_elem4(E* p, float4 x) {
    if constexpr (sizeof(E) == 2) {
        __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
        *reinterpret_cast<uint2*>(p) =
            make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
    } else {
        *reinterpret_cast<float4*>(p) = x;
    }
}

// V = 1 or 2 consecutive elements as loaded (2: one 4- or 8-byte access), to and from fp32.
template <typename E, int V> struct RawVec;
template <> struct RawVec<__nv_bfloat16, 1> { using T = unsigned short; };
template <> struct RawVec<__nv_bfloat16, 2> { using T = uint32_t; };
template <> struct RawVec<float, 1> { using T = float; };
template <> struct RawVec<float, 2> { using T = float2; };

__device__ __forceinline__ void unpack(unsigned short r, float* f) { f[0] = __uint_as_float((uint32_t)r << 16); }
__device__ __forceinline__ void unpack(uint32_t r, float* f) {
    f[0] = __uint_as_float(r << 16);
    f[1] = __uint_as_float(r & 0xffff0000u);
}
__device__ __forceinline__ void unpack(float r, float* f) { f[0] = r; }
__device__ __forceinline__ void unpack(float2 r, float* f) {
    f[0] = r.x;
    f[1] = r.y;
}
__device__ __forceinline__ void pack(const float* f, unsigned short& r) {
    r = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
}
__device__ __forceinline__ void pack(const float* f, uint32_t& r) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[0], f[1]);
    r = *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ void pack(const float* f, float& r) { r = f[0]; }
__device__ __forceinline__ void pack(const float* f, float2& r) { r = make_float2(f[0], f[1]); }

template <typename E, int V>
__device__ __forceinline__ typename RawVec<E, V>::T ld_raw(const E* p) {
    return *reinterpret_cast<const typename RawVec<E, V>::T*>(p);
}
template <typename E, int V>
__device__ __forceinline__ void st_vec(E* p, const float* f) {
    typename RawVec<E, V>::T r;
    pack(f, r);
    *reinterpret_cast<typename RawVec<E, V>::T*>(p) = r;
}

// Two fp32 operations in one instruction (pairs of neighbours; d may be an operand).
__device__ __forceinline__ void fma2(const float* a, const float* b, const float* c, float* d) {
    asm("{ .reg .b64 a, b, c, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7};\n"
        "  fma.rn.f32x2 d, a, b, c; mov.b64 {%0, %1}, d; }"
        : "=f"(d[0]), "=f"(d[1])
        : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]), "f"(c[0]), "f"(c[1]));
}
__device__ __forceinline__ void add2(const float* a, const float* b, float* d) {
    asm("{ .reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5};\n"
        "  add.rn.f32x2 d, a, b; mov.b64 {%0, %1}, d; }"
        : "=f"(d[0]), "=f"(d[1])
        : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]));
}
__device__ __forceinline__ void mul2(const float* a, const float* b, float* d) {
    asm("{ .reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5};\n"
        "  mul.rn.f32x2 d, a, b; mov.b64 {%0, %1}, d; }"
        : "=f"(d[0]), "=f"(d[1])
        : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]));
}

// A [d] parameter vector in fp32 or bf16.
struct ParamVec {
    const void* p;  // null: not given
    int bf16;
    int vec;        // 16-byte aligned
};
__device__ __forceinline__ float ld_param(const ParamVec& v, int j) {
    return v.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(v.p)[j])
                  : static_cast<const float*>(v.p)[j];
}

}  // namespace dn
