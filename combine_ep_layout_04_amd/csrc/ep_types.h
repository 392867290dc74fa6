// ep_types.h -- the element types of the router, permute and 4-bit product
// kernels: 16-byte vectors of bf16, fp16 or fp32, unpacked to fp32.
//
// Conversions to 16 bits round to nearest even: the error is at most half a
// step (2^-9 of the value's binade for bf16, 2^-12 for fp16) on top of the
// fp32 value; a value past fp16's range becomes an infinity.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ep {

struct Bf16 {
    uint16_t bits;
};
struct Fp16 {
    uint16_t bits;
};

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 fp16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(Bf16 v) { return __uint_as_float((uint32_t)v.bits << 16); }
__device__ __forceinline__ float to_float(Fp16 v) { return (float)__builtin_bit_cast(_Float16, v.bits); }

template <typename T>
__device__ __forceinline__ T from_float(float f);
template <>
__device__ __forceinline__ float from_float<float>(float f)
{
    return f;
}
template <>
__device__ __forceinline__ Bf16 from_float<Bf16>(float f)
{
    return Bf16{__builtin_bit_cast(uint16_t, (__bf16)f)};
}
template <>
__device__ __forceinline__ Fp16 from_float<Fp16>(float f)
{
    return Fp16{__builtin_bit_cast(uint16_t, (_Float16)f)};
}

// One 16-byte vector holds kVec elements of T.
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

__device__ __forceinline__ void unpack(const uint4& d, float (&f)[4], const float*)
{
    f[0] = __uint_as_float(d.x);
    f[1] = __uint_as_float(d.y);
    f[2] = __uint_as_float(d.z);
    f[3] = __uint_as_float(d.w);
}
__device__ __forceinline__ void unpack(const uint4& d, float (&f)[8], const Bf16*)
{
    const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack(const uint4& d, float (&f)[8], const Fp16*)
{
    const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const fp16x2_t h = __builtin_bit_cast(fp16x2_t, w[i]);
        f[2 * i] = (float)h.x;
        f[2 * i + 1] = (float)h.y;
    }
}
template <typename T>
__device__ __forceinline__ void unpack(const uint4& d, float (&f)[kVec<T>])
{
    unpack(d, f, static_cast<const T*>(nullptr));
}

__device__ __forceinline__ uint4 pack(const float (&f)[4], const float*)
{
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 pack(const float (&f)[8], const Bf16*)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f32x2_t p = {f[2 * i], f[2 * i + 1]};
        w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2_t));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 pack(const float (&f)[8], const Fp16*)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f32x2_t p = {f[2 * i], f[2 * i + 1]};
        w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, fp16x2_t));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float (&f)[kVec<T>])
{
    return pack(f, static_cast<const T*>(nullptr));
}

// 16 bytes at any multiple of T's size (the hardware takes unaligned vector
// accesses to global memory; the attribute keeps the compiler from assuming
// more than the element's alignment).
template <typename T>
struct Unaligned16;
template <>
struct Unaligned16<float> {
    typedef uint32_t type __attribute__((ext_vector_type(4), aligned(4)));
};
template <>
struct Unaligned16<Bf16> {
    typedef uint32_t type __attribute__((ext_vector_type(4), aligned(2)));
};
template <>
struct Unaligned16<Fp16> {
    typedef uint32_t type __attribute__((ext_vector_type(4), aligned(2)));
};

}  // namespace ep
