// Vectors of 1 to 8 consecutive elements in one memory access, and the checks
// that choose their width.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "device_math.cuh"

namespace ms {

struct alignas(16) Raw32 { uint4 a, b; };   // eight float32 beside eight bfloat16

template <int BYTES> struct RawOf;
template <> struct RawOf<32> { using type = Raw32; };
template <> struct RawOf<16> { using type = uint4; };
template <> struct RawOf<8> { using type = uint2; };
template <> struct RawOf<4> { using type = uint32_t; };
template <> struct RawOf<2> { using type = uint16_t; };

template <typename T, int VEC> using Raw = typename RawOf<VEC * (int)sizeof(T)>::type;

template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> load_raw(const T *p) {
    if constexpr (sizeof(T) * VEC == 32)
        return {__ldg(reinterpret_cast<const uint4 *>(p)), __ldg(reinterpret_cast<const uint4 *>(p) + 1)};
    else
        return __ldg(reinterpret_cast<const Raw<T, VEC> *>(p));
}

template <typename T, int VEC>
__device__ __forceinline__ void store_raw(T *p, const Raw<T, VEC> &r) {
    *reinterpret_cast<Raw<T, VEC> *>(p) = r;
}

// Widen one raw vector to float32 (exact).
template <typename T, int VEC>
__device__ __forceinline__ void widen(const Raw<T, VEC> &r, float (&v)[VEC]) {
    union { Raw<T, VEC> r; T t[VEC]; uint32_t w[(VEC * sizeof(T) + 3) / 4]; } u;
    u.r = r;
    if constexpr (sizeof(T) == 2 && VEC >= 2) {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            v[2 * i] = bf16_lo(u.w[i]);
            v[2 * i + 1] = bf16_hi(u.w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = to_f32<T>(u.t[i]);
    }
}

// Round to the storage type (bf16: to nearest even).
template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> narrow(const float (&v)[VEC]) {
    union { Raw<T, VEC> r; T t[VEC]; __nv_bfloat162 b[(VEC + 1) / 2]; } u;
    if constexpr (sizeof(T) == 2 && VEC >= 2) {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) u.b[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) u.t[i] = from_f32<T>(v[i]);
    }
    return u.r;
}

// VEC float32 values from a pointer aligned to min(16, 4 VEC) bytes.
template <int VEC>
__device__ __forceinline__ void load_f32(const float *p, float (&v)[VEC]) {
    if constexpr (VEC >= 4) {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            const float4 q = __ldg(reinterpret_cast<const float4 *>(p) + i);
            v[4 * i] = q.x; v[4 * i + 1] = q.y; v[4 * i + 2] = q.z; v[4 * i + 3] = q.w;
        }
    } else if constexpr (VEC == 2) {
        const float2 q = __ldg(reinterpret_cast<const float2 *>(p));
        v[0] = q.x; v[1] = q.y;
    } else {
        v[0] = __ldg(p);
    }
}

// Whether a tensor (NULL: always) with this row stride, in elements of eb
// bytes, can be accessed in vectors of vec elements that start at multiples of vec.
inline bool vec_ok(const void *ptr, int64_t stride, int eb, int vec) {
    const int64_t bytes = static_cast<int64_t>(vec) * eb < 16 ? static_cast<int64_t>(vec) * eb : 16;
    return !ptr || (reinterpret_cast<uintptr_t>(ptr) % bytes == 0 && (stride * eb) % bytes == 0);
}

// sigmoid(z) = 1 / (1 + e^-z); e^-z = inf gives 0.
__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// sigmoid of a pair, 1 / (1 + e^-z), to a few float32 roundings (e^-z = inf gives 0).
__device__ __forceinline__ float2 sigmoid2(float2 z) {
    const float2 e = ex2x2(mul2(z, f2(-kLog2e, -kLog2e)));
    const float2 s = add2(e, f2(1.f, 1.f));
    float2 r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(s.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(s.y));
    return r;
}

// softplus close to float32 rounding (log1p(e) = e p(e), p of degree 9 by
// fit_log1p.py 9: 1.6e-7 relative), for steps that enter float32 states.
__device__ __forceinline__ float softplus_fine(float v) {
    const float e = ex2_approx(-fabsf(v) * kLog2e);
    float p = -0.0033387341536581516f;
    p = fmaf(p, e, 0.02027779072523117f);
    p = fmaf(p, e, -0.05775919556617737f);
    p = fmaf(p, e, 0.1068454384803772f);
    p = fmaf(p, e, -0.15353283286094666f);
    p = fmaf(p, e, 0.19692456722259521f);
    p = fmaf(p, e, -0.2495734840631485f);
    p = fmaf(p, e, 0.333302766084671f);
    p = fmaf(p, e, -0.49999913573265076f);
    p = fmaf(p, e, 1.0f);
    return fmaf(p, e, fmaxf(v, 0.f));
}

}  // namespace ms
