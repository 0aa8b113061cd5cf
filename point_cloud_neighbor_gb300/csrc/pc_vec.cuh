// pc_vec.cuh -- element types of the token operators (layer norm, rotary,
// attention): float32 and bfloat16 in memory, float32 in registers, loaded
// and stored V elements at a time.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace pcn {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float2 unpack_bf16(uint32_t u) {
    // a bfloat16 is the upper half of the float32 of the same value
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// Two float32 rounded to bfloat16 (to nearest even), `lo` in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// V elements of T at p (aligned to V * sizeof(T)).
template <class T, int V>
struct Vec;

template <>
struct Vec<float, 1> {
    static __device__ __forceinline__ void load(const float *p, float *v) { v[0] = *p; }
    static __device__ __forceinline__ void store(float *p, const float *v) { *p = v[0]; }
};
template <>
struct Vec<float, 4> {
    static __device__ __forceinline__ void load(const float *p, float *v) {
        const float4 t = *reinterpret_cast<const float4 *>(p);
        v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
    }
    static __device__ __forceinline__ void store(float *p, const float *v) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
};
template <>
struct Vec<float, 2> {
    static __device__ __forceinline__ void load(const float *p, float *v) {
        const float2 t = *reinterpret_cast<const float2 *>(p);
        v[0] = t.x, v[1] = t.y;
    }
    static __device__ __forceinline__ void store(float *p, const float *v) {
        *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
    }
};
template <>
struct Vec<float, 8> {
    static __device__ __forceinline__ void load(const float *p, float *v) {
        Vec<float, 4>::load(p, v);
        Vec<float, 4>::load(p + 4, v + 4);
    }
    static __device__ __forceinline__ void store(float *p, const float *v) {
        Vec<float, 4>::store(p, v);
        Vec<float, 4>::store(p + 4, v + 4);
    }
};
template <>
struct Vec<bf16, 1> {
    static __device__ __forceinline__ void load(const bf16 *p, float *v) {
        v[0] = __bfloat162float(*p);
    }
    static __device__ __forceinline__ void store(bf16 *p, const float *v) {
        *p = __float2bfloat16_rn(v[0]);
    }
};
template <>
struct Vec<bf16, 2> {
    static __device__ __forceinline__ void load(const bf16 *p, float *v) {
        const float2 t = unpack_bf16(*reinterpret_cast<const uint32_t *>(p));
        v[0] = t.x, v[1] = t.y;
    }
    static __device__ __forceinline__ void store(bf16 *p, const float *v) {
        *reinterpret_cast<uint32_t *>(p) = pack_bf16(v[0], v[1]);
    }
};
template <>
struct Vec<bf16, 4> {
    static __device__ __forceinline__ void load(const bf16 *p, float *v) {
        const uint2 t = *reinterpret_cast<const uint2 *>(p);
        const float2 a = unpack_bf16(t.x), b = unpack_bf16(t.y);
        v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    }
    static __device__ __forceinline__ void store(bf16 *p, const float *v) {
        *reinterpret_cast<uint2 *>(p) =
            make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    }
};
template <>
struct Vec<bf16, 8> {
    static __device__ __forceinline__ void load(const bf16 *p, float *v) {
        const uint4 t = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 a = unpack_bf16(w[i]);
            v[2 * i] = a.x, v[2 * i + 1] = a.y;
        }
    }
    static __device__ __forceinline__ void store(bf16 *p, const float *v) {
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                       pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    }
};

// V elements as they are in memory.
template <int BYTES>
struct Raw;
template <>
struct Raw<16> {
    using type = uint4;
};
template <>
struct Raw<8> {
    using type = uint2;
};
template <>
struct Raw<4> {
    using type = uint32_t;
};
template <>
struct Raw<2> {
    using type = uint16_t;
};
template <class T, int V>
using RawV = typename Raw<V * int(sizeof(T))>::type;

template <class T, int V>
__device__ __forceinline__ void widen(const RawV<T, V> &r, float *v) {
    Vec<T, V>::load(reinterpret_cast<const T *>(&r), v);
}

// What rounding v to T leaves: v is T(v) + rest<T>(v).
template <class T>
__device__ __forceinline__ float rest(float v);
template <>
__device__ __forceinline__ float rest<float>(float) {
    return 0.0f;
}
template <>
__device__ __forceinline__ float rest<bf16>(float v) {
    return v - __bfloat162float(__float2bfloat16_rn(v));
}

// Unsigned division by a divisor fixed per launch: n / d for n < 2^31 as one
// high product and a shift.  m = floor(2^32 (2^s - d) / d) + 1 with
// 2^(s-1) < d <= 2^s (the round-up method of Granlund and Montgomery).
struct FastDiv {
    uint32_t d = 1, m = 1, s = 0;
    FastDiv() = default;
    explicit FastDiv(uint32_t div) : d(div) {
        while ((uint64_t(1) << s) < d) ++s;
        m = uint32_t(((uint64_t(1) << 32) * ((uint64_t(1) << s) - d)) / d + 1);
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const {
        return (__umulhi(n, m) + n) >> s;
    }
};

}  // namespace pcn
