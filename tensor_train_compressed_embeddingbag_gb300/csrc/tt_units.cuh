// tt_units.cuh -- rows of the three types read and written a unit at a time: 16 bytes, or fewer where
// rows do not begin on 16-byte boundaries, down to one element.
#pragma once

#include <type_traits>

#include "tt_head.cuh"

namespace ttemb {

// The raw unit of VEC elements: 16, 8 or 4 bytes, or one element.
template <int BYTES>
struct RawBytes;
template <>
struct RawBytes<16> {
    using type = uint4;
};
template <>
struct RawBytes<8> {
    using type = uint2;
};
template <>
struct RawBytes<4> {
    using type = uint32_t;
};
template <class T, int VEC>
struct RawOf {
    using type = typename RawBytes<VEC * (int)sizeof(T)>::type;
};
template <class T>
struct RawOf<T, 1> {
    using type = T;
};
template <class T, int VEC>
using Raw = typename RawOf<T, VEC>::type;

template <class T, int VEC>
__device__ __forceinline__ Raw<T, VEC> raw_zero() {
    if constexpr (VEC == 1) {
        return T(0.f);
    } else {
        Raw<T, VEC> r;
        uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
        for (int i = 0; i < VEC * (int)sizeof(T) / 4; ++i) w[i] = 0;
        return r;
    }
}
template <class T, int VEC>
__device__ __forceinline__ void unpack(const Raw<T, VEC>& r, float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        v[0] = to_f32(r);
    } else {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
        for (int i = 0; i < VEC * (int)sizeof(T) / 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                v[i] = __uint_as_float(w[i]);
            } else if constexpr (std::is_same<T, __half>::value) {
                const float2 f = unpack_f16(w[i]);
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            } else {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
    }
}
template <class T>
__device__ __forceinline__ T from_f32(float x) {
    if constexpr (sizeof(T) == 4)
        return x;
    else if constexpr (std::is_same<T, __half>::value)
        return __float2half_rn(x);
    else
        return __float2bfloat16_rn(x);
}
template <class T, int VEC>
__device__ __forceinline__ Raw<T, VEC> pack(const float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        return from_f32<T>(v[0]);
    } else {
        Raw<T, VEC> r;
        uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
        for (int i = 0; i < VEC * (int)sizeof(T) / 4; ++i) {
            if constexpr (sizeof(T) == 4)
                w[i] = __float_as_uint(v[i]);
            else
                w[i] = pack16(v[2 * i], v[2 * i + 1], !std::is_same<T, __half>::value);
        }
        return r;
    }
}
template <class T, int VEC>
__device__ __forceinline__ Raw<T, VEC>* unit_at(T* p, int64_t row, int64_t stride, int u) {
    return reinterpret_cast<Raw<T, VEC>*>(p + row * stride) + u;
}
template <class T, int VEC>
__device__ __forceinline__ const Raw<T, VEC>* unit_at(const T* p, int64_t row, int64_t stride, int u) {
    return reinterpret_cast<const Raw<T, VEC>*>(p + row * stride) + u;
}

inline bool aligned(const void* p, int to) { return (uintptr_t)p % to == 0; }

// The smallest power of two that is at least x, at most `most`.
inline int pow2_at_least(int64_t x, int most) {
    int p = 1;
    while (p < x && p < most) p *= 2;
    return p;
}

// A kernel that begins before the one ahead of it in the stream has ended, and waits for it in pdl_wait.  What that one
// writes it reads by ordinary loads: __ldg promises data that nobody writes while the kernel is there.  Some block of it has to
// wait whatever the data are: the launch behind waits for this one only, so one that ended without waiting would let it run
// beside the launch ahead.
// Not for a call's first: the one ahead of that is another call's, whose outputs may be its inputs.
template <class... Params, class... Args>
bool launch_ahead(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess) return true;
    cudaGetLastError();  // this call's failure, not the next one's
    return false;
}

}  // namespace ttemb
