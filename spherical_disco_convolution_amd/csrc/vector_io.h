// V consecutive elements in and out of registers as float32, at any element
// alignment (gfx950 global memory takes wide accesses at any).
#pragma once

#include "kernels_common.h"

namespace disco {

template <typename T, int V>
__device__ __forceinline__ void load_v(const T* p, float* f) {
    struct __attribute__((packed, aligned(sizeof(T)))) U { T e[V]; };
    const U u = *reinterpret_cast<const U*>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = load_f(u.e, i);
}

// bfloat16: the conversion instruction rounds to nearest even, two at a time
template <typename T, int V>
__device__ __forceinline__ void store_v(T* p, const float* f) {
    if constexpr (sizeof(T) == 2) {
        struct __attribute__((packed, aligned(2))) U { __bf16 e[V]; };
        U u;
#pragma unroll
        for (int i = 0; i < V; ++i) u.e[i] = (__bf16)f[i];
        *reinterpret_cast<U*>(p) = u;
    } else {
        struct __attribute__((packed, aligned(4))) U { T e[V]; };
        U u;
#pragma unroll
        for (int i = 0; i < V; ++i) u.e[i] = f[i];
        *reinterpret_cast<U*>(p) = u;
    }
}

}  // namespace disco
