// N consecutive elements of a tensor as one load or store: 16 bytes (8 bf16 or 4
// fp32), 8 bytes (4 bf16, next to 4 fp32 of another tensor) or one element.
// Addresses need element alignment only, as for Vec16.
#pragma once

#include <type_traits>

#include "op_util.h"

namespace nsq {

template <typename T, int N> struct Elems {
    typedef typename std::conditional<sizeof(T) == 2, uint16_t, float>::type E;
    typedef E raw __attribute__((ext_vector_type(N)));
    typedef raw __attribute__((aligned(sizeof(T)))) raw_u;
    // NT: with the non-temporal hint, for data past what the caches can keep.
    template <bool NT = false> static __device__ inline raw load(const T *p) {
        if constexpr (N == 1) return raw{*reinterpret_cast<const E *>(p)};
        else if constexpr (NT) return __builtin_nontemporal_load(reinterpret_cast<const raw_u *>(p));
        else return *reinterpret_cast<const raw_u *>(p);
    }
    static __device__ inline float at(raw r, int i) {
        if constexpr (sizeof(T) == 2) return __builtin_bit_cast(float, (uint32_t)r[i] << 16);
        else return r[i];
    }
    static __device__ inline void widen(raw r, float (&v)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = at(r, i);
    }
    template <bool NT = false> static __device__ inline void store(T *p, const float (&v)[N]) {
        raw r;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (sizeof(T) == 2) r[i] = __builtin_bit_cast(uint16_t, (__bf16)v[i]);
            else r[i] = v[i];
        }
        if constexpr (N == 1) *reinterpret_cast<E *>(p) = r[0];
        else if constexpr (NT) __builtin_nontemporal_store(r, reinterpret_cast<raw_u *>(p));
        else *reinterpret_cast<raw_u *>(p) = r;
    }
};

}  // namespace nsq
