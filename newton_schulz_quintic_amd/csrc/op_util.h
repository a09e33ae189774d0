// Helpers of the training-step operators (heads.hip, experts.hip, distill.hip):
// 16-byte vectors of bf16 or fp32 elements at any element alignment, fp32
// arithmetic on them, wave reductions, and the argument checks they share.
#pragma once

#include "hip_util.h"

namespace nsq {

// One vector: 16 bytes, 8 bf16 or 4 fp32 elements. Addresses need only element
// alignment: the GPU's unaligned access mode serves such a vector as one load
// or store, so tensors with odd widths or offsets take the same path.
template <typename T> struct Vec16;
template <> struct Vec16<__bf16> {
    static constexpr int N = 8;
    typedef uint16_t raw __attribute__((ext_vector_type(8)));
    typedef raw __attribute__((aligned(2))) raw_u;
};
template <> struct Vec16<float> {
    static constexpr int N = 4;
    typedef float raw __attribute__((ext_vector_type(4)));
    typedef raw __attribute__((aligned(4))) raw_u;
};

// NT: with the non-temporal hint, for data past what the caches can keep.
template <typename T, bool NT = false>
__device__ inline typename Vec16<T>::raw load_vec(const T *p) {
    const auto *q = reinterpret_cast<const typename Vec16<T>::raw_u *>(p);
    if constexpr (NT) return __builtin_nontemporal_load(q);
    else return *q;
}
template <typename T, bool NT = false>
__device__ inline void store_vec(T *p, typename Vec16<T>::raw v) {
    auto *q = reinterpret_cast<typename Vec16<T>::raw_u *>(p);
    if constexpr (NT) __builtin_nontemporal_store(v, q);
    else *q = v;
}

template <typename T> __device__ inline float elem(typename Vec16<T>::raw v, int i);
template <> __device__ inline float elem<__bf16>(Vec16<__bf16>::raw v, int i) {
    return __builtin_bit_cast(float, (uint32_t)v[i] << 16);
}
template <> __device__ inline float elem<float>(Vec16<float>::raw v, int i) { return v[i]; }

// fp32 to the stored type, rounded to nearest even (fp32: unchanged).
template <typename T> __device__ inline void set_elem(typename Vec16<T>::raw &v, int i, float x);
template <> __device__ inline void set_elem<__bf16>(Vec16<__bf16>::raw &v, int i, float x) {
    v[i] = __builtin_bit_cast(uint16_t, (__bf16)x);
}
template <> __device__ inline void set_elem<float>(Vec16<float>::raw &v, int i, float x) { v[i] = x; }

__device__ inline float wave_sum(float v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
    return v;
}

// The last-level cache (MALL).
constexpr int64_t kMallBytes = 256ll << 20;

// Host side -----------------------------------------------------------------

inline hipStream_t as_stream(void *s) { return reinterpret_cast<hipStream_t>(s); }

// Bytes of one element, or 0 for an unsupported type.
inline int dtype_bytes(int32_t dtype) { return dtype == NS_BF16 ? 2 : dtype == NS_F32 ? 4 : 0; }

inline bool misaligned(const void *p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }

// Whether count x size (both >= 0) exceeds 2^62, so that sums of two such
// extents still fit in 63 bits.
inline bool too_far(int64_t count, int64_t size) {
    int64_t r;
    return __builtin_mul_overflow(count, size, &r) || r > (int64_t(1) << 62);
}

}  // namespace nsq
