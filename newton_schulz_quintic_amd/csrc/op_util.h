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

// Memory that no running kernel writes: loads from uniform addresses go through the scalar cache.
#define NSQ_CONST __attribute__((address_space(4)))

// Butterfly over a wave's lanes: after steps 0 .. n-1 every lane of a group of
// 2^n holds the group's result. partner() is the value of a lane of the
// neighbouring group: within rows of 16 lanes a VALU operand modifier (a shuffle
// through LDS takes some 60 cycles), across them a shuffle.
template <int STEP>
__device__ inline float partner(float v) {
    if constexpr (STEP >= 4) return __shfl_xor(v, 1 << STEP);
    constexpr int ctrl = STEP == 0 ? 0xB1 : STEP == 1 ? 0x4E : STEP == 2 ? 0x141 : 0x140;   // quad_perm, mirrors
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), ctrl, 0xf, 0xf, true));
}
template <int STEP, int STEPS, typename Op>
__device__ inline float lanes_join(float v, const Op &op) {
    if constexpr (STEP < STEPS) return lanes_join<STEP + 1, STEPS>(op(v, partner<STEP>(v)), op);
    return v;
}
// The same of a double, in halves.
template <int STEP>
__device__ inline double partner(double v) {
    typedef float halves __attribute__((ext_vector_type(2)));
    halves h = __builtin_bit_cast(halves, v);
    return __builtin_bit_cast(double, halves{partner<STEP>(h.x), partner<STEP>(h.y)});
}
template <int STEP = 0>
__device__ inline double wave_sum(double v) {
    if constexpr (STEP < 6) return wave_sum<STEP + 1>(v + partner<STEP>(v));
    return v;
}
__device__ inline float wave_sum(float v) {
    return lanes_join<0, 6>(v, [](float a, float b) { return a + b; });
}
__device__ inline float wave_max(float v) {
    return lanes_join<0, 6>(v, [](float a, float b) { return fmaxf(a, b); });
}
// Sum over groups of 2^lg lanes.
__device__ inline float group_sum(float v, int lg) {
    const auto add = [](float a, float b) { return a + b; };
    if (lg > 0) v = lanes_join<0, 1>(v, add);
    if (lg > 1) v = lanes_join<1, 2>(v, add);
    if (lg > 2) v = lanes_join<2, 3>(v, add);
    if (lg > 3) v = lanes_join<3, 4>(v, add);
    if (lg > 4) v = lanes_join<4, 5>(v, add);
    if (lg > 5) v = lanes_join<5, 6>(v, add);
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
