// Loss of a student's logits against a teacher's top logits, and its gradient.
//
// A row has V student logits z and K pairs (token, teacher logit t); pairs
// whose token is outside [0, V) are absent. At temperature tau:
//   q = softmax(z / tau),  p_k = softmax over the row's pairs of t / tau,
//   loss = sum_k p_k (log p_k - log q[token_k]),
//   dz_j = g / tau (P q_j - sum of p_k over the pairs of token j),
// where P, all classes' p together, is 1.
// With the teacher's logsumexp over its whole vocabulary (at tau), p_k =
// exp(t_k / tau - lse_T) and all other tokens form one more class with
// p_r = max(0, 1 - sum p_k) and q_r = the sum of their q:
//   loss += p_r (log p_r - log q_r),  their dz_j = g / tau (P q_r - p_r) q_j / q_r,
// q_j / q_r being the softmax over them alone, finite however small q_r is. P is
// 1 again where p_r > 0, and the pairs' sum where p_r is 0: more than 1 where a
// token is listed twice or lse_T is too small for the teacher's (rounded) logits,
// less where the pairs hold every token. Where the student gives all others no
// mass at all, a p_r that may be rounding of the teacher's side alone is 0.
// Terms with p = 0 count as 0. A row without pairs (or, without lse_T, with
// every teacher logit -inf) has loss and gradient 0 and its logits are not used.
//
// q_r comes from a logsumexp of its own over the other tokens, found while the
// row is read (a bit per token in LDS marks the pairs' tokens): 1 - sum of the
// pairs' q would lose all its digits where q_r is small.
//
// Bound by memory: loss and gradient in one call read the row once and write
// its gradient once, the row staying in registers in between. 4096 x 131072 bf16
// with 64 pairs: 454-459 us, 4.7 TB/s, where a large copy here reaches 5.1: the
// exponentials (two a value) overlap with the memory only as far as the CUs'
// phases differ. 1025 x 50021 fp32, loss and then gradient in two calls: 119 us.
// 4 rows are bound by two launches and their latency, 9.0 us.

#include <algorithm>
#include <type_traits>

#include "op_util.h"

namespace nsq {
namespace {

constexpr int kMaxTop = 1024;
constexpr int kMaxVocab = 1 << 24;
constexpr int kMaxRows = 1 << 24;
constexpr int kMaxChunks = 64;            // parts of a row that is split over workgroups
constexpr int kScanPairs = 128;           // up to so many pairs each one looks for its token in all others
constexpr int kBitVocab = 1 << 18;        // tokens one workgroup marks in LDS (32 KiB)
constexpr int kSplitThreads = 256;
constexpr int kHeldVecs = 16;             // vectors of a row that a thread holds
constexpr int kKeptVecs = 8;              // vectors a thread keeps of a row too long to hold
static_assert(kKeptVecs <= kHeldVecs);
constexpr int kAhead = 4;                 // vectors a thread of a split row loads ahead of everything else
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kNonTemporal = 2;           // a buffer store's cache policy

struct DistillArgs {
    const void *logits;
    const void *ids;
    const void *teacher;
    const float *teacher_lse;
    const float *grad_loss;
    float *loss, *lse, *rest_lse;
    void *dlogits;
    int64_t ld, dld;
    float2 *partial;        // split rows: [rows][chunks] largest value and sum of each part
    float *top_z;           // split rows: [rows][top_k] student logits of the pairs
    int32_t rows, vocab, top_k;
    int32_t id_bytes, teacher_f32;
    int32_t chunks, chunk;  // parts of a row, tokens of one
    float inv_tau;
    int32_t large;          // gradient alone: which rows, by their logsumexp (too_large)
    double inv_tau64;
};

// Rows with a large logsumexp: with the others, left out, by themselves.
enum { kLargeToo = 0, kLargeNone = 1, kLargeOnly = 2 };

// ---------------------------------------------------------------------------
// sums of exponentials
// ---------------------------------------------------------------------------

// s = the sum of exp((x - m) / tau) over some x, m the largest of them.
struct Lse {
    float m, s;
};
constexpr float kNegInf = -__builtin_inff();

// exp((x - m) / tau) with c = log2(e) / tau; 0 where both are -inf.
__device__ inline float shifted(float x, float m, float c) {
    return __builtin_amdgcn_exp2f((x - (m == kNegInf ? 0.f : m)) * c);
}
__device__ inline Lse join(Lse a, Lse b, float c) {
    const float m = fmaxf(a.m, b.m);
    return {m, a.s * shifted(a.m, m, c) + b.s * shifted(b.m, m, c)};
}
// The same sum relative to an m that lies log2(s) / c, rounded, further: s is then
// near 1. (Relative to an m far above the largest x the exponentials fall below
// the normal numbers where q does not; far below it 1 / s times a small factor
// does, and log s loses digits that m takes up again.)
__device__ inline Lse near(Lse l, float c) {
    const float m = l.m + __builtin_amdgcn_logf(l.s) / c, d = m - l.m, e = d * c;
    return {m, l.s * __builtin_amdgcn_exp2f(-e) * __builtin_amdgcn_exp2f(-fmaf(d, c, -e))};
}
template <int STEP = 0>
__device__ inline Lse wave_join(Lse v, float c) {
    if constexpr (STEP < 6) return wave_join<STEP + 1>(join(v, {partner<STEP>(v.m), partner<STEP>(v.s)}, c), c);
    return v;
}

// q of a logit z is exp((z - m) / tau) scale.
struct Norm {
    float m, scale;
};
__device__ inline Norm norm_of(Lse l) { return {l.m == kNegInf ? 0.f : l.m, 1.f / l.s}; }
// From a logsumexp rounded to fp32: m is lse tau rounded, and the scale takes
// up the rest of it, so q is off by no more than lse's own rounding.
__device__ inline Norm norm_of_lse(float lse, float inv_tau) {
    const float m = lse / inv_tau, rest = fmaf(m, inv_tau, -lse);
    return {m, expf(rest)};
}
// Whether q from that logsumexp is too far off: by 2^-24 of it, 1.2e-4 at the bound,
// what a quotient z / tau of the size is off by itself.
__device__ inline bool too_large(float lse) { return fabsf(lse) > 1024.f; }
__device__ inline float q_of(float z, const Norm &n, float c) { return __builtin_amdgcn_exp2f((z - n.m) * c) * n.scale; }

// exp(x) in 64 bits, off by 2^-44 of itself: x = n ln 2 + 256 r with |r| < 2^-9.4, the
// series to r^4 (r^5 / 120 is below 2^-53), then eight squarings, each of which
// doubles the relative error of the 2^-53 before it. Few constants and few
// registers: the usual polynomial's made the kernels that hold a row spill.
__device__ inline double exp64(double x) {
    x = x < -800. ? -800. : x > 800. ? 800. : x;   // 0 and infinity; NaN stays
    const float n = rintf((float)x * kLog2e);
    const double r = fma(-(double)n, 0.69314718055994530942, x) * 0x1p-8;
    double e = fma(r, fma(r, fma(r, fma(r, 1. / 24, 1. / 6), 0.5), 1.), 1.);
#pragma unroll
    for (int i = 0; i < 8; ++i) e *= e;
    return ldexp(e, (int)n);
}

// ---------------------------------------------------------------------------
// a row's pairs
// ---------------------------------------------------------------------------

template <int TOP>             // room for so many pairs
struct PairLds {
    int32_t id[TOP + 4];       // token, -1 if absent
    float p[TOP + 4];
    float t[TOP];              // teacher logit, then log p
    float z[TOP];              // student logit
    float p_token[TOP];        // p summed over the token's pairs
    int32_t owner[TOP];        // the token, in the lowest of its pairs; -1 in the others
    Lse wave[16];
    float wave_sum[16];
    double wave_p[16];
    // many pairs: marks of the tokens' hashes, seen and seen again, and the pairs whose hash was seen again
    static constexpr int kMarks = TOP > kScanPairs ? TOP : 1;
    uint32_t once[kMarks], again[kMarks];
    int32_t listed[kMarks], listed_count;
};

struct Pairs {
    bool some;      // the row has a loss
    float t_max, t_sub;   // without a rest: the largest teacher logit, and log of the sum relative to it
    float p_rest;
    float mass;     // P
};

// One pair as it lies in memory (so that a load can be under way while other
// work is done), and its token (-1 if absent) and teacher logit.
struct RawPair {
    uint32_t id, id_high, t;
};
__device__ inline RawPair pair_at(const DistillArgs &A, int64_t row, int k) {
    const int64_t at = row * A.top_k + k;
    RawPair p = {0, 0, 0};
    if (A.id_bytes == 8) {
        const uint2 w = reinterpret_cast<const uint2 *>(A.ids)[at];
        p.id = w.x;
        p.id_high = w.y;
    } else {
        p.id = reinterpret_cast<const uint32_t *>(A.ids)[at];
    }
    if (A.teacher_f32) p.t = reinterpret_cast<const uint32_t *>(A.teacher)[at];
    else p.t = reinterpret_cast<const uint16_t *>(A.teacher)[at];
    return p;
}
__device__ inline int32_t token_of(const DistillArgs &A, const RawPair &p) {
    const bool here = p.id < (uint32_t)A.vocab && p.id_high == 0;   // negative ones have their top bit set
    return here ? (int32_t)p.id : -1;
}
__device__ inline float teacher_of(const DistillArgs &A, const RawPair &p) {
    return __builtin_bit_cast(float, A.teacher_f32 ? p.t : p.t << 16);
}

// Whether the row, whose tokens and teacher logits are in LDS, has a loss; its
// largest teacher logit. Every wave for itself.
template <bool REST, int TOP>
__device__ inline Pairs look_at_pairs(const DistillArgs &A, const PairLds<TOP> &L) {
    float mx = kNegInf;
    bool any = false, nan = false;
    for (int k = threadIdx.x & 63; k < A.top_k; k += 64)
        if (L.id[k] >= 0) {
            any = true;
            nan |= L.t[k] != L.t[k];
            mx = fmaxf(mx, L.t[k]);
        }
    Pairs r;
    r.t_max = wave_max(mx);
    if (__any(nan)) r.t_max = __builtin_nanf("");
    r.some = __any(any) && (REST || r.t_max != kNegInf);
    r.t_sub = r.p_rest = 0.f;
    r.mass = 1.f;
    return r;
}

// Clears what a row's pairs are added to.
template <bool REST, int TOP>
__device__ inline void clear_pairs(const DistillArgs &A, PairLds<TOP> &L, uint32_t *bits, int words) {
    if (threadIdx.x < 4) L.id[A.top_k + threadIdx.x] = -1, L.p[A.top_k + threadIdx.x] = 0.f;
    if constexpr (REST)
        for (int i = threadIdx.x; i < words; i += blockDim.x) bits[i] = 0;
    if constexpr (TOP > kScanPairs)
        if (A.top_k > kScanPairs) {
            for (int i = threadIdx.x; i < TOP; i += blockDim.x) L.once[i] = L.again[i] = 0;
            if (threadIdx.x == 0) L.listed_count = 0;
        }
}

// Where a token's mark is: 32 marks for each pair there is room for.
template <int TOP> __device__ inline int mark_of(int id) { return (uint32_t)id * 2654435769u >> 17 & (TOP * 32 - 1); }

// Brings the row's pairs into LDS; says whether the row has a loss. Ends with
// every thread past the barrier.
template <bool REST, int TOP>
__device__ inline Pairs read_pairs(const DistillArgs &A, int64_t row, PairLds<TOP> &L, uint32_t *bits, int words) {
    for (int k = threadIdx.x; k < A.top_k; k += blockDim.x) {
        const RawPair p = pair_at(A, row, k);
        L.id[k] = token_of(A, p);
        L.t[k] = teacher_of(A, p);
    }
    clear_pairs<REST>(A, L, bits, words);
    __syncthreads();
    return look_at_pairs<REST>(A, L);
}

template <bool REST>
__device__ inline float teacher_lse(const DistillArgs &A, int64_t row) {
    return REST ? A.teacher_lse[row] : 0.f;
}

// p of every pair, the tokens' lowest pairs, and with REST the tokens' bits
// among [e0, e1). Ends with every thread past a barrier. With REST p and its sum
// are found in 64 bits: p_r = 1 - sum is often 1e-3 to 1e-6, and all other
// tokens' gradients hang on it, while an fp32 sum is off by some 1e-7. Few pairs are compared
// all with all. Of many, those whose token's hash no other has are alone; a wave
// compares each of the rest with all (loss of 2048 x 32000 bf16 with 1024 pairs:
// 562 us all with all, 78 by hashes; 50257 tokens, 256 pairs: 74 and 67).
template <bool REST, int TOP>
__device__ inline void weigh_pairs(const DistillArgs &A, float lse, PairLds<TOP> &L, Pairs &r, uint32_t *bits, int e0,
                                   int e1) {
    const int lane = threadIdx.x & 63, threads = blockDim.x;
    const bool many = TOP > kScanPairs && A.top_k > kScanPairs;
    const auto settle = [&](int k, int id, bool lowest, float p) {
        L.owner[k] = lowest ? id : -1;
        L.p_token[k] = p;
        if constexpr (REST)
            if (lowest && id >= e0 && id < e1) atomicOr(&bits[(id - e0) >> 5], 1u << ((id - e0) & 31));
    };
    if constexpr (!REST) {
        float s = 0.f;
        for (int k = lane; k < A.top_k; k += 64)
            if (L.id[k] >= 0) s += __builtin_amdgcn_exp2f((L.t[k] - r.t_max) * (A.inv_tau * kLog2e));
        r.t_sub = logf(wave_sum(s));
    }
    __syncthreads();   // L.t has been read by every wave
    double own = 0.;
    for (int k = threadIdx.x; k < A.top_k; k += threads) {
        float log_p, p;
        if constexpr (REST) {
            const double exact = L.t[k] * A.inv_tau64 - lse, p64 = L.id[k] >= 0 ? exp64(exact) : 0.;
            own += p64;
            log_p = (float)exact, p = (float)p64;
        } else {
            log_p = (L.t[k] - r.t_max) * A.inv_tau - r.t_sub;
            p = L.id[k] >= 0 ? __builtin_amdgcn_exp2f(log_p * kLog2e) : 0.f;
        }
        L.t[k] = log_p;
        L.p[k] = p;
        if (many && L.id[k] >= 0) {
            const int at = mark_of<TOP>(L.id[k]);
            const uint32_t bit = 1u << (at & 31);
            if (atomicOr(&L.once[at >> 5], bit) & bit) atomicOr(&L.again[at >> 5], bit);
        }
    }
    if constexpr (REST) {
        own = wave_sum(own);
        if (lane == 0) L.wave_p[threadIdx.x >> 6] = own;
    }
    __syncthreads();
    if (many) {
        for (int k = threadIdx.x; k < A.top_k; k += threads) {
            const int id = L.id[k], at = mark_of<TOP>(id);
            if (id >= 0 && (L.again[at >> 5] >> (at & 31) & 1)) L.listed[atomicAdd(&L.listed_count, 1)] = k;
            else settle(k, id, id >= 0, L.p[k]);
        }
        __syncthreads();
        for (int i = threadIdx.x >> 6; i < L.listed_count; i += threads >> 6) {   // a wave each
            const int k = L.listed[i], id = L.id[k];
            float sum = 0.f;
            bool lower = false;
            for (int j = lane; j < A.top_k; j += 64)
                if (L.id[j] == id) {
                    sum += L.p[j];
                    lower |= j < k;
                }
            sum = wave_sum(sum);
            const bool lowest = !__any(lower);
            if (lane == 0) settle(k, id, lowest, sum);
        }
    } else {
        for (int k = threadIdx.x; k < A.top_k; k += threads) {
            const int id = L.id[k];
            bool lowest = id >= 0;
            float sum = 0.f;
#pragma unroll 1
            for (int j = 0; j < A.top_k; j += 4) {
                const int4 other = *reinterpret_cast<const int4 *>(&L.id[j]);
                const float4 p = *reinterpret_cast<const float4 *>(&L.p[j]);
                lowest = lowest && !(other.x == id && j < k) && !(other.y == id && j + 1 < k) &&
                         !(other.z == id && j + 2 < k) && !(other.w == id && j + 3 < k);
                sum += (other.x == id ? p.x : 0.f) + (other.y == id ? p.y : 0.f) + (other.z == id ? p.z : 0.f) +
                       (other.w == id ? p.w : 0.f);
            }
            settle(k, id, lowest, sum);
        }
    }
    __syncthreads();
    if constexpr (REST) {
        double sum = 0.;
        for (int w = 0; w < threads >> 6; ++w) sum += L.wave_p[w];
        int tokens = 0;
        for (int k = lane; k < A.top_k; k += 64) tokens += L.owner[k] >= 0;
        r.p_rest = (float)(1. - sum);
        // nothing outside the pairs: no class to hold what rounding leaves
        if (r.p_rest < 0.f || (int)wave_sum((float)tokens) == A.vocab) r.p_rest = 0.f;
        if (r.p_rest == 0.f) r.mass = (float)sum;
    }
}

// ---------------------------------------------------------------------------
// a part of a row
// ---------------------------------------------------------------------------

// Tokens [e0, e1): whole vectors dealt to the threads in turn, the few tokens
// behind them one each to the first threads.
template <typename T> struct Span {
    static constexpr int N = Vec16<T>::N;
    int e0, e1, vecs, tail;
    __device__ Span(int from, int to) : e0(from), e1(to), vecs((to - from) / N), tail((to - from) % N) {}
    // The thread that holds a token of the span.
    __device__ int thread_of(int token, int threads) const {
        const int j = token - e0;
        return j < vecs * N ? j / N % threads : j - vecs * N;
    }
};

__device__ inline uint32_t vec_bits(const uint32_t *bits, int v, int n) {
    return reinterpret_cast<const uint8_t *>(bits)[v * n >> 3] >> (v * n & 7) & ((1u << n) - 1);
}

// The thread's value behind the span's vectors.
template <typename T>
__device__ inline float tail_of(const T *z, const Span<T> &S) {
    return (int)threadIdx.x < S.tail ? (float)z[S.e0 + S.vecs * S.N + threadIdx.x] : 0.f;
}

// Adds a vector's values to a thread's running sum; with REST only those whose bit is clear.
template <typename T, bool REST>
__device__ inline void add_vec(Lse &a, typename Vec16<T>::raw v, uint32_t skip, float c) {
    constexpr int N = Vec16<T>::N;
    float x[N], mx = a.m;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = REST && (skip >> i & 1) ? kNegInf : elem<T>(v, i);
        mx = fmaxf(mx, x[i]);
    }
    float s = 0.f;
    const float m = mx == kNegInf ? 0.f : mx;
#pragma unroll
    for (int i = 0; i < N; ++i) s += __builtin_amdgcn_exp2f((x[i] - m) * c);
    a.s = a.s * __builtin_amdgcn_exp2f((a.m - m) * c) + s;
    a.m = mx;
}

// The thread's value of the span's tail, x, likewise.
template <typename T, bool REST>
__device__ inline void add_tail(Lse &a, float x, const Span<T> &S, const uint32_t *bits, float c) {
    if ((int)threadIdx.x >= S.tail) return;
    const int j = S.vecs * S.N + threadIdx.x;
    if (REST && (bits[j >> 5] >> (j & 31) & 1)) return;
    a = join(a, {x, x == x && x != __builtin_inff() && x != kNegInf ? 1.f : x == kNegInf ? 0.f : __builtin_nanf("")}, c);
}

// The sum over a span of a row in memory, joined over the workgroup.
template <typename T, bool REST, int B = 4>
__device__ inline Lse sum_span(const T *z, float zt, const Span<T> &S, const uint32_t *bits, float c) {
    const int threads = blockDim.x;
    Lse a = {kNegInf, 0.f};
    int v = threadIdx.x;
    for (; v + (B - 1) * threads < S.vecs; v += B * threads) {
        typename Vec16<T>::raw r[B];
#pragma unroll
        for (int i = 0; i < B; ++i) r[i] = load_vec<T>(z + S.e0 + (int64_t)(v + i * threads) * S.N);
#pragma unroll
        for (int i = 0; i < B; ++i) add_vec<T, REST>(a, r[i], REST ? vec_bits(bits, v + i * threads, S.N) : 0, c);
    }
    for (; v < S.vecs; v += threads)
        add_vec<T, REST>(a, load_vec<T>(z + S.e0 + (int64_t)v * S.N), REST ? vec_bits(bits, v, S.N) : 0, c);
    add_tail<T, REST>(a, zt, S, bits, c);
    return a;
}

// Joins the threads' sums; every thread gets the result. One barrier inside.
template <int TOP>
__device__ inline Lse block_join(Lse a, PairLds<TOP> &L, float c) {
    a = wave_join(a, c);
    if ((threadIdx.x & 63) == 0) L.wave[threadIdx.x >> 6] = a;
    __syncthreads();
    a = {kNegInf, 0.f};
    for (int w = 0; w < (int)(blockDim.x >> 6); ++w) a = join(a, L.wave[w], c);
    return a;
}

// The threads' sum, in every thread; the workgroup has THREADS of them. One barrier inside.
template <int THREADS, int TOP>
__device__ inline float block_sum(float v, PairLds<TOP> &L) {
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0) L.wave_sum[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
    if constexpr (THREADS >= 256) {
#pragma unroll
        for (int w = 0; w < THREADS / 64; w += 4) {
            const float4 q = *reinterpret_cast<const float4 *>(&L.wave_sum[w]);
            v += (q.x + q.y) + (q.z + q.w);
        }
    } else {
        for (int w = 0; w < THREADS / 64; ++w) v += L.wave_sum[w];
    }
    return v;
}

// The sum over the pairs' tokens (each once); every wave for itself.
template <int TOP>
__device__ inline Lse sum_tokens(const DistillArgs &A, const PairLds<TOP> &L, float c) {
    Lse a = {kNegInf, 0.f};
    for (int k = threadIdx.x & 63; k < A.top_k; k += 64)
        if (L.owner[k] >= 0) {
            const float x = L.z[k];
            a = join(a, {x, x == kNegInf ? 0.f : shifted(x, x, c)}, c);
        }
    return wave_join(a, c);
}

// g q of a vector's logits.
template <typename T>
__device__ inline typename Vec16<T>::raw grad_vec(typename Vec16<T>::raw v, const Norm &n, float c, float g) {
    typename Vec16<T>::raw o;
    const float factor = g * n.scale;
#pragma unroll
    for (int i = 0; i < Vec16<T>::N; ++i)
        set_elem<T>(o, i, factor * __builtin_amdgcn_exp2f((elem<T>(v, i) - n.m) * c));
    return o;
}

// The same two with exp((z - m) / tau) = 2^(z c + hi) 2^-lo, where m is the
// pairs' largest logit: one fma a value, and no maximum to find. They serve
// unless some logit lies so far above m that the sum overflows, or (REST) all
// lie so far below that it is lost, or one is NaN or infinite, or (bf16) m lies
// where the gradient's exponent is too coarse; such a row is summed again relative
// to its own largest.
template <typename T, bool REST>
__device__ inline float fast_sum(typename Vec16<T>::raw v, uint32_t skip, float c, float hi) {
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < Vec16<T>::N; ++i) s[i & 1] += __builtin_amdgcn_exp2f(fmaf(elem<T>(v, i), c, hi));
    if (REST && skip) {   // few vectors: without the pairs' tokens, in the same order
        s[0] = s[1] = 0.f;
#pragma unroll
        for (int i = 0; i < Vec16<T>::N; ++i)
            s[i & 1] += skip >> i & 1 ? 0.f : __builtin_amdgcn_exp2f(fmaf(elem<T>(v, i), c, hi));
    }
    return s[0] + s[1];
}
template <typename T, bool REST>
__device__ inline float fast_tail(float zt, const Span<T> &S, const uint32_t *bits, float c, float hi) {
    if ((int)threadIdx.x >= S.tail || (REST && vec_bits(bits, S.vecs * S.N + threadIdx.x, 1))) return 0.f;
    return __builtin_amdgcn_exp2f(fmaf(zt, c, hi));
}
// The exponent's offset for sums relative to the pairs' largest logit m, and
// whether such a sum can be used.
struct FastBase {
    float m, hi, lo;
};
template <int TOP>
__device__ inline FastBase fast_base(const DistillArgs &A, const PairLds<TOP> &L, float c) {
    float m = kNegInf;
    for (int k = threadIdx.x & 63; k < A.top_k; k += 64)
        if (L.id[k] >= 0) m = fmaxf(m, L.z[k]);
    m = wave_max(m);
    const float hi = -m * c;
    return {m, hi, fmaf(m, c, hi)};
}
__device__ inline bool fast_holds(const Lse &s) { return s.s > 1e-10f && s.s < 1e30f; }

// factor 2^(z c + hi). For bf16 results log2 |factor| goes into the exponent and
// the sign is set afterwards. That sum is rounded: with both parts below 1024 by
// 2^-14, 4e-5 of the result or 1 % of a bf16 half step.
struct FastFactor {
    float hi, factor;
    uint32_t sign;
};
// Whether hi stays below that, given the offset of the sum that m moves by.
template <typename T> __device__ inline bool offset_holds(float hi) { return sizeof(T) == 4 || fabsf(hi) < 900.f; }
// g q of any logit, from a norm near its row's logsumexp.
template <typename T> __device__ inline FastFactor fast_factor(const Norm &n, float g, float c) {
    const bool fold = sizeof(T) == 2;
    const float hi = -n.m * c, factor = g * n.scale * __builtin_amdgcn_exp2f(-fmaf(n.m, c, hi));
    return {fold ? hi + __builtin_amdgcn_logf(fabsf(factor)) : hi, factor, fold && factor < 0.f ? 0x80008000u : 0u};
}
template <typename T>
__device__ inline typename Vec16<T>::raw fast_grad(typename Vec16<T>::raw v, float c, const FastFactor &f) {
    typename Vec16<T>::raw o;
#pragma unroll
    for (int i = 0; i < Vec16<T>::N; ++i) {
        const float e = __builtin_amdgcn_exp2f(fmaf(elem<T>(v, i), c, f.hi));
        set_elem<T>(o, i, sizeof(T) == 2 ? e : e * f.factor);
    }
    if constexpr (sizeof(T) == 2) {
        typedef uint32_t dwords __attribute__((ext_vector_type(4)));
        o = __builtin_bit_cast(typename Vec16<T>::raw, __builtin_bit_cast(dwords, o) ^ f.sign);
    }
    return o;
}

// The thread's part of a span's sum from the given vector on, read from memory, likewise.
template <typename T, bool REST, int B>
__device__ inline float fast_span(const T *z, float zt, const Span<T> &S, const uint32_t *bits, float c, float hi, int from) {
    const int threads = blockDim.x;
    float sum = 0.f;
    int v = from + threadIdx.x;
    for (; v + (B - 1) * threads < S.vecs; v += B * threads) {
        typename Vec16<T>::raw r[B];
#pragma unroll
        for (int i = 0; i < B; ++i) r[i] = load_vec<T>(z + S.e0 + (int64_t)(v + i * threads) * S.N);
#pragma unroll
        for (int i = 0; i < B; ++i)
            sum += fast_sum<T, REST>(r[i], REST ? vec_bits(bits, v + i * threads, S.N) : 0, c, hi);
    }
    for (; v < S.vecs; v += threads)
        sum += fast_sum<T, REST>(load_vec<T>(z + S.e0 + (int64_t)v * S.N), REST ? vec_bits(bits, v, S.N) : 0, c, hi);
    return sum + fast_tail<T, REST>(zt, S, bits, c, hi);
}

// The gradient of a span's vectors from the given one on, read from memory.
template <typename T, bool NT>
__device__ inline void grad_span(const T *z, T *dz, const Span<T> &S, const Norm &n, float c, float g, int from = 0) {
    constexpr int B = 4;
    const int threads = blockDim.x;
    int v = from + threadIdx.x;
    for (; v + (B - 1) * threads < S.vecs; v += B * threads) {
        typename Vec16<T>::raw w[B];
#pragma unroll
        for (int i = 0; i < B; ++i) w[i] = load_vec<T>(z + S.e0 + (int64_t)(v + i * threads) * S.N);
#pragma unroll
        for (int i = 0; i < B; ++i)
            store_vec<T, NT>(dz + S.e0 + (int64_t)(v + i * threads) * S.N, grad_vec<T>(w[i], n, c, g));
    }
    for (; v < S.vecs; v += threads)
        store_vec<T, NT>(dz + S.e0 + (int64_t)v * S.N, grad_vec<T>(load_vec<T>(z + S.e0 + (int64_t)v * S.N), n, c, g));
}

// The tail's gradient, then that of the pairs' tokens, each written over the
// other tokens' formula by the thread that wrote it. n: of the pairs' tokens, P q.
template <typename T, typename Put, int TOP>
__device__ inline void finish_span(const DistillArgs &A, const PairLds<TOP> &L, const Put &put, const Span<T> &S, float zt,
                                   const Norm &n, const Norm &others, float c, float g, float g_others) {
    if ((int)threadIdx.x < S.tail) put(S.e0 + S.vecs * S.N + threadIdx.x, (T)(g_others * q_of(zt, others, c)));
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int k0 = 0; k0 < A.top_k; k0 += 64) {
        const int k = k0 + lane;
        const int id = k < A.top_k ? L.owner[k] : -1;
        int thread = -1;
        float val = 0.f;
        if (id >= S.e0 && id < S.e1) {
            thread = S.thread_of(id, blockDim.x);
            val = g * (q_of(L.z[k], n, c) - L.p_token[k]);
        }
        uint64_t mine = __ballot(thread >= 0 && thread >> 6 == wave);
        while (mine) {
            const int b = __builtin_ctzll(mine);
            mine &= mine - 1;
            const int to = __shfl(thread, b) & 63, token = __shfl(id, b);
            const float x = __shfl(val, b);
            if (lane == to) put(token, (T)x);
        }
    }
}

// The row's loss and logsumexps, by the first wave.
template <bool REST, int TOP>
__device__ inline void write_loss(const DistillArgs &A, const PairLds<TOP> &L, const Pairs &r, int64_t row, const Norm &n,
                                  Lse all, Lse rest) {
    if (threadIdx.x >= 64) return;
    const float log_all = logf(all.s);
    float sum = 0.f;
    for (int k = threadIdx.x; k < A.top_k; k += 64) {
        const float p = L.p[k];
        if (p != 0.f) sum += p * (L.t[k] - ((L.z[k] - n.m) * A.inv_tau - log_all));
    }
    sum = wave_sum(sum);
    if (threadIdx.x) return;
    if constexpr (REST) {
        const float log_rest = logf(rest.s);
        if (r.p_rest != 0.f) {
            const float log_q = (rest.m - n.m) * A.inv_tau + log_rest - log_all;
            sum += r.p_rest * (logf(r.p_rest) - log_q);
        }
        A.rest_lse[row] = rest.m * A.inv_tau + log_rest;
    }
    A.loss[row] = sum;
    A.lse[row] = all.m * A.inv_tau + log_all;
}

template <bool REST>
__device__ inline void write_no_loss(const DistillArgs &A, int64_t row) {
    A.loss[row] = A.lse[row] = 0.f;
    if constexpr (REST) A.rest_lse[row] = 0.f;
}

// A row without a loss: zeros. `first`: also its loss and logsumexps.
template <typename T, bool REST>
__device__ inline void write_empty(const DistillArgs &A, int64_t row, const Span<T> &S, bool first) {
    if (A.dlogits) {
        T *dz = reinterpret_cast<T *>(A.dlogits) + row * A.dld;
        for (int v = threadIdx.x; v < S.vecs; v += blockDim.x) {
            const typename Vec16<T>::raw o = {};
            store_vec<T>(dz + S.e0 + (int64_t)v * S.N, o);
        }
        if ((int)threadIdx.x < S.tail) dz[S.e0 + S.vecs * S.N + threadIdx.x] = (T)0.f;
    }
    if (first && threadIdx.x == 0) write_no_loss<REST>(A, row);
}

// ---------------------------------------------------------------------------
// kernels
// ---------------------------------------------------------------------------

// What the loss and the gradient of a row take from its sums.
struct RowSums {
    Lse all, rest;
    Norm n, others;    // P q of any token, and what the others' gradient is g_others times
    float g, g_others;
};
// The others' factor, from their share of the student's mass.
template <bool REST>
__device__ inline float others_factor(const Pairs &r, float g, float q_rest) {
    return REST ? g * (r.mass * q_rest - r.p_rest) : g;
}
// For rows whose others have no mass in the student: a p_r no larger than what
// rounding can leave of 1 - sum p becomes 0, or the loss of a student masked to
// the pairs' tokens would be infinite for an lse_T over just these, half the
// time. Rounded are teacher logits (bf16: by half a step, counted whole for the
// exponential's sake) and lse_T, a logsumexp in fp32 (its parts by four half steps).
template <int TOP>
__device__ inline void drop_rounding(const DistillArgs &A, const PairLds<TOP> &L, Pairs &r, int64_t row) {
    if (!(r.p_rest > 0.f)) return;
    const float lse = A.teacher_lse[row];   // read again: seldom needed here
    float left = 0.f;
    for (int k = threadIdx.x & 63; k < A.top_k; k += 64)
        if (L.p[k] > 0.f) {
            const float size = fabsf(L.t[k] + lse);   // of t / tau
            left += L.p[k] * (size * (A.teacher_f32 ? 0.f : 0x1p-7f) + 0x1p-22f * (size + fabsf(lse) + 4.f));
        }
    if (r.p_rest > wave_sum(left)) return;
    r.mass = 1.f - r.p_rest;
    r.p_rest = 0.f;
}
template <bool REST, int TOP>
__device__ inline RowSums row_sums(const DistillArgs &A, const PairLds<TOP> &L, Pairs &r, int64_t row, float grad_loss,
                                   Lse rest, float c) {
    RowSums s;
    if (REST && rest.s == 0.f) drop_rounding(A, L, r, row);
    s.rest = rest;
    s.all = REST ? join(rest, sum_tokens(A, L, c), c) : rest;
    s.n = norm_of(s.all);
    if constexpr (REST) s.n.scale *= r.mass;
    s.others = norm_of(s.rest);
    if (REST && rest.s == 0.f && r.p_rest == 0.f) s.others.scale = 0.f;   // no others, or all masked: q is 0
    s.g = grad_loss * A.inv_tau;
    s.g_others = others_factor<REST>(r, s.g, rest.s / s.all.s * shifted(rest.m, s.all.m, c));
    return s;
}

// Loss and gradient, the row in registers in between: kHeldVecs vectors and at
// most one pair a thread, in the fewest threads that this takes (64 to 1024), so
// that a CU's registers hold as many rows at once as they can. A workgroup takes
// rows in turn and loads each vector of its next row as soon as it has written
// the one before. Loads return in order, so what the next row needs besides (its
// tokens' logits, and the pairs of the row after it, whose tokens those logits'
// addresses come from) is asked for ahead of its vectors: its pairs are then
// weighed while its vectors come in.
// Vectors go through buffer descriptors: lanes past the row's last whole vector
// read zeros (not used) and write nothing.
template <typename T, int THREADS, bool REST, int TOP>
__global__ __launch_bounds__(THREADS, 4) void distill_held_kernel(DistillArgs A) {
    extern __shared__ uint32_t bits[];
    __shared__ __attribute__((aligned(16))) PairLds<TOP> L;
    typedef uint32_t dwords __attribute__((ext_vector_type(4)));
    typedef typename Vec16<T>::raw raw;
    const Span<T> S(0, A.vocab);
    const float c = A.inv_tau * kLog2e;
    const int tid = threadIdx.x;
    const auto row_of = [&](const void *base, int64_t row, int64_t ld) {
        return reinterpret_cast<T *>(const_cast<void *>(base)) + row * ld;
    };
    const auto vecs_of = [&](const void *base, int64_t row, int64_t ld, bool there) {
        return __builtin_amdgcn_make_buffer_rsrc(row_of(base, there ? row : 0, ld), (short)0, there ? S.vecs * 16 : 0,
                                                 0x00020000);
    };
    const auto all_of = [&](const void *base, int64_t row, int64_t ld) {   // element by element, to the row's end
        return __builtin_amdgcn_make_buffer_rsrc(row_of(base, row, ld), (short)0, A.vocab * (int)sizeof(T), 0x00020000);
    };
    const auto get = [](__amdgpu_buffer_rsrc_t r, int j) {
        if constexpr (sizeof(T) == 2) return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b16(r, j * 2, 0, 0));
        else return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(r, j * 4, 0, 0));
    };
    // What a row needs besides its vectors; nothing of it is looked at before the row's turn.
    const auto pair_of = [&](int64_t row) { return tid < A.top_k && row < A.rows ? pair_at(A, row, tid) : RawPair{~0u, 0, 0}; };
    struct Beside {
        T pz, zt;             // logits of the thread's pair and of its place behind the vectors
        float g, teacher_lse;
    };
    const auto beside_of = [&](int64_t row, const RawPair &p) {
        Beside b = {(T)0.f, (T)0.f, 0.f, 0.f};
        if (row < A.rows) {
            const auto z = all_of(A.logits, row, A.ld);
            const int32_t id = token_of(A, p);
            if (id >= 0) b.pz = get(z, id);
            if (tid < S.tail) b.zt = get(z, S.vecs * S.N + tid);
            b.g = A.grad_loss[row];
            if constexpr (REST) b.teacher_lse = A.teacher_lse[row];
        }
        return b;
    };

    // The waits for what is under way count the loads and stores issued since, over every path to them. So that the
    // counts are exact there is no branch around a vector's load or store (past the row, or for no next row, their
    // descriptors end before them), and the first row's loads go out like the others': in order, each behind a store
    // (to a descriptor of length zero).
    // With one workgroup a CU and equal rows the CUs stay in step: all load, then all compute while memory rests.
    // Over many bf16 rows of a length that needs a CU's registers those of four neighbouring XCDs start a quarter of
    // a row apart, 1024 cycles for 1024 vectors (4096 x 131072: 472 us become 456, 4096 x 70000: 307 become 300; 1024
    // rows of 131072 132 become 138 if they do; f32 rows, with half the work a byte, 224 become 227).
    if (THREADS == 1024 && sizeof(T) == 2 && S.vecs > kHeldVecs * THREADS / 2 && A.rows >= 8 * (int)gridDim.x)
        for (int i = 0; i < (int)(blockIdx.x & 3) * S.vecs / 1024; ++i) __builtin_amdgcn_s_sleep(16);
    dwords held[kHeldVecs];
    int64_t row = blockIdx.x;
    RawPair p = pair_of(row), ahead = pair_of(row + gridDim.x);
    Beside now = beside_of(row, p);
    {
        const auto z = vecs_of(A.logits, row, A.ld, true), nowhere = vecs_of(A.logits, row, A.ld, false);
#pragma unroll
        for (int i = 0; i < kHeldVecs; ++i) {
            __builtin_amdgcn_raw_buffer_store_b128(dwords{0, 0, 0, 0}, nowhere, tid * 16 + i * THREADS * 16, 0, 0);
            held[i] = __builtin_amdgcn_raw_buffer_load_b128(z, tid * 16 + i * THREADS * 16, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    for (; row < A.rows; row += gridDim.x) {
        const int64_t next = row + gridDim.x;
        if (tid < A.top_k) {
            L.id[tid] = token_of(A, p);
            L.t[tid] = teacher_of(A, p);
            L.z[tid] = (float)now.pz;
        }
        clear_pairs<REST>(A, L, bits, (A.vocab + 31) >> 5);
        __syncthreads();
        Pairs r = look_at_pairs<REST>(A, L);
        weigh_pairs<REST>(A, now.teacher_lse, L, r, bits, 0, A.vocab);
        int at = tid;
        asm volatile("" : "+v"(at));   // what follows from it is found anew for each row, not held in 2 kHeldVecs registers
        const float zt = (float)now.zt;
        const FastBase f0 = fast_base(A, L, c);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kHeldVecs; ++i) {
            const int left = S.vecs - i * THREADS;
            if (left > 0 && (left >= THREADS || at < left)) {
                const uint32_t skip = REST ? vec_bits(bits, at + i * THREADS, S.N) : 0;
                sum += fast_sum<T, REST>(__builtin_bit_cast(raw, held[i]), skip, c, f0.hi);
            }
        }
        sum += fast_tail<T, REST>(zt, S, bits, c, f0.hi);
        Lse rest = {f0.m, block_sum<THREADS>(sum, L) * __builtin_amdgcn_exp2f(-f0.lo)};
        const bool fast = !r.some || (fast_holds(rest) && offset_holds<T>(f0.hi));
        rest = near(rest, c);
        if (!fast) {
            Lse a = {kNegInf, 0.f};
#pragma unroll
            for (int i = 0; i < kHeldVecs; ++i) {
                const int v = at + i * THREADS;
                if (v < S.vecs) add_vec<T, REST>(a, __builtin_bit_cast(raw, held[i]), REST ? vec_bits(bits, v, S.N) : 0, c);
            }
            add_tail<T, REST>(a, zt, S, bits, c);
            __syncthreads();
            rest = block_join(a, L, c);
        }
        const RowSums s = row_sums<REST>(A, L, r, row, now.g, rest, c);
        // The next row: first what lies besides its vectors, and the pairs of the row after it.
        p = ahead;
        now = beside_of(next, p);
        ahead = pair_of(next + gridDim.x);
        const auto dz = vecs_of(A.dlogits, row, A.dld, true), z = vecs_of(A.logits, next, A.ld, next < A.rows);
        const FastFactor f = fast_factor<T>(s.others, s.g_others, c);
        const auto turn = [&](auto value) {
#pragma unroll
            for (int i = 0; i < kHeldVecs; ++i) {
                raw o = {};
                if (r.some && S.vecs > i * THREADS) o = value(__builtin_bit_cast(raw, held[i]));
                // soffset stays 0: with an SGPR there the compiler takes it that the store has read its data at
                // once, but a VALU write to the last two dwords right behind it was seen to reach memory.
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(dwords, o), dz, at * 16 + i * THREADS * 16, 0, kNonTemporal);
                held[i] = __builtin_amdgcn_raw_buffer_load_b128(z, at * 16 + i * THREADS * 16, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        if (fast) turn([&](raw v) { return fast_grad<T>(v, c, f); });
        else turn([&](raw v) { return grad_vec<T>(v, s.others, c, s.g_others); });
        asm volatile("" ::: "memory");   // the pairs' tokens are written over what these stores left
        const auto out = all_of(A.dlogits, row, A.dld);
        const auto put = [&](int j, T x) {
            if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, x), out, j * 2, 0, 0);
            else __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, x), out, j * 4, 0, 0);
        };
        if (r.some) {
            finish_span<T>(A, L, put, S, zt, s.n, s.others, c, s.g, s.g_others);
            write_loss<REST>(A, L, r, row, s.n, s.all, s.rest);
        } else {
            if (tid < S.tail) put(S.vecs * S.N + tid, (T)0.f);
            if (tid == 0) write_no_loss<REST>(A, row);
        }
        __syncthreads();   // the next row's pairs go into the same LDS
    }
}

// Loss by itself, or (TRAIN) with the gradient of rows too long to hold. These
// are read a second time for the gradient, except for the first kKept vectors of
// each thread: one workgroup a CU, so that the 256 rows under way stay in the
// last-level cache in between (2048 x 151936 bf16: 361 us with many workgroups of
// 256 threads, 326 with 256 of 1024 threads, 279 with 8 vectors kept; 12 spill,
// 287; 2000 x 100000 f32 448, 360 and 315). Loss alone keeps 8 waves a SIMD, with
// the rest 7 (8192 x 8192 bf16: 5 waves of 91 registers 54 us, 8 waves 40; with the
// rest 5 waves 65, 7 waves 53; 4096 x 131072: 5 waves 183, 8 waves 188).
template <typename T, bool REST, int TOP, bool TRAIN, int THREADS>
__global__ __launch_bounds__(THREADS, TRAIN || TOP > kScanPairs ? 1 : REST ? 7 : 8) void distill_row_kernel(DistillArgs A) {
    extern __shared__ uint32_t bits[];
    __shared__ __attribute__((aligned(16))) PairLds<TOP> L;
    constexpr int kKept = !TRAIN ? 0 : REST && sizeof(T) == 2 ? kKeptVecs - 2 : kKeptVecs;   // without spilling
    const Span<T> S(0, A.vocab);
    const float c = A.inv_tau * kLog2e;
    for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x) {
        const T *z = reinterpret_cast<const T *>(A.logits) + row * A.ld;
        typename Vec16<T>::raw kept[kKept + 1];   // a row too long to hold has kHeldVecs vectors a thread and more
#pragma unroll
        for (int i = 0; i < kKept; ++i) kept[i] = load_vec<T>(z + (int64_t)(threadIdx.x + i * THREADS) * S.N);
        Pairs r = read_pairs<REST>(A, row, L, bits, (A.vocab + 31) >> 5);
        if (!r.some) {
            write_empty<T, REST>(A, row, S, true);
            __syncthreads();
            continue;
        }
        for (int k = threadIdx.x; k < A.top_k; k += THREADS) L.z[k] = L.id[k] >= 0 ? (float)z[L.id[k]] : 0.f;
        const float zt = tail_of<T>(z, S);
        weigh_pairs<REST>(A, teacher_lse<REST>(A, row), L, r, bits, 0, A.vocab);
        const FastBase f = fast_base(A, L, c);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kKept; ++i)
            sum += fast_sum<T, REST>(kept[i], REST ? vec_bits(bits, threadIdx.x + i * THREADS, S.N) : 0, c, f.hi);
        sum += fast_span<T, REST, TRAIN && REST ? 4 : 8>(z, zt, S, bits, c, f.hi, kKept * THREADS);
        Lse rest = {f.m, block_sum<THREADS>(sum, L) * __builtin_amdgcn_exp2f(-f.lo)};
        if (fast_holds(rest)) {
            rest = near(rest, c);
        } else {
            __syncthreads();
            rest = block_join(sum_span<T, REST>(z, zt, S, bits, c), L, c);
        }
        const RowSums s = row_sums<REST>(A, L, r, row, TRAIN ? A.grad_loss[row] : 0.f, rest, c);
        if constexpr (TRAIN) {
            T *dz = reinterpret_cast<T *>(A.dlogits) + row * A.dld;
#pragma unroll
            for (int i = 0; i < kKept; ++i)
                store_vec<T, true>(dz + (int64_t)(threadIdx.x + i * THREADS) * S.N, grad_vec<T>(kept[i], s.others, c, s.g_others));
            grad_span<T, true>(z, dz, S, s.others, c, s.g_others, kKept * THREADS);
            finish_span<T>(A, L, [&](int j, T x) { dz[j] = x; }, S, zt, s.n, s.others, c, s.g, s.g_others);
        }
        write_loss<REST>(A, L, r, row, s.n, s.all, s.rest);
        __syncthreads();   // the next row's pairs go into the same LDS
    }
}

// Few or very long rows: workgroup (chunk, row) sums its part of the row.
template <typename T, bool REST, int TOP>
__global__ __launch_bounds__(kSplitThreads) void distill_partial_kernel(DistillArgs A) {
    extern __shared__ uint32_t bits[];
    __shared__ __attribute__((aligned(16))) PairLds<TOP> L;
    const float c = A.inv_tau * kLog2e;
    for (uint32_t b = blockIdx.x; b < (uint32_t)A.rows * A.chunks; b += gridDim.x) {
        const int64_t row = b / (uint32_t)A.chunks;
        const int chunk = b % (uint32_t)A.chunks;
        const int e0 = chunk * A.chunk, e1 = min(e0 + A.chunk, A.vocab);
        const Span<T> S(e0, e1);
        const T *z = reinterpret_cast<const T *>(A.logits) + row * A.ld;
        const float zt = tail_of<T>(z, S);
        if (chunk == 0)
            for (int k = threadIdx.x; k < A.top_k; k += kSplitThreads) {
                const int id = token_of(A, pair_at(A, row, k));
                A.top_z[row * A.top_k + k] = id >= 0 ? (float)z[id] : 0.f;
            }
        if constexpr (REST) {
            const float lse = teacher_lse<REST>(A, row);
            Pairs r = read_pairs<REST>(A, row, L, bits, (A.chunk + 31) >> 5);
            weigh_pairs<REST>(A, lse, L, r, bits, e0, e1);
        }
        const Lse a = block_join(sum_span<T, REST>(z, zt, S, bits, c), L, c);
        if (threadIdx.x == 0) A.partial[row * A.chunks + chunk] = make_float2(a.m, a.s);
        __syncthreads();   // the next part uses the same LDS
    }
}

// The others' sum of a whole row (its pairs are in LDS and weighed), in parts
// whose marks fit: the largest logit, then the sum relative to it. One vector at
// a time: few registers, for a kernel that seldom needs it.
template <typename T, bool REST, int TOP>
__device__ inline Lse sum_row(const DistillArgs &A, PairLds<TOP> &L, const T *z, float c) {
    constexpr int N = Vec16<T>::N, kPart = kSplitThreads * N;   // a vector a thread
    __shared__ uint32_t marks[REST ? kPart / 32 : 1];
    float m = kNegInf, s = 0.f;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        if (pass) {
            m = wave_max(m);
            __syncthreads();
            if ((threadIdx.x & 63) == 0) L.wave_sum[threadIdx.x >> 6] = m;
            __syncthreads();
            m = fmaxf(fmaxf(L.wave_sum[0], L.wave_sum[1]), fmaxf(L.wave_sum[2], L.wave_sum[3]));
            __syncthreads();
        }
        const float base = m == kNegInf ? 0.f : m;
#pragma unroll 1
        for (int e0 = 0; e0 < A.vocab; e0 += kPart) {
            if constexpr (REST) {
                __syncthreads();   // the part before has been read
                for (int i = threadIdx.x; i < kPart / 32; i += kSplitThreads) marks[i] = 0;
                __syncthreads();
                for (int k = threadIdx.x; k < A.top_k; k += kSplitThreads) {
                    const int at = L.owner[k] - e0;
                    if (L.owner[k] >= 0 && at >= 0 && at < kPart) atomicOr(&marks[at >> 5], 1u << (at & 31));
                }
                __syncthreads();
            }
#pragma unroll 1
            for (int i = 0; i < N; ++i) {
                const int at = threadIdx.x + i * kSplitThreads;
                if (e0 + at >= A.vocab || (REST && (marks[at >> 5] >> (at & 31) & 1))) continue;
                const float x = (float)z[e0 + at];
                if (pass) s += __builtin_amdgcn_exp2f((x - base) * c);
                else m = fmaxf(m, x);
            }
        }
    }
    __syncthreads();
    return {m, block_sum<kSplitThreads>(s, L)};
}

// Workgroup (chunk, row) writes its part of the gradient, from the parts' sums
// (LOSS: the first one also the loss) or from the logsumexps of a forward call:
// each a whole row's sum again where they are too large. The gradient alone with
// the rest keeps 5 waves a SIMD (8192 x 8192 bf16: 4 waves 90 us, 5 waves 82).
template <typename T, bool REST, int TOP, bool LOSS, bool NT>
__global__ __launch_bounds__(kSplitThreads, !LOSS && REST && TOP <= kScanPairs ? 5 : 1) void distill_apply_kernel(DistillArgs A, int32_t parts) {
    extern __shared__ uint32_t bits[];
    __shared__ __attribute__((aligned(16))) PairLds<TOP> L;
    const float c = A.inv_tau * kLog2e;
    for (uint32_t b = blockIdx.x; b < (uint32_t)A.rows * A.chunks; b += gridDim.x) {
        const int64_t row = b / (uint32_t)A.chunks;
        const int chunk = b % (uint32_t)A.chunks;
        const int e0 = chunk * A.chunk, e1 = min(e0 + A.chunk, A.vocab);
        const Span<T> S(e0, e1);
        const T *z = reinterpret_cast<const T *>(A.logits) + row * A.ld;
        // what the part needs last is asked for first
        typename Vec16<T>::raw ahead[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int v = threadIdx.x + i * kSplitThreads;
            if (A.dlogits && v < S.vecs) ahead[i] = load_vec<T>(z + e0 + (int64_t)v * S.N);
        }
        const float zt = tail_of<T>(z, S);
        float2 part = make_float2(kNegInf, 0.f);   // at most kMaxChunks = 64: one a lane
        if (LOSS && (int)(threadIdx.x & 63) < parts) part = A.partial[row * parts + (threadIdx.x & 63)];
        const float g = A.dlogits ? A.grad_loss[row] : 0.f, t_lse = teacher_lse<REST>(A, row);
        if (LOSS)
            for (int k = threadIdx.x; k < A.top_k; k += kSplitThreads) L.z[k] = A.top_z[row * A.top_k + k];
        Pairs r = read_pairs<REST>(A, row, L, bits, 0);
        if (!r.some) {
            write_empty<T, REST>(A, row, S, LOSS && chunk == 0);
            __syncthreads();
            continue;
        }
        const float lse = LOSS ? 0.f : A.lse[row], rest_lse = !LOSS && REST ? A.rest_lse[row] : 0.f;
        const bool again = !LOSS && (too_large(lse) || too_large(rest_lse));   // -inf too: no others, or below fp32's range
        if (!LOSS && A.large != (again ? kLargeOnly : kLargeNone) && A.large != kLargeToo) {   // the other launch's row
            __syncthreads();
            continue;
        }
        if (!LOSS)
            for (int k = threadIdx.x; k < A.top_k; k += kSplitThreads) {
                const int id = L.id[k];
                L.z[k] = id >= (again ? 0 : e0) && id < (again ? A.vocab : e1) ? (float)z[id] : 0.f;
            }
        weigh_pairs<REST>(A, t_lse, L, r, bits, 0, 0);
        RowSums s{};
        if constexpr (LOSS) {
            s = row_sums<REST>(A, L, r, row, g, wave_join({part.x, part.y}, c), c);
        } else {
            if (again) {
                s = row_sums<REST>(A, L, r, row, g, sum_row<T, REST>(A, L, z, c), c);
            } else {
                s.n = s.others = norm_of_lse(lse, A.inv_tau);
                s.g = s.g_others = g * A.inv_tau;
                if constexpr (REST) {
                    s.others = norm_of_lse(rest_lse, A.inv_tau);
                    s.g_others = others_factor<REST>(r, s.g, expf(rest_lse - lse));
                    s.n.scale *= r.mass;
                }
            }
        }
        if (A.dlogits) {
            T *dz = reinterpret_cast<T *>(A.dlogits) + row * A.dld;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int v = threadIdx.x + i * kSplitThreads;
                if (v < S.vecs) store_vec<T, NT>(dz + e0 + (int64_t)v * S.N, grad_vec<T>(ahead[i], s.others, c, s.g_others));
            }
            grad_span<T, NT>(z, dz, S, s.others, c, s.g_others, kAhead * kSplitThreads);
            finish_span<T>(A, L, [&](int j, T x) { dz[j] = x; }, S, zt, s.n, s.others, c, s.g, s.g_others);
        }
        if (LOSS && chunk == 0) write_loss<REST>(A, L, r, row, s.n, s.all, s.rest);
        __syncthreads();   // the next part uses the same LDS
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// Parts of a row for the split kernels: 512 workgroups over few rows if parts of
// 2048 tokens give as many, up to 4096 of parts of 16384 (and no part longer than
// one workgroup marks in LDS).
void set_chunks(DistillArgs &a) {
    const auto deal = [&](int64_t workgroups, int64_t tokens) {
        return std::min((workgroups + a.rows - 1) / a.rows, (a.vocab + tokens - 1) / tokens);
    };
    int64_t parts = std::max(deal(512, 2048), deal(4096, 16384));
    parts = std::max<int64_t>(parts, (a.vocab + kBitVocab - 1) / kBitVocab);
    parts = std::max<int64_t>(1, std::min<int64_t>(parts, kMaxChunks));
    a.chunk = (int32_t)(((a.vocab + parts - 1) / parts + 31) / 32 * 32);
    a.chunks = (a.vocab + a.chunk - 1) / a.chunk;
}

// Threads that hold a row in registers and have a pair each; over 1024 for a row
// that cannot be held. (More of them where few rows leave some idle gained
// nothing: 300 x 8192 bf16 13.7 us, with 512 threads in place of 64 15.8.)
int64_t held_threads(const DistillArgs &a, int es) {
    const int64_t vecs = (int64_t)a.vocab * es / 16;
    int64_t threads = 64;
    while (threads <= 1024 && (vecs > kHeldVecs * threads || a.top_k > threads)) threads *= 2;
    return threads;
}
// Which calls split their rows over workgroups and run two kernels. Training
// takes a row to a workgroup from 256 on (one a CU; 600 x 131072 bf16, held: 81 us,
// split 91; 900 x 160000 bf16, not held: 140 us, split 181; 300 x 100001 f32 66 and
// 79); loss alone reads rows one to a workgroup of 256 threads once these fill the
// GPU (600 x 131072 bf16: split 38 us, a workgroup a row 44).
bool split_rows(const DistillArgs &a) {
    if (a.teacher_lse && a.vocab > kBitVocab) return true;
    return a.rows < (a.dlogits ? 256 : 1024);
}

size_t distill_workspace(int64_t rows, int32_t top_k, bool split) {
    return split ? (size_t)rows * ((size_t)kMaxChunks * sizeof(float2) + (size_t)top_k * sizeof(float)) : 0;
}

ns_status check_sizes(int64_t rows, int32_t vocab, int32_t top_k) {
    if (rows < 0 || rows > kMaxRows) return fail(NS_ERR_INVALID_ARG, "rows = %lld outside [0, %d]", (long long)rows, kMaxRows);
    if (vocab < 1 || vocab > kMaxVocab) return fail(NS_ERR_INVALID_ARG, "vocab = %d outside [1, %d]", vocab, kMaxVocab);
    if (top_k < 1 || top_k > kMaxTop) return fail(NS_ERR_INVALID_ARG, "top_k = %d outside [1, %d]", top_k, kMaxTop);
    return NS_OK;
}

ns_status check_distill(int64_t rows, int32_t vocab, int32_t top_k, int32_t dtype, const void *logits, int64_t ld,
                        const void *ids, int32_t id_bytes, const void *teacher, int32_t teacher_dtype,
                        const float *teacher_lse, float temperature, const float *grad_loss, void *dlogits,
                        int64_t dld, bool grad, DistillArgs *a) {
    const int es = dtype_bytes(dtype);
    if (!es) return fail(NS_ERR_DTYPE, "dtype %d is not NS_BF16 or NS_F32", dtype);
    if (!dtype_bytes(teacher_dtype)) return fail(NS_ERR_DTYPE, "teacher_dtype %d is not NS_BF16 or NS_F32", teacher_dtype);
    if (ns_status s = check_sizes(rows, vocab, top_k)) return s;
    if (id_bytes != 4 && id_bytes != 8) return fail(NS_ERR_DTYPE, "id_bytes = %d (must be 4 or 8)", id_bytes);
    const float inv_tau = 1.f / temperature;
    if (!(temperature > 0.f) || !(inv_tau > 0.f) || inv_tau > 1e30f || temperature > 1e30f)
        return fail(NS_ERR_INVALID_ARG, "temperature must be within [1e-30, 1e30]");
    if (ld < vocab || (dlogits && dld < vocab)) return fail(NS_ERR_INVALID_ARG, "row stride < vocab");
    if (too_far(rows, ld) || too_far(rows * ld, es) || (dlogits && (too_far(rows, dld) || too_far(rows * dld, es))))
        return fail(NS_ERR_OVERFLOW, "logits: offsets overflow");
    if (rows > 0 && (!logits || !ids || !teacher)) return fail(NS_ERR_INVALID_ARG, "logits, ids and teacher are required");
    if (rows > 0 && grad && (!dlogits || !grad_loss))
        return fail(NS_ERR_INVALID_ARG, "dlogits and grad_loss are required together");
    if (misaligned(logits, es) || misaligned(dlogits, es) || misaligned(ids, id_bytes) ||
        misaligned(teacher, dtype_bytes(teacher_dtype)) || misaligned(teacher_lse, 4) || misaligned(grad_loss, 4))
        return fail(NS_ERR_INVALID_ARG, "a buffer is not aligned to its type");
    if (dlogits == logits && dlogits && dld != ld)
        return fail(NS_ERR_INVALID_ARG, "dlogits in place of logits needs the same row stride");
    *a = DistillArgs{};
    a->logits = logits;
    a->ld = ld;
    a->ids = ids;
    a->id_bytes = id_bytes;
    a->teacher = teacher;
    a->teacher_f32 = teacher_dtype == NS_F32;
    a->teacher_lse = teacher_lse;
    a->grad_loss = grad_loss;
    a->dlogits = dlogits;
    a->dld = dld;
    a->rows = (int32_t)rows;
    a->vocab = vocab;
    a->top_k = top_k;
    a->inv_tau = inv_tau;
    a->inv_tau64 = 1. / temperature;
    return NS_OK;
}

// Workgroups of a split launch: at most 2^20, which then take several parts each.
unsigned split_grid(const DistillArgs &a) { return (unsigned)std::min<int64_t>((int64_t)a.rows * a.chunks, 1 << 20); }

// Whether reading the logits and writing their gradient passes more than the
// last-level cache holds; the gradient is then stored past it (1025 x 50021 f32
// backward: 83 -> 67 us; 300 x 131072 bf16, 157 MB: no difference).
bool past_cache(const DistillArgs &a, int es) { return 2.0 * a.rows * a.vocab * es > (double)kMallBytes; }

template <typename T, bool REST, int TOP>
ns_status launch_rows(const DistillArgs &a, hipStream_t st) {
    const size_t lds = REST ? (size_t)((a.vocab + 31) / 32 + 1) * 4 : 0;   // lanes past the row read one byte behind it
    auto go = [&](auto kernel, int threads, int64_t most) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)std::min<int64_t>(a.rows, most)), dim3(threads), lds, st, a);
    };
    // Held rows: as many workgroups as are resident at once, 16 waves a CU.
    const auto held = [&](auto kernel, int threads) { go(kernel, threads, 256 * (1024 / threads)); };
    switch (a.dlogits ? held_threads(a, sizeof(T)) : 2048) {
    case 64: held(distill_held_kernel<T, 64, REST, std::min(64, TOP)>, 64); break;
    case 128: held(distill_held_kernel<T, 128, REST, std::min(128, TOP)>, 128); break;
    case 256: held(distill_held_kernel<T, 256, REST, std::min(256, TOP)>, 256); break;
    case 512: held(distill_held_kernel<T, 512, REST, std::min(512, TOP)>, 512); break;
    case 1024: held(distill_held_kernel<T, 1024, REST, std::min(1024, TOP)>, 1024); break;
    default:
        if (a.dlogits) go(distill_row_kernel<T, REST, TOP, true, 1024>, 1024, 256);   // one a CU
        else go(distill_row_kernel<T, REST, TOP, false, kSplitThreads>, kSplitThreads, 1 << 20);
    }
    NSQ_HIP(hipGetLastError());
    return NS_OK;
}

template <typename T, bool REST, int TOP>
ns_status launch_split(DistillArgs a, hipStream_t st) {
    set_chunks(a);
    const size_t lds = REST ? (size_t)((a.chunk + 31) / 32) * 4 : 0;
    hipLaunchKernelGGL((distill_partial_kernel<T, REST, TOP>), dim3(split_grid(a)), dim3(kSplitThreads), lds, st, a);
    NSQ_HIP(hipGetLastError());
    const int32_t parts = a.chunks;
    if (!a.dlogits) a.chunks = 1, a.chunk = a.vocab;
    hipLaunchKernelGGL((distill_apply_kernel<T, REST, TOP, true, false>), dim3(split_grid(a)), dim3(kSplitThreads), 0, st, a, parts);
    NSQ_HIP(hipGetLastError());
    return NS_OK;
}

// The gradient in place of the logits leaves rows that are summed again to a
// second launch, in which one workgroup takes all of a row (parts of it would read
// what others have written).
template <typename T, bool REST, int TOP>
ns_status launch_backward(DistillArgs a, hipStream_t st) {
    set_chunks(a);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(split_grid(a)), dim3(kSplitThreads), 0, st, a, 0); };
    const auto rows = [&](int32_t large) {
        a.large = large;
        past_cache(a, sizeof(T)) ? go(distill_apply_kernel<T, REST, TOP, false, true>) : go(distill_apply_kernel<T, REST, TOP, false, false>);
    };
    const bool place = a.dlogits == a.logits && a.chunks > 1;
    rows(place ? kLargeNone : kLargeToo);
    NSQ_HIP(hipGetLastError());
    if (place) {
        a.chunks = 1;
        a.chunk = a.vocab;
        rows(kLargeOnly);
        NSQ_HIP(hipGetLastError());
    }
    return NS_OK;
}

// go(T, teacher's rest, room for pairs) for a call's types and sizes.
template <typename Go> ns_status by_type(const DistillArgs &a, int32_t dtype, const Go &go) {
    const auto by_top = [&](auto t, auto rest) {
        if (a.top_k <= kScanPairs) return go(t, rest, std::integral_constant<int, kScanPairs>());
        return go(t, rest, std::integral_constant<int, kMaxTop>());
    };
    const auto by_rest = [&](auto t) {
        if (a.teacher_lse) return by_top(t, std::true_type());
        return by_top(t, std::false_type());
    };
    return dtype == NS_BF16 ? by_rest((__bf16)0.f) : by_rest(0.f);
}

}  // namespace
}  // namespace nsq

using namespace nsq;

extern "C" ns_status ns_distill_workspace_bytes(int64_t rows, int32_t vocab, int32_t top_k, size_t *bytes) {
    if (!bytes) return fail(NS_ERR_INVALID_ARG, "bytes is NULL");
    if (ns_status s = check_sizes(rows, vocab, top_k)) return s;
    *bytes = distill_workspace(rows, top_k, rows < 1024 || vocab > kBitVocab);
    return NS_OK;
}

extern "C" ns_status ns_distill_topk(int64_t rows, int32_t vocab, int32_t top_k, ns_dtype dtype, const void *logits,
                                     int64_t logits_ld, const void *ids, int32_t id_bytes, const void *teacher,
                                     ns_dtype teacher_dtype, const float *teacher_lse, float temperature,
                                     const float *grad_loss, float *loss, float *lse, float *rest_lse, void *dlogits,
                                     int64_t dlogits_ld, void *workspace, size_t workspace_bytes, void *stream) {
    DistillArgs a;
    if (ns_status s = check_distill(rows, vocab, top_k, dtype, logits, logits_ld, ids, id_bytes, teacher, teacher_dtype,
                                    teacher_lse, temperature, grad_loss, dlogits, dlogits_ld, dlogits || grad_loss, &a))
        return s;
    if (rows > 0 && (!loss || !lse)) return fail(NS_ERR_INVALID_ARG, "loss and lse are required");
    if (rows > 0 && teacher_lse && !rest_lse) return fail(NS_ERR_INVALID_ARG, "teacher_lse needs rest_lse");
    if (misaligned(loss, 4) || misaligned(lse, 4) || misaligned(rest_lse, 4))
        return fail(NS_ERR_INVALID_ARG, "loss, lse or rest_lse not 4-byte aligned");
    const bool split = split_rows(a);
    const size_t need = distill_workspace(rows, top_k, split);
    if (need && (!workspace || workspace_bytes < need))
        return fail(NS_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : 0, need);
    if (misaligned(workspace, 256)) return fail(NS_ERR_INVALID_ARG, "workspace not 256-byte aligned");
    if (rows == 0) return NS_OK;
    a.loss = loss;
    a.lse = lse;
    a.rest_lse = rest_lse;
    const hipStream_t st = as_stream(stream);
    if (split) {
        a.partial = reinterpret_cast<float2 *>(workspace);
        a.top_z = reinterpret_cast<float *>(a.partial + rows * kMaxChunks);
        return by_type(a, dtype, [&](auto t, auto rest, auto top) {
            return launch_split<decltype(t), decltype(rest)::value, decltype(top)::value>(a, st);
        });
    }
    return by_type(a, dtype, [&](auto t, auto rest, auto top) {
        return launch_rows<decltype(t), decltype(rest)::value, decltype(top)::value>(a, st);
    });
}

extern "C" ns_status ns_distill_topk_backward(int64_t rows, int32_t vocab, int32_t top_k, ns_dtype dtype,
                                              const void *logits, int64_t logits_ld, const void *ids, int32_t id_bytes,
                                              const void *teacher, ns_dtype teacher_dtype, const float *teacher_lse,
                                              float temperature, const float *lse, const float *rest_lse,
                                              const float *grad_loss, void *dlogits, int64_t dlogits_ld,
                                              void *stream) {
    DistillArgs a;
    if (ns_status s = check_distill(rows, vocab, top_k, dtype, logits, logits_ld, ids, id_bytes, teacher, teacher_dtype,
                                    teacher_lse, temperature, grad_loss, dlogits, dlogits_ld, true, &a))
        return s;
    if (rows > 0 && !lse) return fail(NS_ERR_INVALID_ARG, "lse is required");
    if (rows > 0 && teacher_lse && !rest_lse) return fail(NS_ERR_INVALID_ARG, "teacher_lse needs rest_lse");
    if (misaligned(lse, 4) || misaligned(rest_lse, 4)) return fail(NS_ERR_INVALID_ARG, "lse or rest_lse not 4-byte aligned");
    if (rows == 0) return NS_OK;
    a.lse = const_cast<float *>(lse);
    a.rest_lse = const_cast<float *>(rest_lse);
    const hipStream_t st = as_stream(stream);
    return by_type(a, dtype, [&](auto t, auto rest, auto top) {
        return launch_backward<decltype(t), decltype(rest)::value, decltype(top)::value>(a, st);
    });
}
