// Per-head RMS norm of queries and keys with the position rotation in the same
// pass, and its gradient.
//
// For one head x of D values at position p, with weight w and the angles of p:
//   r = rsqrt(mean(x^2) + eps),  n = x r,  u = n w,
//   y = u with the pairs (i, i + R/2) (or (2i, 2i + 1)) of its first R values
//       turned by angle i: (a cos - b sin, b cos + a sin).
// Backward, from g = dL/dy: du is g turned by the negative angles,
//   dw = sum over tokens and heads of du n,  dn = du w,
//   dx = r (dn - n mean(dn n)).
// r is computed again from x, so the forward pass saves nothing.
//
// Layout: a group of G lanes (a power of two) holds one head, each lane two
// pieces of 8 elements of it that the rotation pairs up (pieces at 8i and 8i +
// R/2, or two neighbours for (2i, 2i + 1) pairs), so a rotation needs no other
// lane and the sums need log2 G exchanges. A wave holds 64 / G heads of one
// token at a time and loads its next token's while it computes. Heads whose size
// or rotated part does not split into such pieces take the same code with pieces
// of 4 elements or of one (VEC), a lane then holding up to eight pairs of them.
//
// Bound by memory: each input is read once and each output written once.

#include <algorithm>
#include <type_traits>

#include "op_util.h"

namespace nsq {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxHeadDim = 1024;
constexpr int kMaxHeads = 1024;
// Workgroups of a launch, for pieces of 8, 4 and 1 elements: as many as are
// resident at once by the kernels' registers, so that a wave keeps its weights
// and its place in a head over all its tokens. 16384 tokens of 32 + 8 bf16 heads
// of 128, forward: 1024 workgroups 63.6 us, 2048 64.2, 1536 (a second, partial
// round) 67.4. Backward: 512 94 us, 768 100, 1024 110, 384 110.
constexpr int blocks_for(int vec, bool backward) {
    return backward ? (vec == 4 ? 1024 : 512) : (vec == 8 ? 1024 : vec == 4 ? 2048 : 768);
}
constexpr int kMostPartials = 1024;
// Outputs of calls that move more than the last-level cache holds are stored
// past it: 66 us became 63 in the case above, 104 102. Smaller ones stay in
// it for the kernel that reads them next (35 us against 43 for 45 MB each way):
// see deal().

// One (batch, seq, heads, head_dim) tensor: address, and element strides of batch, token and head.
struct Operand {
    char *p;
    int64_t b, t, h;
};

struct HeadArgs {
    Operand x[2], g[2], y[2];        // of the queries and of the keys: input, gradient of the output (backward), output
    const void *w[2];
    float *dw[2];
    int32_t heads[2];
    uint32_t seq, tokens;            // tokens = batch x seq
    uint32_t chunks, stride;         // chunks of 64 / G heads, queries before keys; tokens taken at once
    uint32_t step_i, step_s;         // stride = step_i seq + step_s
    int32_t blocks;
    int32_t D, R, P, RP;             // head size, rotated part, pairs of pieces per head, rotated ones
    int32_t lg;                      // log2 G
    int32_t interleaved, w_f32;
    float eps;
    const float *cos, *sin;
    int64_t table_rows;
    const void *pos;
    int32_t pos_bytes;
    int64_t pos_bs;
    float *partial;                  // backward: [workgroups][queries, keys][D]
};

// VEC elements at any element alignment, as one or two loads or stores.
template <typename T, int VEC> struct Piece {
    typedef typename std::conditional<sizeof(T) == 2, uint16_t, float>::type E;
    typedef E raw __attribute__((ext_vector_type(VEC)));
    typedef raw __attribute__((aligned(sizeof(T)))) raw_u;
    static __device__ inline raw load(const T *p) {
        if constexpr (VEC == 1) return raw{*reinterpret_cast<const E *>(p)};
        else return *reinterpret_cast<const raw_u *>(p);
    }
    static __device__ inline void widen(raw r, float (&v)[VEC]) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            if constexpr (sizeof(T) == 2) v[i] = __builtin_bit_cast(float, (uint32_t)r[i] << 16);
            else v[i] = r[i];
        }
    }
    template <bool NT> static __device__ inline void store(T *p, const float (&v)[VEC]) {
        raw r;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            if constexpr (sizeof(T) == 2) r[i] = __builtin_bit_cast(uint16_t, (__bf16)v[i]);
            else r[i] = v[i];
        }
        if constexpr (VEC == 1) *reinterpret_cast<E *>(p) = r[0];
        else if constexpr (NT) __builtin_nontemporal_store(r, reinterpret_cast<raw_u *>(p));
        else *reinterpret_cast<raw_u *>(p) = r;
    }
};

// A lane's two pieces of a head: element offsets a and b, and their angles' place in a table row.
struct Place {
    int a, b, angle;
    bool in, has_b, turned;
};

template <int VEC>
__device__ inline Place place_of(const HeadArgs &A, int i) {
    Place p;
    p.in = i < A.P;
    p.turned = i < A.RP;
    p.angle = i * VEC;
    if (p.turned) {
        p.a = A.interleaved ? 2 * i * VEC : i * VEC;
        p.b = A.interleaved ? p.a + VEC : p.a + A.R / 2;
    } else {
        p.a = A.R + 2 * (i - A.RP) * VEC;
        p.b = p.a + VEC;
    }
    p.has_b = p.in && p.b < A.D;   // VEC = 1: an odd unrotated tail has no partner
    // lanes without a piece read the head's first one, so that loads need no branch
    if (!p.in) p.a = 0;
    if (!p.has_b) p.b = p.a;
    return p;
}

template <int VEC>
__device__ inline void load_weight(const HeadArgs &A, const void *w, const Place &p, float (&wa)[VEC], float (&wb)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) wa[i] = wb[i] = 1.f;
    if (!w) return;
    if (A.w_f32) {
        Piece<float, VEC>::widen(Piece<float, VEC>::load(reinterpret_cast<const float *>(w) + p.a), wa);
        Piece<float, VEC>::widen(Piece<float, VEC>::load(reinterpret_cast<const float *>(w) + p.b), wb);
    } else {
        Piece<__bf16, VEC>::widen(Piece<__bf16, VEC>::load(reinterpret_cast<const __bf16 *>(w) + p.a), wa);
        Piece<__bf16, VEC>::widen(Piece<__bf16, VEC>::load(reinterpret_cast<const __bf16 *>(w) + p.b), wb);
    }
}

// cos and sin of a position's angles: from a descriptor of one table row, of length
// zero for a position outside the table; such a row's values are then set to NaN.
template <int VEC, int NP> struct Angles {
    float c[NP][VEC], s[NP][VEC];
    __device__ inline void load(const HeadArgs &A, int64_t at, const Place (&pl)[NP]) {
        const bool in = at >= 0 && at < A.table_rows;
        const int64_t row = in ? at * (A.R / 2) : 0;
        const auto rc = __builtin_amdgcn_make_buffer_rsrc(const_cast<float *>(A.cos + row), (short)0, in ? A.R * 2 : 0, 0x00020000);
        const auto rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<float *>(A.sin + row), (short)0, in ? A.R * 2 : 0, 0x00020000);
        typedef float f4 __attribute__((ext_vector_type(4)));
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            if constexpr (VEC == 1) {
                c[n][0] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rc, pl[n].angle * 4, 0, 0));
                s[n][0] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, pl[n].angle * 4, 0, 0));
            } else {
#pragma unroll
                for (int q = 0; q < VEC / 4; ++q) {
                    const f4 x = __builtin_bit_cast(f4, __builtin_amdgcn_raw_buffer_load_b128(rc, pl[n].angle * 4 + 16 * q, 0, 0));
                    const f4 y = __builtin_bit_cast(f4, __builtin_amdgcn_raw_buffer_load_b128(rs, pl[n].angle * 4 + 16 * q, 0, 0));
#pragma unroll
                    for (int i = 0; i < 4; ++i) c[n][4 * q + i] = x[i], s[n][4 * q + i] = y[i];
                }
            }
        }
    }
    __device__ inline void check(const HeadArgs &A, int64_t at) {
        if (at >= 0 && at < A.table_rows) return;
#pragma unroll
        for (int n = 0; n < NP; ++n)
#pragma unroll
            for (int i = 0; i < VEC; ++i) c[n][i] = s[n][i] = __builtin_nanf("");
    }
};

// Turns the pieces a, b by the angles (dir = 1) or back (dir = -1).
template <int VEC>
__device__ inline void turn(bool interleaved, float dir, float (&a)[VEC], float (&b)[VEC], const float (&c)[VEC],
                            const float (&s)[VEC]) {
    if (VEC == 1 || !interleaved) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float x = a[i], y = b[i], t = dir * s[i];
            a[i] = x * c[i] - y * t;
            b[i] = y * c[i] + x * t;
        }
    } else if constexpr (VEC > 1) {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            const float x = a[2 * i], y = a[2 * i + 1], t = dir * s[i];
            a[2 * i] = x * c[i] - y * t;
            a[2 * i + 1] = y * c[i] + x * t;
            const float u = b[2 * i], v = b[2 * i + 1], r = dir * s[VEC / 2 + i];
            b[2 * i] = u * c[VEC / 2 + i] - v * r;
            b[2 * i + 1] = v * c[VEC / 2 + i] + u * r;
        }
    }
}

// A wave's place in (batch, seq), moved on by `stride` tokens at a time, and an
// operand's address there as a lane sees it (its set's strides, its head), which
// follows by additions: the way of one step, and of the turn into the next batch.
struct Cursor {
    uint32_t i, s;
    __device__ inline bool step(const HeadArgs &A) {
        i += A.step_i;
        s += A.step_s;
        const bool turned = s >= A.seq;
        if (turned) i += 1, s -= A.seq;
        return turned;
    }
};

// The token's position (read through the scalar cache: no kernel writes it).
__device__ inline int64_t position(const HeadArgs &A, Cursor c) {
    if (!A.pos) return c.s;
    const int64_t at = c.i * A.pos_bs + c.s;
    if (A.pos_bytes == 8) return *(const int64_t NSQ_CONST *)(reinterpret_cast<const int64_t *>(A.pos) + at);
    return *(const int32_t NSQ_CONST *)(reinterpret_cast<const int32_t *>(A.pos) + at);
}

template <typename T> struct Walk {
    T *p;
    int64_t step, turn;
    __device__ Walk(const HeadArgs &A, const Operand (&of)[2], bool key, int64_t head, Cursor at) {
        const int64_t b = key ? of[1].b : of[0].b, t = key ? of[1].t : of[0].t;
        p = reinterpret_cast<T *>(key ? of[1].p : of[0].p) + head * (key ? of[1].h : of[0].h) + at.i * b + at.s * t;
        step = A.step_i * b + A.step_s * t;
        turn = b - (int64_t)A.seq * t;
    }
    __device__ inline void move(bool turned) {
        p += step;
        if (turned) p += turn;
    }
};

// Forward, or with BWD the gradient. A wave holds chunk w % chunks of the heads
// (queries, then keys) and takes the tokens w / chunks, + stride, ...; the next
// token's values and angles are on their way while it computes. Lanes without a
// head or a piece load another's and store nothing.
template <typename T, int VEC, int NP, bool BWD, bool NT>
__global__ __launch_bounds__(kThreads) void qk_kernel(HeadArgs A) {
    typedef Piece<T, VEC> PT;
    typedef typename PT::raw raw;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t w = blockIdx.x * kWaves + wave;
    const uint32_t first = w / A.chunks, chunk = w - first * A.chunks;
    const int head = (int)chunk * (64 >> A.lg) + (lane >> A.lg);
    const bool here = head < A.heads[0] + A.heads[1];
    const bool key = A.heads[0] == 0 || (here && head >= A.heads[0]);
    const int64_t h = !here ? 0 : key ? head - A.heads[0] : head;
    Place pl[NP];
    float wa[NP][VEC], wb[NP][VEC], dwa[NP][VEC], dwb[NP][VEC];
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        pl[n] = place_of<VEC>(A, (lane & ((1 << A.lg) - 1)) + (n << A.lg));
        load_weight<VEC>(A, key ? A.w[1] : A.w[0], pl[n], wa[n], wb[n]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) dwa[n][i] = dwb[n][i] = 0.f;
    }
    // waves past the last whole round of chunks have no tokens
    const uint32_t stride = A.stride, begin = first < stride ? first : A.tokens;
    Cursor ahead;
    ahead.i = begin < A.tokens ? begin / A.seq : 0;
    ahead.s = begin < A.tokens ? begin - ahead.i * A.seq : 0;
    Walk<T> X(A, A.x, key, h, ahead), G(A, A.g, key, h, ahead), Y(A, A.y, key, h, ahead);
    const float inv_d = 1.f / (float)A.D;
    raw xa[NP], xb[NP], ga[NP], gb[NP];
    Angles<VEC, NP> ang;
    const auto load = [&] {
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            xa[n] = PT::load(X.p + pl[n].a);
            xb[n] = PT::load(X.p + pl[n].b);
            if constexpr (BWD) {
                ga[n] = PT::load(G.p + pl[n].a);
                gb[n] = PT::load(G.p + pl[n].b);
            }
        }
    };
    // tokens and stride are below 2^31: no wrap
    int64_t pos = 0, pos_next = 0;
    bool turned = false;   // the step to the next token enters another batch
    if (begin < A.tokens) {
        pos = position(A, ahead);
        load();
        ang.load(A, pos, pl);
        if (begin + stride < A.tokens) turned = ahead.step(A);
        pos_next = position(A, ahead);
    }
    for (uint32_t t = begin; t < A.tokens; t += stride) {
        float va[NP][VEC], vb[NP][VEC], da[NP][VEC], db[NP][VEC];
        Angles<VEC, NP> now = ang;
        now.check(A, pos);
        float ss = 0.f, sd = 0.f;
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            PT::widen(xa[n], va[n]);
            PT::widen(xb[n], vb[n]);
            if constexpr (BWD) {
                PT::widen(ga[n], da[n]);
                PT::widen(gb[n], db[n]);
            }
        }
        const bool more = t + stride < A.tokens;
        if (more) {
            X.move(turned);
            if constexpr (BWD) G.move(turned);
        }
        load();
        ang.load(A, pos_next, pl);
        pos = pos_next;
        bool turned_next = false;
        if (more && t + stride + stride < A.tokens) turned_next = ahead.step(A);
        pos_next = position(A, ahead);
#pragma unroll
        for (int n = 0; n < NP; ++n) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                if (!pl[n].in) va[n][i] = 0.f;
                if (!pl[n].has_b) vb[n][i] = 0.f;
            }
            if constexpr (BWD) {
                if (pl[n].turned) turn<VEC>(A.interleaved, -1.f, da[n], db[n], now.c[n], now.s[n]);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    if (!pl[n].in) da[n][i] = 0.f;
                    if (!pl[n].has_b) db[n][i] = 0.f;
                }
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                ss += va[n][i] * va[n][i] + vb[n][i] * vb[n][i];
                if constexpr (BWD) sd += da[n][i] * wa[n][i] * va[n][i] + db[n][i] * wb[n][i] * vb[n][i];
            }
        }
        ss = group_sum(ss, A.lg);
        const float r = 1.f / sqrtf(ss * inv_d + A.eps);
        float m = 0.f;
        if constexpr (BWD) m = group_sum(sd, A.lg) * r * inv_d;   // mean(dn n)
#pragma unroll
        for (int n = 0; n < NP; ++n) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float na = va[n][i] * r, nb = vb[n][i] * r;
                if constexpr (BWD) {
                    if (here) {
                        dwa[n][i] += da[n][i] * na;
                        dwb[n][i] += db[n][i] * nb;
                    }
                    va[n][i] = r * (da[n][i] * wa[n][i] - na * m);
                    vb[n][i] = r * (db[n][i] * wb[n][i] - nb * m);
                } else {
                    va[n][i] = na * wa[n][i];
                    vb[n][i] = nb * wb[n][i];
                }
            }
            if constexpr (!BWD)
                if (pl[n].turned) turn<VEC>(A.interleaved, 1.f, va[n], vb[n], now.c[n], now.s[n]);
            if (here && pl[n].in) {
                PT::template store<NT>(Y.p + pl[n].a, va[n]);
                if (pl[n].has_b) PT::template store<NT>(Y.p + pl[n].b, vb[n]);
            }
        }
        if (more) Y.move(turned);
        turned = turned_next;
    }
    if constexpr (BWD) {
        // The workgroup's parts of dw, queries' and keys': each thread sums an element over
        // the waves and their heads, in a fixed order that starts where its banks are free.
        __shared__ float lds[kWaves][2 * VEC * NP][64];
        __shared__ uint64_t keys[kWaves];
#pragma unroll
        for (int n = 0; n < NP; ++n)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                lds[wave][(n * 2) * VEC + i][lane] = dwa[n][i];
                lds[wave][(n * 2 + 1) * VEC + i][lane] = dwb[n][i];
            }
        const uint64_t mine = __ballot(key);
        if (lane == 0) keys[wave] = mine;
        __syncthreads();
        const int groups = 64 >> A.lg, per_set = 2 * VEC * NP << A.lg;
        for (int j = threadIdx.x; j < 2 * per_set; j += kThreads) {
            const int set = j >= per_set, r = j - (set ? per_set : 0), e = r >> A.lg, l = r & ((1 << A.lg) - 1);
            if (!(set ? A.dw[1] : A.dw[0])) continue;
            const Place at = place_of<VEC>(A, l + ((e / (2 * VEC)) << A.lg));
            const bool second = (e / VEC) & 1;
            if (!at.in || (second && !at.has_b)) continue;
            float sum = 0.f;
            for (int v = 0; v < kWaves; ++v) {
                const uint64_t k = set ? keys[v] : ~keys[v];
                for (int i = 0; i < groups; ++i) {
                    const int from = (((i + e) & (groups - 1)) << A.lg) + l;
                    sum += k >> from & 1 ? lds[v][e][from] : 0.f;
                }
            }
            A.partial[((int64_t)blockIdx.x * 2 + set) * A.D + (second ? at.b : at.a) + e % VEC] = sum;
        }
    }
}

// dw[j] = sum of the workgroups' partials: 16 values a workgroup, 64 threads
// down the rows of each, joined in a fixed order.
constexpr int kJoinCols = 16, kJoinRows = 64;
__global__ __launch_bounds__(kJoinCols * kJoinRows) void qk_join_kernel(HeadArgs A) {
    __shared__ float part[kJoinRows / 4][kJoinCols];
    const int col = threadIdx.x % kJoinCols, down = threadIdx.x / kJoinCols;
    const int j = blockIdx.x * kJoinCols + col;
    const bool key = blockIdx.y;
    float *dw = key ? A.dw[1] : A.dw[0];
    if (!dw) return;
    const float *partial = A.partial + (key ? A.D : 0);
    float sum = 0.f;
    if (j < A.D) {
#pragma unroll 8
        for (int r = down; r < A.blocks; r += kJoinRows) sum += partial[(int64_t)r * 2 * A.D + j];
    }
    sum += __shfl_xor(sum, 16);   // a wave holds four rows of the 16 values
    sum += __shfl_xor(sum, 32);
    if ((threadIdx.x & 63) < kJoinCols) part[threadIdx.x >> 6][col] = sum;
    __syncthreads();
    if (threadIdx.x < kJoinCols && j < A.D) {
        sum = 0.f;
        for (int i = 0; i < kJoinRows / 4; ++i) sum += part[i][col];
        dw[j] = sum;
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// One head tensor's checks. want_heads: the heads an output or its gradient has to
// have. out: it is written, so no two of its heads may lie closer than their size.
ns_status check_heads(const char *name, const ns_heads *h, int64_t batch, int64_t seq, int32_t D, int es,
                      int32_t want_heads, bool out = false) {
    if (!h) return fail(NS_ERR_INVALID_ARG, "%s is NULL", name);
    if (h->heads < 0) return fail(NS_ERR_INVALID_ARG, "%s: heads = %d < 0", name, h->heads);
    if (h->heads > kMaxHeads) return fail(NS_ERR_OVERFLOW, "%s: more than %d heads", name, kMaxHeads);
    if (want_heads >= 0 && h->heads != want_heads)
        return fail(NS_ERR_INVALID_ARG, "%s has %d heads, not %d", name, h->heads, want_heads);
    if (h->heads == 0 || batch == 0 || seq == 0) return NS_OK;
    if (!h->data) return fail(NS_ERR_INVALID_ARG, "%s: data is NULL", name);
    if (misaligned(h->data, es)) return fail(NS_ERR_INVALID_ARG, "%s: data not %d-byte aligned", name, es);
    if (h->batch_stride < 0 || h->token_stride < 0 || h->head_stride < 0)
        return fail(NS_ERR_INVALID_ARG, "%s: negative stride", name);
    if (out && ((batch > 1 && h->batch_stride < D) || (seq > 1 && h->token_stride < D) ||
                (h->heads > 1 && h->head_stride < D)))
        return fail(NS_ERR_INVALID_ARG, "%s: an output's heads overlap (a stride below head_dim)", name);
    if (too_far(batch, h->batch_stride) || too_far(seq, h->token_stride) || too_far(h->heads, h->head_stride))
        return fail(NS_ERR_OVERFLOW, "%s: offsets overflow", name);
    if (batch * (double)h->batch_stride + seq * (double)h->token_stride + h->heads * (double)h->head_stride + D >
        4.6e18 / es)
        return fail(NS_ERR_OVERFLOW, "%s: offsets overflow", name);
    return NS_OK;
}

Operand operand(const ns_heads *h) { return {(char *)h->data, h->batch_stride, h->token_stride, h->head_stride}; }

struct HeadCall {
    HeadArgs a;
    int vec;       // elements of a piece: 8, 4 or 1
    bool past_cache;
    int es;
};

ns_status plan_heads(int64_t batch, int64_t seq, int32_t head_dim, int32_t dtype, const ns_heads *q, const ns_heads *k,
                     const void *q_weight, const void *k_weight, int32_t weight_dtype, float eps, const float *cos,
                     const float *sin, int64_t table_rows, int32_t rope_dim, int32_t interleaved, const void *pos,
                     int32_t pos_bytes, int64_t pos_batch_stride, HeadCall *c) {
    c->es = dtype_bytes(dtype);
    if (!c->es) return fail(NS_ERR_DTYPE, "dtype %d is not NS_BF16 or NS_F32", dtype);
    if (!dtype_bytes(weight_dtype)) return fail(NS_ERR_DTYPE, "weight_dtype %d is not NS_BF16 or NS_F32", weight_dtype);
    if (batch < 0 || seq < 0) return fail(NS_ERR_INVALID_ARG, "batch and seq must be >= 0");
    if (too_far(batch, seq) || batch * seq >= int64_t(1) << 31)
        return fail(NS_ERR_OVERFLOW, "batch x seq does not fit in 31 bits");
    if (head_dim < 1 || head_dim > kMaxHeadDim)
        return fail(NS_ERR_INVALID_ARG, "head_dim = %d outside [1, %d]", head_dim, kMaxHeadDim);
    if (rope_dim < 0 || rope_dim > head_dim || rope_dim % 2)
        return fail(NS_ERR_INVALID_ARG, "rope_dim = %d must be even and within [0, head_dim]", rope_dim);
    if (!(eps >= 0.f) || eps > 3.4e38f) return fail(NS_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (interleaved != 0 && interleaved != 1) return fail(NS_ERR_INVALID_ARG, "interleaved must be 0 or 1");
    if (ns_status s = check_heads("q", q, batch, seq, head_dim, c->es, -1)) return s;
    if (ns_status s = check_heads("k", k, batch, seq, head_dim, c->es, -1)) return s;
    if (misaligned(q_weight, dtype_bytes(weight_dtype)) || misaligned(k_weight, dtype_bytes(weight_dtype)))
        return fail(NS_ERR_INVALID_ARG, "weights not aligned to their type");
    if (rope_dim > 0) {
        if (table_rows < 0) return fail(NS_ERR_INVALID_ARG, "table_rows < 0");
        if (table_rows > 0 && (!cos || !sin)) return fail(NS_ERR_INVALID_ARG, "cos and sin are required");
        if (misaligned(cos, 4) || misaligned(sin, 4)) return fail(NS_ERR_INVALID_ARG, "cos / sin not 4-byte aligned");
        if (too_far(table_rows, 4 * (int64_t)rope_dim)) return fail(NS_ERR_OVERFLOW, "the angle table overflows");
        if (pos) {
            if (pos_bytes != 4 && pos_bytes != 8) return fail(NS_ERR_DTYPE, "pos_bytes = %d (must be 4 or 8)", pos_bytes);
            if (misaligned(pos, pos_bytes)) return fail(NS_ERR_INVALID_ARG, "pos not %d-byte aligned", pos_bytes);
            if (pos_batch_stride < 0) return fail(NS_ERR_INVALID_ARG, "pos_batch_stride < 0");
            if (too_far(batch, pos_batch_stride) || too_far(seq, 8)) return fail(NS_ERR_OVERFLOW, "pos overflows");
        }
    }
    HeadArgs &a = c->a;
    a = HeadArgs{};
    a.seq = (uint32_t)seq;
    a.tokens = (uint32_t)(batch * seq);
    a.D = head_dim;
    a.R = rope_dim;
    a.interleaved = interleaved;
    a.w_f32 = weight_dtype == NS_F32;
    a.eps = eps;
    a.cos = cos;
    a.sin = sin;
    a.table_rows = table_rows;
    a.pos = rope_dim > 0 ? pos : nullptr;
    a.pos_bytes = pos_bytes;
    a.pos_bs = pos_batch_stride;
    const ns_heads *hs[2] = {q, k};
    const void *ws[2] = {q_weight, k_weight};
    for (int i = 0; i < 2; ++i) {
        a.x[i] = operand(hs[i]);
        a.heads[i] = hs[i]->heads;
        a.w[i] = ws[i];
    }
    // The rotated half and the rest have to split into whole pieces.
    c->vec = (rope_dim | head_dim) % 16 == 0 ? 8 : (rope_dim | head_dim) % 8 == 0 && head_dim <= 512 ? 4 : 1;
    const int v = c->vec;
    a.RP = rope_dim / 2 / v;
    a.P = a.RP + (head_dim - rope_dim + 2 * v - 1) / (2 * v);
    const int np = v == 1 ? 8 : 1;   // pairs of pieces per lane
    a.lg = 0;
    while ((np << a.lg) < a.P) ++a.lg;
    return NS_OK;
}

// Deals the work: a wave for each (token, chunk of heads), or several tokens of
// one chunk a wave.
void deal(HeadCall &c, bool backward) {
    HeadArgs &a = c.a;
    const int64_t heads = (int64_t)a.heads[0] + a.heads[1], per = 64 >> a.lg;
    c.past_cache = (double)a.tokens * heads * a.D * c.es * (backward ? 3 : 2) > (double)kMallBytes;
    a.chunks = (uint32_t)((heads + per - 1) / per);
    const int64_t full = ((int64_t)a.tokens * a.chunks + kWaves - 1) / kWaves, least = (a.chunks + kWaves - 1) / kWaves;
    a.blocks = (int32_t)std::min(full, std::max<int64_t>(blocks_for(c.vec, backward), least));
    if (!a.blocks) return;
    a.stride = (uint32_t)((int64_t)a.blocks * kWaves / a.chunks);
    a.step_i = a.stride / a.seq;
    a.step_s = a.stride % a.seq;
}

template <bool BWD> ns_status launch(const HeadCall &c, int32_t dtype, void *stream) {
    if (!c.a.blocks) return NS_OK;
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(c.a.blocks), dim3(kThreads), 0, as_stream(stream), c.a); };
    auto pick = [&](auto t) {
        typedef decltype(t) T;
        if (c.vec == 8) c.past_cache ? go(qk_kernel<T, 8, 1, BWD, true>) : go(qk_kernel<T, 8, 1, BWD, false>);
        else if (c.vec == 4) go(qk_kernel<T, 4, 1, BWD, false>);
        else go(qk_kernel<T, 1, 8, BWD, false>);
    };
    if (dtype == NS_BF16) pick((__bf16)0.f);
    else pick(0.f);
    NSQ_HIP(hipGetLastError());
    return NS_OK;
}

}  // namespace
}  // namespace nsq

using namespace nsq;

extern "C" ns_status ns_qk_norm_rope(int64_t batch, int64_t seq, int32_t head_dim, ns_dtype dtype, const ns_heads *q,
                                     const ns_heads *k, const void *q_weight, const void *k_weight,
                                     ns_dtype weight_dtype, float eps, const float *cos, const float *sin,
                                     int64_t table_rows, int32_t rope_dim, int32_t interleaved, const void *pos,
                                     int32_t pos_bytes, int64_t pos_batch_stride, const ns_heads *q_out,
                                     const ns_heads *k_out, void *stream) {
    HeadCall c;
    if (ns_status s = plan_heads(batch, seq, head_dim, dtype, q, k, q_weight, k_weight, weight_dtype, eps, cos, sin,
                                 table_rows, rope_dim, interleaved, pos, pos_bytes, pos_batch_stride, &c))
        return s;
    if (ns_status s = check_heads("q_out", q_out, batch, seq, head_dim, c.es, q->heads, true)) return s;
    if (ns_status s = check_heads("k_out", k_out, batch, seq, head_dim, c.es, k->heads, true)) return s;
    c.a.y[0] = operand(q_out);
    c.a.y[1] = operand(k_out);
    deal(c, false);
    return launch<false>(c, dtype, stream);
}

extern "C" ns_status ns_qk_norm_rope_workspace_bytes(int64_t batch, int64_t seq, int32_t head_dim, size_t *bytes) {
    if (!bytes) return fail(NS_ERR_INVALID_ARG, "bytes is NULL");
    if (batch < 0 || seq < 0) return fail(NS_ERR_INVALID_ARG, "batch and seq must be >= 0");
    if (too_far(batch, seq) || batch * seq >= int64_t(1) << 31)
        return fail(NS_ERR_OVERFLOW, "batch x seq does not fit in 31 bits");
    if (head_dim < 1 || head_dim > kMaxHeadDim)
        return fail(NS_ERR_INVALID_ARG, "head_dim = %d outside [1, %d]", head_dim, kMaxHeadDim);
    static_assert(2 * kMaxHeads / kWaves <= kMostPartials, "a wave for every chunk of heads");
    *bytes = (size_t)kMostPartials * 2 * head_dim * sizeof(float);
    return NS_OK;
}

extern "C" ns_status ns_qk_norm_rope_backward(int64_t batch, int64_t seq, int32_t head_dim, ns_dtype dtype,
                                              const ns_heads *q, const ns_heads *k, const ns_heads *dq_out,
                                              const ns_heads *dk_out, const void *q_weight, const void *k_weight,
                                              ns_dtype weight_dtype, float eps, const float *cos, const float *sin,
                                              int64_t table_rows, int32_t rope_dim, int32_t interleaved,
                                              const void *pos, int32_t pos_bytes, int64_t pos_batch_stride,
                                              const ns_heads *dq, const ns_heads *dk, float *dq_weight,
                                              float *dk_weight, void *workspace, size_t workspace_bytes,
                                              void *stream) {
    HeadCall c;
    if (ns_status s = plan_heads(batch, seq, head_dim, dtype, q, k, q_weight, k_weight, weight_dtype, eps, cos, sin,
                                 table_rows, rope_dim, interleaved, pos, pos_bytes, pos_batch_stride, &c))
        return s;
    if (ns_status s = check_heads("dq_out", dq_out, batch, seq, head_dim, c.es, q->heads)) return s;
    if (ns_status s = check_heads("dk_out", dk_out, batch, seq, head_dim, c.es, k->heads)) return s;
    if (ns_status s = check_heads("dq", dq, batch, seq, head_dim, c.es, q->heads, true)) return s;
    if (ns_status s = check_heads("dk", dk, batch, seq, head_dim, c.es, k->heads, true)) return s;
    if (misaligned(dq_weight, 4) || misaligned(dk_weight, 4))
        return fail(NS_ERR_INVALID_ARG, "dq_weight / dk_weight not 4-byte aligned");
    const bool weights = dq_weight || dk_weight;
    if (weights) {
        size_t need;
        ns_qk_norm_rope_workspace_bytes(batch, seq, head_dim, &need);
        if (!workspace || workspace_bytes < need)
            return fail(NS_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : 0, need);
        if (misaligned(workspace, 256)) return fail(NS_ERR_INVALID_ARG, "workspace not 256-byte aligned");
    }
    c.a.g[0] = operand(dq_out);
    c.a.g[1] = operand(dk_out);
    c.a.y[0] = operand(dq);
    c.a.y[1] = operand(dk);
    c.a.dw[0] = dq_weight;
    c.a.dw[1] = dk_weight;
    c.a.partial = reinterpret_cast<float *>(workspace);
    deal(c, true);
    if (ns_status s = launch<true>(c, dtype, stream)) return s;
    if (weights) {
        hipLaunchKernelGGL(qk_join_kernel, dim3((head_dim + kJoinCols - 1) / kJoinCols, 2), dim3(kJoinCols * kJoinRows), 0,
                           as_stream(stream), c.a);
        NSQ_HIP(hipGetLastError());
    }
    return NS_OK;
}
