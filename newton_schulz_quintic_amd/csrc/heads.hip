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
// 16-byte pieces of it that the rotation pairs up (pieces at 8i and 8i + R/2 of
// bf16, or two neighbours for (2i, 2i + 1) pairs), so a rotation needs no other
// lane and the sums need log2 G exchanges. A wave holds 64 / G heads of one
// token at a time and takes U such rounds with all their loads in flight. Heads
// whose size or rotated part does not split into such pieces take the same code
// with pieces of one element (VEC = 1).
//
// Bound by memory: each input is read once and each output written once.

#include <type_traits>

#include "op_util.h"

namespace nsq {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxHeadDim = 1024;
constexpr int64_t kMaxGrid = 1 << 20;
// Backward: partial sums of the weights' gradients, one row of 2 D values per workgroup.
constexpr int kMaxPartials = 1024;

struct HeadSet {
    char *x, *g, *y;                 // input, gradient of the output (backward), output
    int64_t xb, xt, xh;              // element strides: batch, token, head
    int64_t gb, gt, gh;
    int64_t yb, yt, yh;
    const void *w;
    int32_t heads, chunks;           // chunks of (64 / G) U heads
    float *dw;
};

struct HeadArgs {
    HeadSet s[2];                    // queries, keys
    int64_t batch, seq, tokens;
    int32_t D, R, P, RP;             // head size, rotated part, pieces pairs per head, rotated ones
    int32_t lg;                      // log2 G
    int32_t interleaved, w_f32;
    float eps;
    const float *cos, *sin;
    int64_t table_rows;
    const void *pos;
    int32_t pos_bytes;
    int64_t pos_bs;
    float *partial;                  // backward: [gridDim.x][2][D]
};

// VEC elements at any element alignment, as one or two loads or stores.
template <typename T, int VEC> struct Piece {
    typedef typename std::conditional<sizeof(T) == 2, uint16_t, float>::type E;
    typedef E raw __attribute__((ext_vector_type(VEC)));
    typedef raw __attribute__((aligned(sizeof(T)))) raw_u;
    static __device__ inline void load(const T *p, float (&v)[VEC]) {
        if constexpr (VEC == 1) {
            v[0] = (float)p[0];
        } else {
            const raw r = *reinterpret_cast<const raw_u *>(p);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                if constexpr (sizeof(T) == 2) v[i] = __builtin_bit_cast(float, (uint32_t)r[i] << 16);
                else v[i] = r[i];
            }
        }
    }
    static __device__ inline void store(T *p, const float (&v)[VEC]) {
        if constexpr (VEC == 1) {
            p[0] = (T)v[0];
        } else {
            raw r;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                if constexpr (sizeof(T) == 2) r[i] = __builtin_bit_cast(uint16_t, (__bf16)v[i]);
                else r[i] = v[i];
            }
            *reinterpret_cast<raw_u *>(p) = r;
        }
    }
};

// A lane's two pieces of a head: element offsets a and b, and their angles' table offset.
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
    return p;
}

template <int VEC>
__device__ inline void load_weight(const HeadArgs &A, const HeadSet &S, const Place &p, float (&wa)[VEC],
                                   float (&wb)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) wa[i] = wb[i] = 1.f;
    if (!S.w || !p.in) return;
    if (A.w_f32) {
        Piece<float, VEC>::load(reinterpret_cast<const float *>(S.w) + p.a, wa);
        if (p.has_b) Piece<float, VEC>::load(reinterpret_cast<const float *>(S.w) + p.b, wb);
    } else {
        Piece<__bf16, VEC>::load(reinterpret_cast<const __bf16 *>(S.w) + p.a, wa);
        if (p.has_b) Piece<__bf16, VEC>::load(reinterpret_cast<const __bf16 *>(S.w) + p.b, wb);
    }
}

// cos and sin of the token's angles; NaN for a position outside the table.
template <int VEC>
__device__ inline void load_angles(const HeadArgs &A, int64_t b, int64_t s, const Place &p, float (&c)[VEC],
                                   float (&sn)[VEC]) {
    if (!p.turned) return;
    int64_t at = s;
    if (A.pos)
        at = A.pos_bytes == 8 ? reinterpret_cast<const int64_t *>(A.pos)[b * A.pos_bs + s]
                              : (int64_t) reinterpret_cast<const int32_t *>(A.pos)[b * A.pos_bs + s];
    if (at < 0 || at >= A.table_rows) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) c[i] = sn[i] = __builtin_nanf("");
        return;
    }
    const int64_t o = at * (A.R / 2) + p.angle;
    Piece<float, VEC>::load(A.cos + o, c);
    Piece<float, VEC>::load(A.sin + o, sn);
}

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

__device__ inline float group_sum(float v, int lg) {
    for (int m = 1 << lg >> 1; m; m >>= 1) v += __shfl_xor(v, m);
    return v;
}

// One item: the heads [h0, h0 + (64 / G) U) of one set at one token. BWD: the
// gradient; dwa / dwb collect the lane's pieces of dw.
template <typename T, int VEC, int NP, int U, bool BWD>
__device__ inline void head_item(const HeadArgs &A, const HeadSet &S, uint32_t token, int h0, const Place (&pl)[NP],
                                 const float (&wa)[NP][VEC], const float (&wb)[NP][VEC], float (&dwa)[NP][VEC],
                                 float (&dwb)[NP][VEC]) {
    const int lane = threadIdx.x & 63;
    const int per = 64 >> A.lg, sub = lane >> A.lg;
    const uint32_t bi = token / (uint32_t)A.seq, si = token - bi * (uint32_t)A.seq;
    const T *x = reinterpret_cast<const T *>(S.x) + bi * S.xb + si * S.xt;
    const T *g = BWD ? reinterpret_cast<const T *>(S.g) + bi * S.gb + si * S.gt : nullptr;
    T *y = reinterpret_cast<T *>(S.y) + bi * S.yb + si * S.yt;
    float c[NP][VEC], sn[NP][VEC];
#pragma unroll
    for (int n = 0; n < NP; ++n) load_angles<VEC>(A, bi, si, pl[n], c[n], sn[n]);
    float va[U][NP][VEC], vb[U][NP][VEC], ga[U][NP][VEC], gb[U][NP][VEC];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = h0 + u * per + sub;
#pragma unroll
        for (int n = 0; n < NP; ++n) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) va[u][n][i] = vb[u][n][i] = ga[u][n][i] = gb[u][n][i] = 0.f;
            if (h < S.heads && pl[n].in) {
                Piece<T, VEC>::load(x + h * S.xh + pl[n].a, va[u][n]);
                if (pl[n].has_b) Piece<T, VEC>::load(x + h * S.xh + pl[n].b, vb[u][n]);
                if constexpr (BWD) {
                    Piece<T, VEC>::load(g + h * S.gh + pl[n].a, ga[u][n]);
                    if (pl[n].has_b) Piece<T, VEC>::load(g + h * S.gh + pl[n].b, gb[u][n]);
                }
            }
        }
    }
    const float inv_d = 1.f / (float)A.D;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = h0 + u * per + sub;
        float ss = 0.f, sd = 0.f;
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            if constexpr (BWD)
                if (pl[n].turned) turn<VEC>(A.interleaved, -1.f, ga[u][n], gb[u][n], c[n], sn[n]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                ss += va[u][n][i] * va[u][n][i] + vb[u][n][i] * vb[u][n][i];
                if constexpr (BWD)
                    sd += ga[u][n][i] * wa[n][i] * va[u][n][i] + gb[u][n][i] * wb[n][i] * vb[u][n][i];
            }
        }
        ss = group_sum(ss, A.lg);
        const float r = 1.f / sqrtf(ss * inv_d + A.eps);
        float m = 0.f;
        if constexpr (BWD) m = group_sum(sd, A.lg) * r * inv_d;   // mean(dn n)
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            if constexpr (BWD) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float na = va[u][n][i] * r, nb = vb[u][n][i] * r;
                    if (h < S.heads) {
                        dwa[n][i] += ga[u][n][i] * na;
                        dwb[n][i] += gb[u][n][i] * nb;
                    }
                    va[u][n][i] = r * (ga[u][n][i] * wa[n][i] - na * m);
                    vb[u][n][i] = r * (gb[u][n][i] * wb[n][i] - nb * m);
                }
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    va[u][n][i] = va[u][n][i] * r * wa[n][i];
                    vb[u][n][i] = vb[u][n][i] * r * wb[n][i];
                }
                if (pl[n].turned) turn<VEC>(A.interleaved, 1.f, va[u][n], vb[u][n], c[n], sn[n]);
            }
            if (h < S.heads && pl[n].in) {
                Piece<T, VEC>::store(y + h * S.yh + pl[n].a, va[u][n]);
                if (pl[n].has_b) Piece<T, VEC>::store(y + h * S.yh + pl[n].b, vb[u][n]);
            }
        }
    }
}

// Items are (token, chunk of heads), a wave each: the query chunks of a token,
// then its key chunks, then the next token's.
template <typename T, int VEC, int NP, int U>
__global__ __launch_bounds__(kThreads) void qk_forward_kernel(HeadArgs A) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t chunks = A.s[0].chunks + A.s[1].chunks;
    const uint32_t items = (uint32_t)A.tokens * chunks;   // < 2^31
    Place pl[NP];
#pragma unroll
    for (int n = 0; n < NP; ++n) pl[n] = place_of<VEC>(A, (lane & ((1 << A.lg) - 1)) + (n << A.lg));
    float none[NP][VEC];
    for (uint32_t it = blockIdx.x * kWaves + wave; it < items; it += gridDim.x * kWaves) {
        const uint32_t token = it / chunks;
        const int ch = (int)(it - token * chunks);
        const bool key = ch >= A.s[0].chunks;
        const HeadSet S = key ? A.s[1] : A.s[0];
        float wa[NP][VEC], wb[NP][VEC];
#pragma unroll
        for (int n = 0; n < NP; ++n) load_weight<VEC>(A, S, pl[n], wa[n], wb[n]);
        head_item<T, VEC, NP, U, false>(A, S, token, (key ? ch - A.s[0].chunks : ch) * ((64 >> A.lg) * U), pl, wa, wb,
                                        none, none);
    }
}

// blockIdx.y: 0 queries, 1 keys. Each workgroup sums its part of dw in
// registers, joins its waves in a fixed order and writes one row of partials.
template <typename T, int VEC, int NP, int U>
__global__ __launch_bounds__(kThreads) void qk_backward_kernel(HeadArgs A) {
    __shared__ float lds[kWaves][2 * VEC * NP * 64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const HeadSet S = blockIdx.y ? A.s[1] : A.s[0];
    const uint32_t items = (uint32_t)A.tokens * S.chunks;   // < 2^31
    Place pl[NP];
    float wa[NP][VEC], wb[NP][VEC], dwa[NP][VEC], dwb[NP][VEC];
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        pl[n] = place_of<VEC>(A, (lane & ((1 << A.lg) - 1)) + (n << A.lg));
        load_weight<VEC>(A, S, pl[n], wa[n], wb[n]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) dwa[n][i] = dwb[n][i] = 0.f;
    }
    for (uint32_t it = blockIdx.x * kWaves + wave; it < items; it += gridDim.x * kWaves) {
        const uint32_t token = it / S.chunks;
        head_item<T, VEC, NP, U, true>(A, S, token, (int)(it - token * S.chunks) * ((64 >> A.lg) * U), pl, wa, wb, dwa,
                                       dwb);
    }
    if (!S.dw) return;
    // join the wave's head groups, then the waves
#pragma unroll
    for (int n = 0; n < NP; ++n)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            for (int m = 1 << A.lg; m < 64; m <<= 1) {
                dwa[n][i] += __shfl_xor(dwa[n][i], m);
                dwb[n][i] += __shfl_xor(dwb[n][i], m);
            }
            lds[wave][((n * VEC + i) * 2) * 64 + lane] = dwa[n][i];
            lds[wave][((n * VEC + i) * 2 + 1) * 64 + lane] = dwb[n][i];
        }
    __syncthreads();
    if (wave == 0 && lane < 1 << A.lg) {
        float *row = A.partial + ((int64_t)blockIdx.x * 2 + blockIdx.y) * A.D;
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            if (!pl[n].in) continue;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float a = 0.f, b = 0.f;
                for (int w = 0; w < kWaves; ++w) {
                    a += lds[w][((n * VEC + i) * 2) * 64 + lane];
                    b += lds[w][((n * VEC + i) * 2 + 1) * 64 + lane];
                }
                row[pl[n].a + i] = a;
                if (pl[n].has_b) row[pl[n].b + i] = b;
            }
        }
    }
}

// dw[j] = sum of the workgroups' partials: one wave per 4 values (16 bytes a
// row at most), 16 lanes down the rows each, joined in a fixed order.
__global__ __launch_bounds__(64) void qk_join_kernel(HeadArgs A, int32_t rows) {
    const int j = blockIdx.x * 4 + (threadIdx.x & 3), k = blockIdx.y;
    if (!A.s[k].dw) return;
    float sum = 0.f;
    if (j < A.D)
        for (int r = threadIdx.x >> 2; r < rows; r += 16) sum += A.partial[((int64_t)r * 2 + k) * A.D + j];
    for (int m = 4; m < 64; m <<= 1) sum += __shfl_xor(sum, m);
    if (threadIdx.x < 4 && j < A.D) A.s[k].dw[j] = sum;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// One head tensor's checks. `out`: whether it is written.
ns_status check_heads(const char *name, const ns_heads *h, int64_t batch, int64_t seq, int32_t D, int es,
                      int32_t want_heads) {
    if (!h) return fail(NS_ERR_INVALID_ARG, "%s is NULL", name);
    if (h->heads < 0) return fail(NS_ERR_INVALID_ARG, "%s: heads = %d < 0", name, h->heads);
    if (want_heads >= 0 && h->heads != want_heads)
        return fail(NS_ERR_INVALID_ARG, "%s has %d heads, not %d", name, h->heads, want_heads);
    if (h->heads == 0 || batch == 0 || seq == 0) return NS_OK;
    if (!h->data) return fail(NS_ERR_INVALID_ARG, "%s: data is NULL", name);
    if (misaligned(h->data, es)) return fail(NS_ERR_INVALID_ARG, "%s: data not %d-byte aligned", name, es);
    if (h->batch_stride < 0 || h->token_stride < 0 || h->head_stride < 0)
        return fail(NS_ERR_INVALID_ARG, "%s: negative stride", name);
    if (too_far(batch, h->batch_stride) || too_far(seq, h->token_stride) || too_far(h->heads, h->head_stride))
        return fail(NS_ERR_OVERFLOW, "%s: offsets overflow", name);
    if (batch * (double)h->batch_stride + seq * (double)h->token_stride + h->heads * (double)h->head_stride + D >
        4.6e18 / es)
        return fail(NS_ERR_OVERFLOW, "%s: offsets overflow", name);
    return NS_OK;
}

struct HeadCall {
    HeadArgs a;
    int vec;       // elements of a piece: 8, 4 or 1
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
    // Work items are (token, chunk of heads), at most one a head, counted in 31 bits.
    if (batch * seq * ((double)q->heads + k->heads) >= 2147483648.0)
        return fail(NS_ERR_OVERFLOW, "batch x seq x heads does not fit in 31 bits");
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
    a.batch = batch;
    a.seq = seq;
    a.tokens = batch * seq;
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
        HeadSet &s = a.s[i];
        s.x = (char *)hs[i]->data;
        s.xb = hs[i]->batch_stride;
        s.xt = hs[i]->token_stride;
        s.xh = hs[i]->head_stride;
        s.heads = hs[i]->heads;
        s.w = ws[i];
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

void set_out(HeadSet &s, const ns_heads *o) {
    s.y = (char *)o->data;
    s.yb = o->batch_stride;
    s.yt = o->token_stride;
    s.yh = o->head_stride;
}

void set_chunks(HeadArgs &a, int U) {
    const int per = (64 >> a.lg) * U;
    for (HeadSet &s : a.s) s.chunks = (s.heads + per - 1) / per;
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
    if (ns_status s = check_heads("q_out", q_out, batch, seq, head_dim, c.es, q->heads)) return s;
    if (ns_status s = check_heads("k_out", k_out, batch, seq, head_dim, c.es, k->heads)) return s;
    set_out(c.a.s[0], q_out);
    set_out(c.a.s[1], k_out);
    if (c.a.tokens == 0 || q->heads + k->heads == 0) return NS_OK;
    constexpr int U = 1;
    set_chunks(c.a, U);
    const int64_t items = c.a.tokens * (c.a.s[0].chunks + c.a.s[1].chunks);
    const int64_t blocks = (items + kWaves - 1) / kWaves;
    const dim3 grid((unsigned)(blocks < kMaxGrid ? blocks : kMaxGrid));
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, as_stream(stream), c.a); };
    auto pick = [&](auto t) {
        typedef decltype(t) T;
        if (c.vec == 8) go(qk_forward_kernel<T, 8, 1, U>);
        else if (c.vec == 4) go(qk_forward_kernel<T, 4, 1, U>);
        else go(qk_forward_kernel<T, 1, 8, U>);
    };
    if (dtype == NS_BF16) pick((__bf16)0.f);
    else pick(0.f);
    NSQ_HIP(hipGetLastError());
    return NS_OK;
}

extern "C" ns_status ns_qk_norm_rope_workspace_bytes(int64_t batch, int64_t seq, int32_t head_dim, size_t *bytes) {
    if (!bytes) return fail(NS_ERR_INVALID_ARG, "bytes is NULL");
    if (batch < 0 || seq < 0) return fail(NS_ERR_INVALID_ARG, "batch and seq must be >= 0");
    if (too_far(batch, seq) || batch * seq >= int64_t(1) << 31)
        return fail(NS_ERR_OVERFLOW, "batch x seq does not fit in 31 bits");
    if (head_dim < 1 || head_dim > kMaxHeadDim)
        return fail(NS_ERR_INVALID_ARG, "head_dim = %d outside [1, %d]", head_dim, kMaxHeadDim);
    *bytes = (size_t)kMaxPartials * 2 * head_dim * sizeof(float);
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
    if (ns_status s = check_heads("dq", dq, batch, seq, head_dim, c.es, q->heads)) return s;
    if (ns_status s = check_heads("dk", dk, batch, seq, head_dim, c.es, k->heads)) return s;
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
    const ns_heads *gs[2] = {dq_out, dk_out}, *os[2] = {dq, dk};
    float *dws[2] = {dq_weight, dk_weight};
    for (int i = 0; i < 2; ++i) {
        HeadSet &s = c.a.s[i];
        s.g = (char *)gs[i]->data;
        s.gb = gs[i]->batch_stride;
        s.gt = gs[i]->token_stride;
        s.gh = gs[i]->head_stride;
        set_out(s, os[i]);
        s.dw = dws[i];
    }
    c.a.partial = reinterpret_cast<float *>(workspace);
    constexpr int U = 1;
    set_chunks(c.a, U);
    // Every workgroup writes its row of both sets' partials, so with no tokens
    // or heads at all the join sums no rows and writes zeros.
    const int32_t most = c.a.s[0].chunks > c.a.s[1].chunks ? c.a.s[0].chunks : c.a.s[1].chunks;
    const int64_t items = c.a.tokens * most;
    const int64_t blocks = (items + kWaves - 1) / kWaves, cap = weights ? kMaxPartials : kMaxGrid;
    const int32_t rows = (int32_t)(blocks < cap ? blocks : cap);
    if (rows > 0) {
        const dim3 grid(rows, 2);
        auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, as_stream(stream), c.a); };
        auto pick = [&](auto t) {
            typedef decltype(t) T;
            if (c.vec == 8) go(qk_backward_kernel<T, 8, 1, U>);
            else if (c.vec == 4) go(qk_backward_kernel<T, 4, 1, U>);
            else go(qk_backward_kernel<T, 1, 8, U>);
        };
        if (dtype == NS_BF16) pick((__bf16)0.f);
        else pick(0.f);
        NSQ_HIP(hipGetLastError());
    }
    if (weights) {
        hipLaunchKernelGGL(qk_join_kernel, dim3((head_dim + 3) / 4, 2), dim3(64), 0, as_stream(stream), c.a, rows);
        NSQ_HIP(hipGetLastError());
    }
    return NS_OK;
}
