// The norms before and after a block of a transformer with its gate and residual
// scale, in one pass, and their gradient. For one row, with x the residual and y
// the block's output:
//   ry = 1 / sqrt(mean(y^2) + eps),  u = y ry (or y),  z = u w_post,
//   r = alpha x + scale gate z                      the new residual
//   rr = 1 / sqrt(mean(r^2) + eps),  h = r rr w_pre     what the next block reads
// Backward, from the gradients g of r and dh of h, with n = r rr:
//   dn = dh w_pre,  dr = g + rr (dn - n mean(dn n)),  dx = alpha dr,
//   a = scale dr,  dw_pre = sum dh n,  dgate = sum a u w_post,  dw_post = sum a gate u,
//   du = a gate w_post,  dy = ry (du - u mean(du u))   (or du).
// Backward computes r again from x and y, so that nothing has to be saved and
// the norm that it differentiates is the forward's own, before r was rounded.
//
// Layout: a team of W waves holds a row, E elements a lane in pieces of V (16
// bytes of the narrower tensors' partner), and walks over a run of rows with the
// next row's loads under way; weights stay in registers. A width that is no
// multiple of V takes its last piece from the row's end, where it overlaps the one
// before; overlapped elements count once. Sums over rows (weights, gates) stay in
// registers and leave as one partial row a team; a second launch adds those.
//
// Bound by memory: each input is read once and each output written once. 16384 rows
// of 4096 bf16 with a gate and both norms: forward 100 us (537 MB, 5.4 TB/s), backward
// 171 us (805 MB, 4.7 TB/s; 5 us of it the second launch). The non-temporal hint
// changed neither. 16 rows: 4.2 us, a launch and two chains of load, sum and barrier.
// Backward, whose forms were settled at 4096, keeps less under way at other widths:
// 16384 x 1024 52 us (3.9 TB/s), x 2141 222 (1.9), x 2560 146 (3.5), x 5120 253 (4.0).

#include <algorithm>

#include "elems.h"

namespace nsq {
namespace {

constexpr int kMaxHidden = 16384;
constexpr int kMaxEmptyGates = 65533;   // gate rows of a call without rows, whose gradients are only cleared
// The most teams of a launch, for teams of one wave, of four and more waves. Backward: one round of workgroups, whose
// partial rows are few to add (16384 x 4096 bf16 173 us; half as many 272, twice as many 178). Forward: several rounds,
// so that one's stores go out under another's loads (16384 x 4096 bf16 with half as many 109, 106, with twice as many
// 111 us; 8192 x 4096 fp32 129, 120, 115).
constexpr int teams_for(int waves, bool backward) {
    return backward ? (waves == 1 ? 1024 : waves == 4 ? 512 : 256) : (waves == 1 ? 32768 : waves == 4 ? 8192 : 4096);
}

struct Rows {
    char *p;
    int64_t ld;
};

struct BlockArgs {
    Rows x, y, gate, x_out, h;         // forward; backward: x_out and h hold the gradients of those outputs
    Rows dx, dy, dgate;
    const void *w_post, *w_pre;
    float *dw_post, *dw_pre;
    float *partial;                    // [team][sets][hidden]: sums of dh n; of a u (many gate rows: gate a u); of a u
    int64_t rows, gate_span;           // rows of one gate row
    int32_t hidden, teams;
    int32_t per, gate_teams;           // rows of a team; teams of one gate row (1: a team has whole gate rows)
    int32_t post_norm, w_f32, gate_f32, has_y, has_gate, many_gates;
    int32_t join_u, sets, whole_gates; // the second partial row is wanted; partial rows of a team; a team has whole gate rows and writes their gradients itself
    float alpha, scale, eps, inv_hidden;
};

template <typename TX, typename TY, int V_, int W_, int E_> struct Form {
    typedef TX X;
    typedef TY Y;
    static constexpr int V = V_, W = W_, E = E_, NP = E / V, LANES = 64 * W;
    static constexpr int THREADS = W < 4 ? 256 : 64 * W, PER_GROUP = THREADS / LANES;   // teams of a workgroup
    typedef typename Elems<TX, V>::raw RX;
    typedef typename Elems<TY, V>::raw RY;
};

// A lane's pieces of a row: where they start and how many of their first elements
// belong to another piece (V: the lane has no such piece).
template <class F> struct Pieces {
    int at[F::NP], skip[F::NP];
    __device__ inline Pieces(int hidden, int lane) {
#pragma unroll
        for (int p = 0; p < F::NP; ++p) {
            const int i = (p * F::LANES + lane) * F::V;
            at[p] = min(i, hidden - F::V);
            skip[p] = min(i - at[p], F::V);
        }
    }
    __device__ inline bool has(int p) const { return skip[p] < F::V; }
};

// Weights or a gate row as fp32, ones if absent.
template <class F>
__device__ inline void load_row(const void *p, int f32, const Pieces<F> &pc, float (&v)[F::NP][F::V]) {
#pragma unroll
    for (int i = 0; i < F::NP; ++i) {
        if (!p) {
#pragma unroll
            for (int k = 0; k < F::V; ++k) v[i][k] = 1.f;
        } else if (f32) {
            if constexpr (F::V == 8) {
                float lo[4], hi[4];
                Elems<float, 4>::widen(Elems<float, 4>::load(reinterpret_cast<const float *>(p) + pc.at[i]), lo);
                Elems<float, 4>::widen(Elems<float, 4>::load(reinterpret_cast<const float *>(p) + pc.at[i] + 4), hi);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[i][k] = lo[k], v[i][4 + k] = hi[k];
            } else {
                Elems<float, F::V>::widen(Elems<float, F::V>::load(reinterpret_cast<const float *>(p) + pc.at[i]), v[i]);
            }
        } else {
            Elems<__bf16, F::V>::widen(Elems<__bf16, F::V>::load(reinterpret_cast<const __bf16 *>(p) + pc.at[i]), v[i]);
        }
    }
}

template <class F, typename T, typename R>
__device__ inline void load_raw(const Rows &t, int64_t row, const Pieces<F> &pc, R (&v)[F::NP]) {
    const T *p = reinterpret_cast<const T *>(t.p) + row * t.ld;
#pragma unroll
    for (int i = 0; i < F::NP; ++i) v[i] = Elems<T, F::V>::load(p + pc.at[i]);
}

template <class F, typename T>
__device__ inline void store_row(const Rows &t, int64_t row, const Pieces<F> &pc, const float (&v)[F::NP][F::V]) {
    T *p = reinterpret_cast<T *>(t.p) + row * t.ld;
#pragma unroll
    for (int i = 0; i < F::NP; ++i) {
        if (pc.skip[i] == 0) {
            Elems<T, F::V>::store(p + pc.at[i], v[i]);
        } else if (pc.has(i)) {   // in place, overlapped elements may have been read after their own lane wrote them
#pragma unroll
            for (int k = 1; k < F::V; ++k)
                if (k >= pc.skip[i]) p[pc.at[i] + k] = (T)v[i][k];
        }
    }
}

// Sums over a team. Each call of a row has a place of its own in LDS, so that one barrier a call is enough.
template <class F>
__device__ inline float team_sum(float v, float (*lds)[16], int which) {
    v = wave_sum(v);
    if constexpr (F::W > 1) {
        if ((threadIdx.x & 63) == 0) lds[which][threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < F::W; ++i) v += lds[which][i];
    }
    return v;
}

// The rows of a team: first, end.
__device__ inline void rows_of(const BlockArgs &a, int team, int64_t *first, int64_t *end) {
    if (a.gate_teams > 1) {   // several teams to a gate row
        const int64_t g = team / a.gate_teams, k = team % a.gate_teams;
        *first = g * a.gate_span + min(k * a.per, a.gate_span);
        *end = g * a.gate_span + min((k + 1) * (int64_t)a.per, a.gate_span);
    } else {
        *first = min((int64_t)team * a.per, a.rows);
        *end = min(*first + a.per, a.rows);
    }
}

#define NSQ_EACH(i, k) \
    _Pragma("unroll") for (int i = 0; i < F::NP; ++i) _Pragma("unroll") for (int k = 0; k < F::V; ++k)

template <class F, bool HAS_Y>
__global__ __launch_bounds__(F::THREADS) void block_norm_kernel(BlockArgs a) {
    typedef typename F::X X;
    typedef typename F::Y Y;
    typedef Elems<X, F::V> EX;
    typedef Elems<Y, F::V> EY;
    __shared__ float lds[4][16];
    const int lane = threadIdx.x % F::LANES;
    const int team = __builtin_amdgcn_readfirstlane(blockIdx.x * F::PER_GROUP + threadIdx.x / F::LANES);
    if (team >= a.teams) return;
    int64_t row, end;
    rows_of(a, team, &row, &end);
    if (row >= end) return;
    const Pieces<F> pc(a.hidden, lane);
    float wn[F::NP][F::V], wp[F::NP][F::V], gate[F::NP][F::V];
    load_row<F>(a.w_pre, a.w_f32, pc, wn);
    if (HAS_Y) load_row<F>(a.w_post, a.w_f32, pc, wp);
    const int gate_size = a.gate_f32 ? 4 : 2;
    const auto gate_at = [&](int64_t g) { return a.has_gate ? a.gate.p + g * a.gate.ld * gate_size : nullptr; };
    int64_t g = HAS_Y && a.many_gates ? row / a.gate_span : 0;
    int64_t left = a.many_gates ? (g + 1) * a.gate_span - row : INT64_MAX;   // rows until the next gate row
    if (HAS_Y) {
        load_row<F>(gate_at(g), a.gate_f32, pc, gate);
        NSQ_EACH(i, k) gate[i][k] *= a.scale;
    }
    typename F::RX x[F::NP];
    typename F::RY y[F::NP];
    load_raw<F, X>(a.x, row, pc, x);
    if (HAS_Y) load_raw<F, Y>(a.y, row, pc, y);
    for (int odd = 0;; odd ^= 2) {
        float r[F::NP][F::V], z[F::NP][F::V];
        NSQ_EACH(i, k) r[i][k] = a.alpha * EX::at(x[i], k);
        if (HAS_Y) {
            NSQ_EACH(i, k) z[i][k] = EY::at(y[i], k);
        }
        const int64_t next = row + 1;
        if (next < end) {
            load_raw<F, X>(a.x, next, pc, x);
            if (HAS_Y) load_raw<F, Y>(a.y, next, pc, y);
        }
        if (HAS_Y) {
            float ry = 1.f;
            if (a.post_norm) {
                float s = 0.f;
                NSQ_EACH(i, k) s = k >= pc.skip[i] ? fmaf(z[i][k], z[i][k], s) : s;
                s = team_sum<F>(s, lds, odd);
                ry = 1.f / sqrtf(s * a.inv_hidden + a.eps);
            }
            NSQ_EACH(i, k) r[i][k] = fmaf(gate[i][k], z[i][k] * ry * wp[i][k], r[i][k]);
            if (a.x_out.p) store_row<F, X>(a.x_out, row, pc, r);
        }
        if (a.h.p) {
            float s = 0.f;
            NSQ_EACH(i, k) s = k >= pc.skip[i] ? fmaf(r[i][k], r[i][k], s) : s;
            s = team_sum<F>(s, lds, odd + 1);
            const float rr = 1.f / sqrtf(s * a.inv_hidden + a.eps);
            NSQ_EACH(i, k) r[i][k] = r[i][k] * rr * wn[i][k];
            store_row<F, Y>(a.h, row, pc, r);
        }
        if (next >= end) return;
        row = next;
        if (HAS_Y && --left == 0) {
            load_row<F>(gate_at(++g), a.gate_f32, pc, gate);
            NSQ_EACH(i, k) gate[i][k] *= a.scale;
            left = a.gate_span;
        }
    }
}

template <class F>
__device__ inline void store_partial(const BlockArgs &a, int team, int set, const Pieces<F> &pc, const float (&v)[F::NP][F::V]) {
    float *to = a.partial + ((int64_t)team * a.sets + set) * a.hidden;
    NSQ_EACH(i, k) if (k >= pc.skip[i]) to[pc.at[i] + k] = v[i][k];
}

template <class F, bool HAS_Y>
__global__ __launch_bounds__(F::THREADS) void block_norm_backward_kernel(BlockArgs a) {
    typedef typename F::X X;
    typedef typename F::Y Y;
    typedef Elems<X, F::V> EX;
    typedef Elems<Y, F::V> EY;
    __shared__ float lds[8][16];
    const int lane = threadIdx.x % F::LANES;
    const int team = __builtin_amdgcn_readfirstlane(blockIdx.x * F::PER_GROUP + threadIdx.x / F::LANES);
    if (team >= a.teams) return;
    int64_t row, end;
    rows_of(a, team, &row, &end);
    const Pieces<F> pc(a.hidden, lane);
    float wn[F::NP][F::V], wp[F::NP][F::V], gate[F::NP][F::V];
    float sum_pre[F::NP][F::V], sum_post[F::NP][F::V], sum_gate[F::NP][F::V];   // of dh n; of gate a u, finished gate rows; of a u
    NSQ_EACH(i, k) sum_pre[i][k] = sum_post[i][k] = sum_gate[i][k] = 0.f;
    load_row<F>(a.w_pre, a.w_f32, pc, wn);
    if (HAS_Y) load_row<F>(a.w_post, a.w_f32, pc, wp);
    const int gate_size = a.gate_f32 ? 4 : 2;
    const auto gate_at = [&](int64_t g) { return a.has_gate ? a.gate.p + g * a.gate.ld * gate_size : nullptr; };
    int64_t g = HAS_Y && a.many_gates && row < end ? row / a.gate_span : 0;
    int64_t left = a.many_gates ? (g + 1) * a.gate_span - row : INT64_MAX;
    if (HAS_Y) load_row<F>(gate_at(g), a.gate_f32, pc, gate);
    typename F::RX x[F::NP], gx[F::NP];
    typename F::RY y[F::NP], gh[F::NP];
    const auto load_all = [&](int64_t at) {
        load_raw<F, X>(a.x, at, pc, x);
        if (HAS_Y) load_raw<F, Y>(a.y, at, pc, y);
        if (a.x_out.p) load_raw<F, X>(a.x_out, at, pc, gx);
        if (a.h.p) load_raw<F, Y>(a.h, at, pc, gh);
    };
    if (row < end) load_all(row);
    for (int odd = 0; row < end; odd ^= 4) {
        float r[F::NP][F::V], u[F::NP][F::V], dr[F::NP][F::V], dn[F::NP][F::V];
        NSQ_EACH(i, k) {
            r[i][k] = a.alpha * EX::at(x[i], k);
            u[i][k] = HAS_Y ? EY::at(y[i], k) : 0.f;
            dr[i][k] = a.x_out.p ? EX::at(gx[i], k) : 0.f;
            dn[i][k] = a.h.p ? EY::at(gh[i], k) : 0.f;
        }
        if (row + 1 < end) load_all(row + 1);
        float ry = 1.f;
        if (HAS_Y) {
            if (a.post_norm) {
                float s = 0.f;
                NSQ_EACH(i, k) s = k >= pc.skip[i] ? fmaf(u[i][k], u[i][k], s) : s;
                s = team_sum<F>(s, lds, odd);
                ry = 1.f / sqrtf(s * a.inv_hidden + a.eps);
                NSQ_EACH(i, k) u[i][k] *= ry;
            }
            NSQ_EACH(i, k) r[i][k] = fmaf(a.scale * gate[i][k], u[i][k] * wp[i][k], r[i][k]);
        }
        if (a.h.p) {
            float s = 0.f, t = 0.f;
            NSQ_EACH(i, k) {
                s = k >= pc.skip[i] ? fmaf(r[i][k], r[i][k], s) : s;
                t = k >= pc.skip[i] ? fmaf(dn[i][k] * wn[i][k], r[i][k], t) : t;
            }
            s = team_sum<F>(s, lds, odd + 1);
            t = team_sum<F>(t, lds, odd + 2);
            const float rr = 1.f / sqrtf(s * a.inv_hidden + a.eps);
            const float mean = t * rr * a.inv_hidden;   // of dn n
            NSQ_EACH(i, k) {
                const float n = r[i][k] * rr;
                sum_pre[i][k] = fmaf(dn[i][k], n, sum_pre[i][k]);
                dr[i][k] += rr * (dn[i][k] * wn[i][k] - n * mean);
            }
        }
        if (HAS_Y) {
            float du[F::NP][F::V], s = 0.f;
            NSQ_EACH(i, k) {
                const float b = a.scale * dr[i][k];
                sum_gate[i][k] = fmaf(b, u[i][k], sum_gate[i][k]);
                du[i][k] = b * gate[i][k] * wp[i][k];
                s = k >= pc.skip[i] ? fmaf(du[i][k], u[i][k], s) : s;
            }
            if (a.post_norm) {
                s = team_sum<F>(s, lds, odd + 3) * a.inv_hidden;
                NSQ_EACH(i, k) du[i][k] = ry * (du[i][k] - u[i][k] * s);
            }
            if (a.dy.p) store_row<F, Y>(a.dy, row, pc, du);
        }
        NSQ_EACH(i, k) dr[i][k] *= a.alpha;
        if (a.dx.p) store_row<F, X>(a.dx, row, pc, dr);
        ++row;
        if (HAS_Y && (--left == 0 || row == end)) {   // the gate row, or this team's part of it, ends
            NSQ_EACH(i, k) sum_post[i][k] = fmaf(gate[i][k], sum_gate[i][k], sum_post[i][k]);
            if (a.dgate.p && a.whole_gates) {
                NSQ_EACH(i, k) sum_gate[i][k] *= wp[i][k];
                if (a.gate_f32) {
                    float *to = reinterpret_cast<float *>(a.dgate.p) + g * a.dgate.ld;
                    NSQ_EACH(i, k) if (k >= pc.skip[i]) to[pc.at[i] + k] = sum_gate[i][k];
                } else {
                    const Rows to = {a.dgate.p, a.dgate.ld};
                    store_row<F, __bf16>(to, g, pc, sum_gate);
                }
            }
            if (row < end) {
                NSQ_EACH(i, k) sum_gate[i][k] = 0.f;
                load_row<F>(gate_at(++g), a.gate_f32, pc, gate);
                left = a.gate_span;
            }
        }
    }
    if (a.dw_pre) store_partial<F>(a, team, 0, pc, sum_pre);
    if (HAS_Y && a.join_u) store_partial<F>(a, team, 1, pc, a.many_gates ? sum_post : sum_gate);
    if (HAS_Y && a.sets == 3) store_partial<F>(a, team, 2, pc, sum_gate);
}

// Adds the teams' partial rows: 32 columns a workgroup, 32 teams at a time. blockIdx.y
// 0: dw_pre. 1: dw_post, from the sums of gate a u or, with a single gate row, of a u;
// and that gate row's gradient. From 2 on: the gate rows' gradients, from their teams.
constexpr int kJoinCols = 32, kJoinRows = 32;
__device__ inline float value_at(const void *p, int f32, int64_t i) {
    return f32 ? reinterpret_cast<const float *>(p)[i] : (float)reinterpret_cast<const __bf16 *>(p)[i];
}
__global__ __launch_bounds__(kJoinCols * kJoinRows) void block_norm_join_kernel(BlockArgs a) {
    __shared__ float part[kJoinRows][kJoinCols];
    const int col = threadIdx.x % kJoinCols, down = threadIdx.x / kJoinCols, j = blockIdx.x * kJoinCols + col;
    const int set = min((int)blockIdx.y, 2), gate_row = blockIdx.y < 2 ? 0 : (int)blockIdx.y - 2;
    if (set == 0 && !a.dw_pre) return;
    const int from = set == 2 ? gate_row * a.gate_teams : 0, to = min(set == 2 ? from + a.gate_teams : a.teams, a.teams);
    float sum = 0.f;
    if (j < a.hidden) {
        const float *p = a.partial + (int64_t)set * a.hidden + j;
        const int64_t ld = (int64_t)a.sets * a.hidden;
#pragma unroll 8
        for (int r = from + down; r < to; r += kJoinRows) sum += p[r * ld];
    }
    part[down][col] = sum;
    __syncthreads();
    if (down != 0 || j >= a.hidden) return;
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kJoinRows; ++i) sum += part[i][col];
    float sum_gate = sum;
    // without rows a gate that is counted may have no address: its sums are zeros as they are
    if (set == 1 && a.gate.p && !a.many_gates) sum *= value_at(a.gate.p, a.gate_f32, j);
    if (blockIdx.y == 0) a.dw_pre[j] = sum;
    if (blockIdx.y == 1 && a.dw_post) a.dw_post[j] = sum;
    if (blockIdx.y >= 2 || (blockIdx.y == 1 && a.dgate.p && !a.many_gates)) {
        if (a.w_post) sum_gate *= value_at(a.w_post, a.w_f32, j);
        if (a.gate_f32) reinterpret_cast<float *>(a.dgate.p)[gate_row * a.dgate.ld + j] = sum_gate;
        else reinterpret_cast<__bf16 *>(a.dgate.p)[gate_row * a.dgate.ld + j] = (__bf16)sum_gate;
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

Rows rows_at(const ns_rows *t) { return t && t->data ? Rows{(char *)t->data, t->ld} : Rows{nullptr, 0}; }

ns_status check_rows(const char *name, const ns_rows *t, int64_t rows, int32_t hidden, int es) {
    if (!t || !t->data || !rows) return NS_OK;
    if (misaligned(t->data, es)) return fail(NS_ERR_INVALID_ARG, "%s not %d-byte aligned", name, es);
    if (t->ld < hidden && rows > 1) return fail(NS_ERR_INVALID_ARG, "%s: rows %lld apart, below hidden", name, (long long)t->ld);
    if (too_far(rows, t->ld) || rows * (double)t->ld > 4.6e18 / es) return fail(NS_ERR_OVERFLOW, "%s: offsets overflow", name);
    return NS_OK;
}

struct BlockCall {
    BlockArgs a{};
    int waves = 1;   // of a team
    int lane_elems = 8;
    bool single = false;
    int xs, ys, form;
};

// The form of a call by its width: the fewest waves whose lanes hold the row in 8 or 16 elements each. 4096 values on eight
// waves of 8 in place of four of 16: 16384 rows bf16 forward 113 -> 109 us, backward, whose sums over rows fill the
// registers, 186 -> 171 (with one partial row less). The backward form keeps some of them in scratch above 8192 (48 to 636 bytes a lane)
// and, all in fp32, above 4096 (92 bytes); forward does with an fp32 residual above 8192 (88, 108). 4096 x 16384 bf16 131 us
// forward, 630 backward.
void pick_form(BlockCall &c, int32_t hidden) {
    const int cap[6][3] = {{512, 1, 8}, {1024, 1, 16}, {2048, 4, 8}, {4096, 8, 8}, {8192, 8, 16}, {16384, 16, 16}};
    for (const auto &f : cap)
        if (hidden <= f[0]) {
            c.waves = f[1];
            c.lane_elems = f[2];
            break;
        }
    c.single = hidden < 8;
    if (c.single) c.lane_elems = 1;
}

// Deals rows to teams: a run each; whole gate rows, or a part of one.
void deal(BlockCall &c, bool backward) {
    BlockArgs &a = c.a;
    a.gate_teams = 1;
    if (!a.rows) {
        a.teams = 0;
        return;
    }
    const int most = teams_for(c.waves, backward);
    int64_t per = (a.rows + most - 1) / most;
    if (a.many_gates) {
        const int64_t gates = a.rows / a.gate_span;
        if (per >= a.gate_span) {
            per = per / a.gate_span * a.gate_span;
        } else {
            a.gate_teams = (int32_t)((a.gate_span + per - 1) / per);
            a.per = (int32_t)((a.gate_span + a.gate_teams - 1) / a.gate_teams);
            a.teams = (int32_t)(gates * a.gate_teams);
            return;
        }
    }
    a.per = (int32_t)per;
    a.teams = (int32_t)((a.rows + per - 1) / per);
}

ns_status plan_block(int64_t rows, int32_t hidden, int32_t residual_dtype, int32_t dtype, const ns_rows *x, const ns_rows *y,
                     const void *post_weight, const void *pre_weight, int32_t weight_dtype, int32_t post_norm,
                     const ns_rows *gate, int64_t gate_rows, int32_t gate_dtype, float alpha, float scale, float eps,
                     BlockCall *c) {
    c->xs = dtype_bytes(residual_dtype);
    c->ys = dtype_bytes(dtype);
    if (!c->xs || !c->ys) return fail(NS_ERR_DTYPE, "dtypes %d, %d are not NS_BF16 or NS_F32", residual_dtype, dtype);
    if (c->xs < c->ys) return fail(NS_ERR_DTYPE, "an fp32 block needs an fp32 residual");
    if (!dtype_bytes(weight_dtype)) return fail(NS_ERR_DTYPE, "weight_dtype %d is not NS_BF16 or NS_F32", weight_dtype);
    if (rows < 0 || rows >= int64_t(1) << 31) return fail(NS_ERR_INVALID_ARG, "rows outside [0, 2^31)");
    if (hidden < 1 || hidden > kMaxHidden) return fail(NS_ERR_INVALID_ARG, "hidden = %d outside [1, %d]", hidden, kMaxHidden);
    if (post_norm != 0 && post_norm != 1) return fail(NS_ERR_INVALID_ARG, "post_norm must be 0 or 1");
    if (!(eps >= 0.f) || eps > 3.4e38f) return fail(NS_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (!(alpha >= -3.4e38f && alpha <= 3.4e38f) || !(scale >= -3.4e38f && scale <= 3.4e38f))
        return fail(NS_ERR_INVALID_ARG, "alpha and scale must be finite");
    const bool has_y = y && (y->data || !rows), has_gate = gate && (gate->data || !rows) && (rows || gate_rows);
    if (rows && (!x || !x->data)) return fail(NS_ERR_INVALID_ARG, "x is NULL");
    if (!has_y && (has_gate || post_weight)) return fail(NS_ERR_INVALID_ARG, "gate and post_weight need y");
    if (!post_norm && post_weight) return fail(NS_ERR_INVALID_ARG, "post_weight without post_norm");
    if (misaligned(post_weight, dtype_bytes(weight_dtype)) || misaligned(pre_weight, dtype_bytes(weight_dtype)))
        return fail(NS_ERR_INVALID_ARG, "weights not aligned to their type");
    if (ns_status s = check_rows("x", x, rows, hidden, c->xs)) return s;
    if (ns_status s = check_rows("y", y, rows, hidden, c->ys)) return s;
    if (has_gate) {
        if (!dtype_bytes(gate_dtype)) return fail(NS_ERR_DTYPE, "gate_dtype %d is not NS_BF16 or NS_F32", gate_dtype);
        if (gate_rows < 0 || (rows ? gate_rows < 1 || rows % gate_rows : gate_rows > kMaxEmptyGates))
            return fail(NS_ERR_INVALID_ARG, "gate_rows = %lld does not divide rows", (long long)gate_rows);
        if (ns_status s = check_rows("gate", gate, gate_rows, hidden, dtype_bytes(gate_dtype))) return s;
    }
    BlockArgs &a = c->a;
    a.x = rows_at(x);
    a.y = rows_at(y);
    a.has_y = has_y;
    a.has_gate = has_gate;
    a.gate = has_gate ? rows_at(gate) : Rows{nullptr, 0};
    a.gate_f32 = has_gate && gate_dtype == NS_F32;
    a.many_gates = has_gate && gate_rows > 1;
    a.gate_span = has_gate && rows ? rows / gate_rows : 1;
    a.w_post = post_weight;
    a.w_pre = pre_weight;
    a.w_f32 = weight_dtype == NS_F32;
    a.post_norm = post_norm;
    a.rows = rows;
    a.hidden = hidden;
    a.alpha = alpha;
    a.scale = scale;
    a.eps = eps;
    a.inv_hidden = 1.f / hidden;
    pick_form(*c, hidden);
    return NS_OK;
}

template <bool BWD, class F> void go(const BlockCall &c, hipStream_t st) {
    const dim3 grid((c.a.teams + F::PER_GROUP - 1) / F::PER_GROUP), block(F::THREADS);
    if constexpr (BWD) {
        if (c.a.has_y) hipLaunchKernelGGL((block_norm_backward_kernel<F, true>), grid, block, 0, st, c.a);
        else hipLaunchKernelGGL((block_norm_backward_kernel<F, false>), grid, block, 0, st, c.a);
    } else {
        if (c.a.has_y) hipLaunchKernelGGL((block_norm_kernel<F, true>), grid, block, 0, st, c.a);
        else hipLaunchKernelGGL((block_norm_kernel<F, false>), grid, block, 0, st, c.a);
    }
}

template <bool BWD, typename TX, typename TY> void pick(const BlockCall &c, hipStream_t st) {
    constexpr int V = sizeof(TX) == 2 ? 8 : 4;
    if (c.single) go<BWD, Form<TX, TY, 1, 1, 1>>(c, st);
    else if (c.waves == 1 && c.lane_elems == 8) go<BWD, Form<TX, TY, V, 1, 8>>(c, st);
    else if (c.waves == 1) go<BWD, Form<TX, TY, V, 1, 16>>(c, st);
    else if (c.waves == 4) go<BWD, Form<TX, TY, V, 4, 8>>(c, st);
    else if (c.waves == 8 && c.lane_elems == 8) go<BWD, Form<TX, TY, V, 8, 8>>(c, st);
    else if (c.waves == 8) go<BWD, Form<TX, TY, V, 8, 16>>(c, st);
    else go<BWD, Form<TX, TY, V, 16, 16>>(c, st);
}

template <bool BWD> ns_status launch(const BlockCall &c, hipStream_t st) {
    if (!c.a.teams) return NS_OK;
    if (c.xs == 2) pick<BWD, __bf16, __bf16>(c, st);
    else if (c.ys == 2) pick<BWD, float, __bf16>(c, st);
    else pick<BWD, float, float>(c, st);
    NSQ_HIP(hipGetLastError());
    return NS_OK;
}

// Partial rows of the most teams that a call of this size can have, whatever its gates.
size_t workspace_bytes_of(int64_t rows, int32_t hidden) {
    BlockCall c;
    pick_form(c, hidden);
    // a gate row's last team may hold fewer rows, so there are up to twice as many teams as asked for
    return (size_t)std::min<int64_t>(rows, 2 * teams_for(c.waves, true)) * 3 * hidden * sizeof(float);
}

}  // namespace
}  // namespace nsq

using namespace nsq;

extern "C" ns_status ns_block_norm(int64_t rows, int32_t hidden, ns_dtype residual_dtype, ns_dtype dtype, const ns_rows *x,
                                   const ns_rows *y, const void *post_weight, const void *pre_weight,
                                   ns_dtype weight_dtype, int32_t post_norm, const ns_rows *gate, int64_t gate_rows,
                                   ns_dtype gate_dtype, float alpha, float scale, float eps, const ns_rows *x_out,
                                   const ns_rows *h, void *stream) {
    BlockCall c;
    if (ns_status s = plan_block(rows, hidden, residual_dtype, dtype, x, y, post_weight, pre_weight, weight_dtype, post_norm,
                                 gate, gate_rows, gate_dtype, alpha, scale, eps, &c))
        return s;
    if (ns_status s = check_rows("x_out", x_out, rows, hidden, c.xs)) return s;
    if (ns_status s = check_rows("h", h, rows, hidden, c.ys)) return s;
    c.a.x_out = rows_at(x_out);
    c.a.h = rows_at(h);
    if (rows && !c.a.x_out.p && !c.a.h.p) return fail(NS_ERR_INVALID_ARG, "x_out or h is required");
    if (rows && c.a.x_out.p && !c.a.has_y) return fail(NS_ERR_INVALID_ARG, "x_out needs y");
    deal(c, false);
    return launch<false>(c, as_stream(stream));
}

extern "C" ns_status ns_block_norm_workspace_bytes(int64_t rows, int32_t hidden, size_t *bytes) {
    if (!bytes) return fail(NS_ERR_INVALID_ARG, "bytes is NULL");
    if (rows < 0 || rows >= int64_t(1) << 31) return fail(NS_ERR_INVALID_ARG, "rows outside [0, 2^31)");
    if (hidden < 1 || hidden > kMaxHidden) return fail(NS_ERR_INVALID_ARG, "hidden = %d outside [1, %d]", hidden, kMaxHidden);
    *bytes = workspace_bytes_of(rows, hidden);
    return NS_OK;
}

extern "C" ns_status ns_block_norm_backward(int64_t rows, int32_t hidden, ns_dtype residual_dtype, ns_dtype dtype,
                                            const ns_rows *x, const ns_rows *y, const void *post_weight,
                                            const void *pre_weight, ns_dtype weight_dtype, int32_t post_norm,
                                            const ns_rows *gate, int64_t gate_rows, ns_dtype gate_dtype, float alpha,
                                            float scale, float eps, const ns_rows *dx_out, const ns_rows *dh,
                                            const ns_rows *dx, const ns_rows *dy, float *dpost_weight,
                                            float *dpre_weight, const ns_rows *dgate, void *workspace,
                                            size_t workspace_bytes, void *stream) {
    BlockCall c;
    if (ns_status s = plan_block(rows, hidden, residual_dtype, dtype, x, y, post_weight, pre_weight, weight_dtype, post_norm,
                                 gate, gate_rows, gate_dtype, alpha, scale, eps, &c))
        return s;
    BlockArgs &a = c.a;
    if (ns_status s = check_rows("dx_out", dx_out, rows, hidden, c.xs)) return s;
    if (ns_status s = check_rows("dh", dh, rows, hidden, c.ys)) return s;
    if (ns_status s = check_rows("dx", dx, rows, hidden, c.xs)) return s;
    if (ns_status s = check_rows("dy", dy, rows, hidden, c.ys)) return s;
    a.x_out = rows_at(dx_out);
    a.h = rows_at(dh);
    a.dx = rows_at(dx);
    a.dy = rows_at(dy);
    if (rows && !a.x_out.p && !a.h.p) return fail(NS_ERR_INVALID_ARG, "dx_out or dh is required");
    if (rows && a.x_out.p && !a.has_y) return fail(NS_ERR_INVALID_ARG, "dx_out needs y");
    if (rows && a.dy.p && !a.has_y) return fail(NS_ERR_INVALID_ARG, "dy needs y");
    if (dpost_weight && !(a.has_y && post_norm)) return fail(NS_ERR_INVALID_ARG, "dpost_weight needs y and post_norm");
    if (misaligned(dpost_weight, 4) || misaligned(dpre_weight, 4))
        return fail(NS_ERR_INVALID_ARG, "dpost_weight / dpre_weight not 4-byte aligned");
    if (dgate && dgate->data) {
        if (!a.has_gate) return fail(NS_ERR_INVALID_ARG, "dgate needs gate");
        if (ns_status s = check_rows("dgate", dgate, gate_rows, hidden, dtype_bytes(gate_dtype))) return s;
        a.dgate = rows_at(dgate);
    }
    a.dw_post = dpost_weight;
    a.dw_pre = dpre_weight;
    deal(c, true);
    a.whole_gates = a.many_gates && a.gate_teams == 1 && rows;   // without rows the second launch clears the gradients
    const bool join_gate = a.dgate.p && !a.whole_gates;
    a.join_u = a.dw_post || join_gate;
    a.sets = join_gate && a.many_gates ? 3 : 2;
    const bool join = a.dw_pre || a.join_u;
    if (join) {
        const size_t need = workspace_bytes_of(rows, hidden);
        if (need && (!workspace || workspace_bytes < need))
            return fail(NS_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : 0, need);
        if (misaligned(workspace, 256)) return fail(NS_ERR_INVALID_ARG, "workspace not 256-byte aligned");
    }
    a.partial = reinterpret_cast<float *>(workspace);
    hipStream_t st = as_stream(stream);
    if (ns_status s = launch<true>(c, st)) return s;
    if (join) {
        const int gates = join_gate && a.many_gates ? (int)gate_rows : 0;
        hipLaunchKernelGGL(block_norm_join_kernel, dim3((hidden + kJoinCols - 1) / kJoinCols, a.join_u ? 2 + gates : 1),
                           dim3(kJoinCols * kJoinRows), 0, st, a);
        NSQ_HIP(hipGetLastError());
    }
    return NS_OK;
}
