// Tokens sorted by expert and back, with the router's weights, and gradients.
//
// The T tokens' K choices are T K slots (slot = token K + choice). ns_moe_sort
// gives every slot a row: kept slots by expert and, within one, by slot (a
// stable counting sort); slots whose id is outside [0, E) are dropped and take
// the rows behind, in slot order, marked by the complement of their row.
//   dispatch            xs[row] = x[token]          (dropped rows: zeros)
//   its gradient        dx[t] = sum_k dxs[row(t, k)]
//   combine             out[t] = sum_k w[t, k] y[row(t, k)]
//   its gradient        dy[row] = w dout[t],  dw[t, k] = <dout[t], y[row]>
// Sums run in fp32 over the choices in order and are rounded once; dropped
// slots' rows and weights take no part, whatever they hold. Every row is
// written once, by its own token, so there are no atomics and each result has
// one order.
//
// Bound by memory: a pass reads or writes K rows a token and one more. 8192
// tokens x 8 bf16 rows of 7168 of 64 experts: sort, dispatch and combine 382 us
// (5.5 TB/s), the two gradients 560 us (5.5); a large copy here reaches 5.1. Few
// tokens are bound by their launches: 8 of them 3.2, 2.7 and 3.2 us.

#include <algorithm>
#include <type_traits>

#include "op_util.h"
#include "sort_split.h"

namespace nsq {
namespace {

// ---------------------------------------------------------------------------
// sort
// ---------------------------------------------------------------------------

constexpr int kMaxExperts = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortRounds = 4;   // rounds of 64 slots that a wave ranks at once

struct SortArgs {
    const void *ids;
    int64_t ids_ld;          // elements from a token's ids to the next one's
    int32_t id_bytes;
    int32_t slots, top_k, experts;
    int32_t per;             // slots per workgroup: a multiple of kSortThreads
    int32_t blocks;
    int32_t *offsets, *slot_of_row, *row_of_slot;
    int32_t *hist;           // [blocks][hist_ld(experts)]: each workgroup's counts
};

// Counts of keys 0 .. experts in whole int4.
__host__ __device__ inline int hist_ld(int experts) { return (experts + 1 + 3) & ~3; }

// The sort key of a slot: its expert, or `experts` if dropped.
__device__ inline int key_of(const SortArgs &A, uint32_t slot) {
    int64_t at = slot;
    if (A.ids_ld != A.top_k) {
        const uint32_t t = slot / (uint32_t)A.top_k;
        at += (int64_t)t * (A.ids_ld - A.top_k);
    }
    const int64_t id = A.id_bytes == 8 ? reinterpret_cast<const int64_t *>(A.ids)[at]
                                       : (int64_t) reinterpret_cast<const int32_t *>(A.ids)[at];
    return id < 0 || id >= A.experts ? A.experts : (int)id;
}

// Counts of each key in one workgroup's slots.
__global__ __launch_bounds__(kSortThreads) void moe_count_kernel(SortArgs A) {
    __shared__ int32_t cnt[kMaxExperts + 1];
    for (int e = threadIdx.x; e <= A.experts; e += kSortThreads) cnt[e] = 0;
    __syncthreads();
    const int64_t s0 = (int64_t)blockIdx.x * A.per;
    const int64_t s1 = s0 + A.per < A.slots ? s0 + A.per : A.slots;
#pragma unroll 4
    for (int64_t s = s0 + threadIdx.x; s < s1; s += kSortThreads) atomicAdd(&cnt[key_of(A, (uint32_t)s)], 1);
    __syncthreads();
    for (int e = threadIdx.x; e < hist_ld(A.experts); e += kSortThreads)
        A.hist[(int64_t)blockIdx.x * hist_ld(A.experts) + e] = e <= A.experts ? cnt[e] : 0;
}

// Rows of one workgroup's slots. Wave w holds the w-th run of per / 8 of
// them; a slot's row is its key's first row, plus the same key's slots in
// earlier workgroups, earlier waves, earlier rounds of this wave and lower
// lanes. A wave's LDS operations run in order, and none of a round's waits for
// another round: the lanes of a key set their bits in its mask and read it, which
// tells each the lower ones, then read the wave's count of the key, to which the
// lowest adds the mask's bits. (Masks from one ballot for each of the key's bits
// keep the vector units busy: 64 slots 4.2 us, so 3.2.) Runs of at most
// kSortRounds rounds are ranked before the counts ahead of them are known,
// longer ones after. ONE: the only workgroup, which counts for itself.
//
// Of 524288 slots and 256 experts (15.0 us with the counts, which stream 6 MB)
// some 7 us go into reading every workgroup's counts in each; two to four
// workgroups counted in one cost as much there as they save here.
template <bool ONE>
__global__ __launch_bounds__(kSortThreads) void moe_rank_kernel(SortArgs A) {
    constexpr int kKeys = kSortWaves * (kMaxExperts + 1);   // [wave][key], K1 apart
    __shared__ __attribute__((aligned(16))) int32_t cnt[kKeys];
    __shared__ __attribute__((aligned(16))) uint64_t same[kKeys];
    __shared__ int32_t before[kMaxExperts + 4], total[kMaxExperts + 4];
    __shared__ int32_t wave_total[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int E = A.experts, K1 = E + 1;
    for (int i = tid; i < K1; i += kSortThreads) before[i] = total[i] = 0;
    for (int i = tid * 4; i < kSortWaves * K1; i += kSortThreads * 4) {   // kSortWaves is a multiple of 4
        *reinterpret_cast<int4 *>(&cnt[i]) = int4{0, 0, 0, 0};
        *reinterpret_cast<int4 *>(&same[i]) = int4{0, 0, 0, 0};
        *reinterpret_cast<int4 *>(&same[i + 2]) = int4{0, 0, 0, 0};
    }
    int32_t *const mine_cnt = cnt + wave * K1;
    __syncthreads();
    const int run = A.per / kSortWaves;
    const int64_t w0 = (int64_t)blockIdx.x * A.per + (int64_t)wave * run;
    const int64_t w1 = w0 + run < A.slots ? w0 + run : A.slots;
    int key[kSortRounds], rank[kSortRounds];
    const auto rank_rounds = [&](int64_t s0) {
        uint64_t m[kSortRounds];
#pragma unroll
        for (int i = 0; i < kSortRounds; ++i) {
            const int64_t s = s0 + i * 64 + lane;
            key[i] = s < w1 ? key_of(A, (uint32_t)s) : -1;
        }
#pragma unroll
        for (int i = 0; i < kSortRounds; ++i) {
            m[i] = 0;
            if (key[i] < 0) continue;
            uint64_t *const mask = &same[wave * K1 + key[i]];
            __hip_atomic_fetch_or(mask, 1ull << lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
            __builtin_amdgcn_wave_barrier();
            m[i] = __hip_atomic_load(mask, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
            __builtin_amdgcn_wave_barrier();
            __hip_atomic_store(mask, 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        }
#pragma unroll
        for (int i = 0; i < kSortRounds; ++i) {
            const int lower = __popcll(m[i] & ((1ull << lane) - 1));
            rank[i] = 0;
            if (key[i] < 0) continue;
            int32_t *const count = &mine_cnt[key[i]];
            rank[i] = lower + __hip_atomic_load(count, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
            __builtin_amdgcn_wave_barrier();
            if (lower == 0) __hip_atomic_fetch_add(count, (int)__popcll(m[i]), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        }
    };
    const bool again = A.per > kSortRounds * kSortThreads;
    if (again) {
#pragma unroll 4
        for (int64_t s = w0 + lane; s < w1; s += 64) atomicAdd(&mine_cnt[key_of(A, (uint32_t)s)], 1);
    } else {
        rank_rounds(w0);
    }
    if constexpr (!ONE) {
        const int cols = hist_ld(E) / 4, groups = kSortThreads / cols, group = tid / cols, col = tid - group * cols;
        if (group < groups) {
            const int4 *hist = reinterpret_cast<const int4 *>(A.hist) + col;
            int4 b = {0, 0, 0, 0}, t = {0, 0, 0, 0};
#pragma unroll 8
            for (int c = group; c < A.blocks; c += groups) {
                const int4 v = hist[(int64_t)c * cols];
                const int earlier = c < (int)blockIdx.x ? -1 : 0;
                t.x += v.x, t.y += v.y, t.z += v.z, t.w += v.w;
                b.x += v.x & earlier, b.y += v.y & earlier, b.z += v.z & earlier, b.w += v.w & earlier;
            }
            const int tv[4] = {t.x, t.y, t.z, t.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                atomicAdd(&before[col * 4 + i], bv[i]);   // integers: any order gives the same sum
                atomicAdd(&total[col * 4 + i], tv[i]);
            }
        }
    }
    __syncthreads();
    for (int e = tid; e < K1; e += kSortThreads) {   // counts to first ranks, wave by wave
        int32_t sum = 0;
        for (int w = 0; w < kSortWaves; ++w) {
            const int32_t v = cnt[w * K1 + e];
            cnt[w * K1 + e] = sum;
            sum += v;
        }
        if constexpr (ONE) total[e] = sum;
    }
    __syncthreads();
    // first row of each expert: an exclusive sum over the (at most 1024) experts
    constexpr int kEach = kMaxExperts / kSortThreads;
    int32_t mine = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) mine += tid * kEach + i < E ? total[tid * kEach + i] : 0;
    int32_t incl = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t up = __shfl_up(incl, d);
        if (lane >= d) incl += up;
    }
    if (lane == 63) wave_total[wave] = incl;
    __syncthreads();
    int32_t first = incl - mine, kept = 0;
    for (int w = 0; w < kSortWaves; ++w) {
        if (w < wave) first += wave_total[w];
        kept += wave_total[w];
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int e = tid * kEach + i;
        if (e >= E) break;
        before[e] += first;
        if (blockIdx.x == 0) A.offsets[e] = first;
        first += total[e];
    }
    if (tid == 0) {
        before[E] += kept;
        if (blockIdx.x == 0) A.offsets[E] = kept;
    }
    __syncthreads();
    for (int64_t s0 = w0; s0 < w1; s0 += 64 * kSortRounds) {
        if (again) rank_rounds(s0);   // now from the counts before this wave on
#pragma unroll
        for (int i = 0; i < kSortRounds; ++i) {
            if (key[i] < 0) continue;
            const int32_t row = before[key[i]] + rank[i] + (again ? 0 : mine_cnt[key[i]]);
            const int32_t slot = (int32_t)(s0 + i * 64 + lane);
            A.row_of_slot[slot] = key[i] == E ? ~row : row;
            A.slot_of_row[row] = key[i] == E ? ~slot : slot;
        }
    }
}

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------

struct RowArgs {
    const void *x, *y;       // token rows, sorted rows (inputs of the pass)
    void *tok, *rows;        // token rows, sorted rows (outputs)
    int64_t x_ld, y_ld, tok_ld, rows_ld;
    const int32_t *row_of_slot;
    const float *w;
    float *dw;
    int64_t tokens;
    int32_t top_k, hidden;
    int32_t units;           // 16-byte units of a row, the last one perhaps partial
    int32_t pieces;          // workgroups per token
    uint32_t blocks;         // tokens x pieces, < 2^31
    uint32_t slots;          // tokens x top_k: rows of the sorted side
};

// A token's map entries and weights, KC choices from k0 on, all asked for at once
// and through the scalar cache (no kernel that reads them writes them). An entry
// that names no row of the buffer (no map of ns_moe_sort's holds one) is left
// alone.
template <int KC, bool W> struct Choices {
    int64_t row[KC];
    bool kept[KC], in[KC];
    float w[KC];
    __device__ Choices(const RowArgs &A, int64_t token, int k0) {
        const int32_t NSQ_CONST *map = (const int32_t NSQ_CONST *)(A.row_of_slot + token * A.top_k);
        const float NSQ_CONST *weights = (const float NSQ_CONST *)(A.w + token * A.top_k);
        int32_t r[KC];
#pragma unroll
        for (int j = 0; j < KC; ++j) {
            const int k = min(k0 + j, A.top_k - 1);
            r[j] = map[k];
            w[j] = W ? weights[k] : 1.f;
        }
#pragma unroll
        for (int j = 0; j < KC; ++j) {
            const uint32_t at = r[j] < 0 ? ~r[j] : r[j];
            row[j] = at;
            in[j] = k0 + j < A.top_k && at < A.slots;
            kept[j] = in[j] && r[j] >= 0;
        }
    }
};

// Unit u of a row of `hidden` elements; elements past its end read as zero and are not written.
// NT: read or written past the cache.
template <typename T, bool NT>
__device__ inline typename Vec16<T>::raw load_unit(const T *row, int u, int hidden) {
    constexpr int N = Vec16<T>::N;
    if ((u + 1) * N <= hidden) return load_vec<T, NT>(row + u * N);
    typename Vec16<T>::raw v = {};
    for (int i = 0; i < N - 1; ++i)
        if (u * N + i < hidden) v[i] = reinterpret_cast<const std::remove_reference_t<decltype(v[0])> *>(row)[u * N + i];
    return v;
}
template <typename T, bool NT>
__device__ inline void store_unit(T *row, int u, int hidden, typename Vec16<T>::raw v) {
    constexpr int N = Vec16<T>::N;
    if ((u + 1) * N <= hidden) {
        store_vec<T, NT>(row + u * N, v);
        return;
    }
    for (int i = 0; i < N - 1; ++i)
        if (u * N + i < hidden) reinterpret_cast<std::remove_reference_t<decltype(v[0])> *>(row)[u * N + i] = v[i];
}

// xs[row] = x[token]: a thread reads one unit and writes it K times.
template <typename T, bool NT>
__global__ __launch_bounds__(128) void moe_dispatch_kernel(RowArgs A) {
    constexpr int KC = 8;
    for (uint32_t b = blockIdx.x; b < A.blocks; b += gridDim.x) {
        const uint32_t t32 = b / (uint32_t)A.pieces;
        const int64_t t = t32;
        const int u = (int)(b - t32 * A.pieces) * blockDim.x + threadIdx.x;
        if (u >= A.units) continue;
        const auto v = load_unit<T, false>(reinterpret_cast<const T *>(A.x) + t * A.x_ld, u, A.hidden);
        for (int k0 = 0; k0 < A.top_k; k0 += KC) {
            const Choices<KC, false> c(A, t, k0);
            const typename Vec16<T>::raw z = {};
#pragma unroll
            for (int j = 0; j < KC; ++j)
                if (c.in[j])
                    store_unit<T, NT>(reinterpret_cast<T *>(A.rows) + c.row[j] * A.rows_ld, u, A.hidden, c.kept[j] ? v : z);
        }
    }
}

// tok[t] = sum_k w[t, k] y[row(t, k)] (W = false: w = 1), up to KC rows in flight.
template <typename T, bool W, int KC, bool NT>
__global__ __launch_bounds__(128) void moe_combine_kernel(RowArgs A) {
    constexpr int N = Vec16<T>::N;
    for (uint32_t b = blockIdx.x; b < A.blocks; b += gridDim.x) {
        const uint32_t t32 = b / (uint32_t)A.pieces;
        const int64_t t = t32;
        const int u = (int)(b - t32 * A.pieces) * blockDim.x + threadIdx.x;
        if (u >= A.units) continue;
        float acc[N] = {};
        for (int k0 = 0; k0 < A.top_k; k0 += KC) {
            const Choices<KC, W> c(A, t, k0);
            typename Vec16<T>::raw v[KC];
#pragma unroll
            for (int j = 0; j < KC; ++j)
                if (c.kept[j]) v[j] = load_unit<T, NT>(reinterpret_cast<const T *>(A.y) + c.row[j] * A.y_ld, u, A.hidden);
#pragma unroll
            for (int j = 0; j < KC; ++j)
                if (c.kept[j])
#pragma unroll
                    for (int i = 0; i < N; ++i) acc[i] += c.w[j] * elem<T>(v[j], i);
        }
        typename Vec16<T>::raw o;
#pragma unroll
        for (int i = 0; i < N; ++i) set_elem<T>(o, i, acc[i]);
        store_unit<T, NT>(reinterpret_cast<T *>(A.tok) + t * A.tok_ld, u, A.hidden, o);
    }
}

// dy[row] = w dout[t] and dw[t, k] = <dout[t], y[row]>: one workgroup per
// token, KC choices at a time, their partial dot products in registers.
template <typename T, int KC, bool NT>
__global__ __launch_bounds__(512) void moe_combine_backward_kernel(RowArgs A) {
    constexpr int N = Vec16<T>::N;
    __shared__ float part[8][KC];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    for (int64_t t = blockIdx.x; t < A.tokens; t += gridDim.x) {
        const T *g = reinterpret_cast<const T *>(A.x) + t * A.x_ld;
        for (int k0 = 0; k0 < A.top_k; k0 += KC) {
            const Choices<KC, true> c(A, t, k0);
            float dot[KC] = {};
            for (int u = threadIdx.x; u < A.units; u += blockDim.x) {
                const auto gv = load_unit<T, NT>(g, u, A.hidden);
                typename Vec16<T>::raw v[KC];
#pragma unroll
                for (int j = 0; j < KC; ++j)
                    if (c.kept[j])
                        v[j] = load_unit<T, NT>(reinterpret_cast<const T *>(A.y) + c.row[j] * A.y_ld, u, A.hidden);
#pragma unroll
                for (int j = 0; j < KC; ++j) {
                    if (!c.in[j]) continue;
                    typename Vec16<T>::raw o = {};
                    if (c.kept[j]) {
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            dot[j] += elem<T>(gv, i) * elem<T>(v[j], i);
                            set_elem<T>(o, i, c.w[j] * elem<T>(gv, i));
                        }
                    }
                    store_unit<T, NT>(reinterpret_cast<T *>(A.rows) + c.row[j] * A.rows_ld, u, A.hidden, o);
                }
            }
#pragma unroll
            for (int j = 0; j < KC; ++j) {
                dot[j] = wave_sum(dot[j]);
                if (lane == 0) part[wave][j] = dot[j];
            }
            __syncthreads();
            if (threadIdx.x < KC && k0 + threadIdx.x < (unsigned)A.top_k) {
                float s = 0.f;
                for (int i = 0; i < waves; ++i) s += part[i][threadIdx.x];
                A.dw[t * A.top_k + k0 + threadIdx.x] = s;
            }
            __syncthreads();
        }
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

ns_status check_slots(int64_t tokens, int32_t top_k) {
    if (tokens < 0) return fail(NS_ERR_INVALID_ARG, "tokens < 0");
    if (top_k < 1) return fail(NS_ERR_INVALID_ARG, "top_k = %d < 1", top_k);
    // top_k: the kernels count choices in steps of 8 in 32 bits
    if (tokens > INT32_MAX / top_k || (tokens > 0 && top_k > 1 << 30))
        return fail(NS_ERR_OVERFLOW, "tokens x top_k does not fit in 31 bits, or top_k in 30");
    return NS_OK;
}

// A (rows, hidden) operand with its row stride.
ns_status check_rows(const char *name, const void *p, int64_t rows, int32_t hidden, int64_t ld, int es) {
    if (ld < hidden) return fail(NS_ERR_INVALID_ARG, "%s: row stride %lld < hidden %d", name, (long long)ld, hidden);
    if (too_far(rows, ld) || too_far(rows * ld, es)) return fail(NS_ERR_OVERFLOW, "%s: offsets overflow", name);
    if (rows == 0 || hidden == 0) return NS_OK;
    if (!p) return fail(NS_ERR_INVALID_ARG, "%s is NULL", name);
    if (misaligned(p, es)) return fail(NS_ERR_INVALID_ARG, "%s not %d-byte aligned", name, es);
    return NS_OK;
}

ns_status check_map(int64_t slots, const int32_t *row_of_slot) {
    if (slots > 0 && !row_of_slot) return fail(NS_ERR_INVALID_ARG, "row_of_slot is NULL");
    if (misaligned(row_of_slot, 4)) return fail(NS_ERR_INVALID_ARG, "row_of_slot not 4-byte aligned");
    return NS_OK;
}

// Workgroups of at most 128 threads over a row's units, evenly filled: small ones
// keep the GPU evenly loaded (8192 tokens x 8 rows of 896 units, dispatch and
// combine: 128 threads 389 us, 64 399, 448 430).
unsigned row_threads(int32_t units, int32_t *pieces) {
    *pieces = units > 128 ? (units + 127) / 128 : 1;
    const int32_t each = (units + *pieces - 1) / *pieces;
    return (unsigned)(each + 63) / 64 * 64;
}

unsigned row_grid(uint32_t blocks) { return blocks < (1u << 22) ? blocks : 1u << 22; }

ns_status check_call(int64_t tokens, int32_t top_k, int32_t hidden, int32_t dtype, int *es) {
    *es = dtype_bytes(dtype);
    if (!*es) return fail(NS_ERR_DTYPE, "dtype %d is not NS_BF16 or NS_F32", dtype);
    if (ns_status s = check_slots(tokens, top_k)) return s;
    if (hidden < 0) return fail(NS_ERR_INVALID_ARG, "hidden < 0");
    const int64_t pieces = (((int64_t)hidden * *es + 15) / 16 + 127) / 128;
    if (hidden > 1 << 28 || tokens * (double)pieces >= 2147483648.0)
        return fail(NS_ERR_OVERFLOW, "%lld tokens of %d values are more than one call counts", (long long)tokens, hidden);
    return NS_OK;
}

// Sizes, map and workgroups; returns the threads of a workgroup.
unsigned fill(RowArgs &a, int64_t tokens, int32_t top_k, int32_t hidden, int es, const int32_t *row_of_slot) {
    a.row_of_slot = row_of_slot;
    a.tokens = tokens;
    a.top_k = top_k;
    a.hidden = hidden;
    a.slots = (uint32_t)(tokens * top_k);
    a.units = (hidden + 16 / es - 1) / (16 / es);
    const unsigned threads = row_threads(a.units, &a.pieces);
    a.blocks = (uint32_t)(tokens * a.pieces);
    return threads;
}

// Whether a call that moves `rows` rows a token moves more than the last-level
// cache holds. Its rows are then read and written past it: 8192 tokens x 8 rows
// of 14 KiB, dispatch 208 -> 176 us (its reads stay as they are: with them 219),
// combine 221 -> 207, its gradient 395 -> 384.
bool past_cache(const RowArgs &a, int es, int64_t rows) {
    return (double)a.tokens * rows * a.hidden * es > (double)kMallBytes;
}

ns_status combine(int64_t tokens, int32_t top_k, int32_t hidden, int32_t dtype, const void *y, int64_t y_ld,
                  const int32_t *row_of_slot, const float *w, void *out, int64_t out_ld, const char *y_name,
                  const char *out_name, void *stream) {
    int es;
    if (ns_status s = check_call(tokens, top_k, hidden, dtype, &es)) return s;
    if (ns_status s = check_rows(y_name, y, tokens * top_k, hidden, y_ld, es)) return s;
    if (ns_status s = check_rows(out_name, out, tokens, hidden, out_ld, es)) return s;
    if (ns_status s = check_map(tokens * top_k, row_of_slot)) return s;
    if (tokens == 0 || hidden == 0) return NS_OK;
    RowArgs a{};
    a.y = y;
    a.y_ld = y_ld;
    a.tok = out;
    a.tok_ld = out_ld;
    a.w = w;
    const unsigned threads = fill(a, tokens, top_k, hidden, es, row_of_slot);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(row_grid(a.blocks)), dim3(threads), 0, as_stream(stream), a);
    };
    auto pick = [&](auto t) {
        typedef decltype(t) T;
        const auto weighted = [&](auto nt) {
            constexpr bool NT = decltype(nt)::value;
            if (w) top_k <= 4 ? go(moe_combine_kernel<T, true, 4, NT>) : go(moe_combine_kernel<T, true, 8, NT>);
            else top_k <= 4 ? go(moe_combine_kernel<T, false, 4, NT>) : go(moe_combine_kernel<T, false, 8, NT>);
        };
        past_cache(a, es, top_k + 1) ? weighted(std::true_type{}) : weighted(std::false_type{});
    };
    if (dtype == NS_BF16) pick((__bf16)0.f);
    else pick(0.f);
    NSQ_HIP(hipGetLastError());
    return NS_OK;
}

}  // namespace
}  // namespace nsq

using namespace nsq;

extern "C" ns_status ns_moe_sort_workspace_bytes(int64_t tokens, int32_t top_k, int32_t experts, size_t *bytes) {
    if (!bytes) return fail(NS_ERR_INVALID_ARG, "bytes is NULL");
    if (ns_status s = check_slots(tokens, top_k)) return s;
    if (experts < 1 || experts > kMaxExperts)
        return fail(NS_ERR_INVALID_ARG, "experts = %d outside [1, %d]", experts, kMaxExperts);
    *bytes = (size_t)kMaxSortBlocks * hist_ld(experts) * sizeof(int32_t);
    return NS_OK;
}

extern "C" ns_status ns_moe_sort(int64_t tokens, int32_t top_k, int32_t experts, const void *expert_ids,
                                 int32_t id_bytes, int64_t ids_ld, int32_t *offsets, int32_t *slot_of_row,
                                 int32_t *row_of_slot, void *workspace, size_t workspace_bytes, void *stream) {
    size_t need;
    if (ns_status s = ns_moe_sort_workspace_bytes(tokens, top_k, experts, &need)) return s;
    if (id_bytes != 4 && id_bytes != 8) return fail(NS_ERR_DTYPE, "id_bytes = %d (must be 4 or 8)", id_bytes);
    if (ids_ld < top_k) return fail(NS_ERR_INVALID_ARG, "ids_ld = %lld < top_k", (long long)ids_ld);
    if (too_far(tokens, ids_ld) || too_far(tokens * ids_ld, id_bytes))
        return fail(NS_ERR_OVERFLOW, "expert_ids: offsets overflow");
    if (!offsets || misaligned(offsets, 4)) return fail(NS_ERR_INVALID_ARG, "offsets is NULL or not 4-byte aligned");
    if (tokens > 0 && (!expert_ids || !slot_of_row || !row_of_slot))
        return fail(NS_ERR_INVALID_ARG, "expert_ids, slot_of_row and row_of_slot are required");
    if (misaligned(expert_ids, id_bytes) || misaligned(slot_of_row, 4) || misaligned(row_of_slot, 4))
        return fail(NS_ERR_INVALID_ARG, "expert_ids, slot_of_row or row_of_slot not aligned to its type");
    if (!workspace || workspace_bytes < need)
        return fail(NS_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : 0, need);
    if (misaligned(workspace, 256)) return fail(NS_ERR_INVALID_ARG, "workspace not 256-byte aligned");
    SortArgs a{};
    a.ids = expert_ids;
    a.ids_ld = ids_ld;
    a.id_bytes = id_bytes;
    a.slots = (int32_t)(tokens * top_k);
    a.top_k = top_k;
    a.experts = experts;
    a.offsets = offsets;
    a.slot_of_row = slot_of_row;
    a.row_of_slot = row_of_slot;
    a.hist = reinterpret_cast<int32_t *>(workspace);
    const SortSplit split = sort_split(a.slots);
    a.per = split.per;
    a.blocks = split.blocks;
    const hipStream_t st = as_stream(stream);
    if (a.blocks == 1) {
        hipLaunchKernelGGL(moe_rank_kernel<true>, dim3(1), dim3(kSortThreads), 0, st, a);
    } else {
        hipLaunchKernelGGL(moe_count_kernel, dim3(a.blocks), dim3(kSortThreads), 0, st, a);
        hipLaunchKernelGGL(moe_rank_kernel<false>, dim3(a.blocks), dim3(kSortThreads), 0, st, a);
    }
    NSQ_HIP(hipGetLastError());
    return NS_OK;
}

extern "C" ns_status ns_moe_dispatch(int64_t tokens, int32_t top_k, int32_t hidden, ns_dtype dtype, const void *x,
                                     int64_t x_ld, const int32_t *row_of_slot, void *xs, int64_t xs_ld,
                                     void *stream) {
    int es;
    if (ns_status s = check_call(tokens, top_k, hidden, dtype, &es)) return s;
    if (ns_status s = check_rows("x", x, tokens, hidden, x_ld, es)) return s;
    if (ns_status s = check_rows("xs", xs, tokens * top_k, hidden, xs_ld, es)) return s;
    if (ns_status s = check_map(tokens * top_k, row_of_slot)) return s;
    if (tokens == 0 || hidden == 0) return NS_OK;
    RowArgs a{};
    a.x = x;
    a.x_ld = x_ld;
    a.rows = xs;
    a.rows_ld = xs_ld;
    const unsigned threads = fill(a, tokens, top_k, hidden, es, row_of_slot);
    const dim3 grid(row_grid(a.blocks));
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, as_stream(stream), a); };
    const bool nt = past_cache(a, es, top_k + 1);
    if (dtype == NS_BF16) nt ? go(moe_dispatch_kernel<__bf16, true>) : go(moe_dispatch_kernel<__bf16, false>);
    else nt ? go(moe_dispatch_kernel<float, true>) : go(moe_dispatch_kernel<float, false>);
    NSQ_HIP(hipGetLastError());
    return NS_OK;
}

extern "C" ns_status ns_moe_dispatch_backward(int64_t tokens, int32_t top_k, int32_t hidden, ns_dtype dtype,
                                              const void *dxs, int64_t dxs_ld, const int32_t *row_of_slot, void *dx,
                                              int64_t dx_ld, void *stream) {
    return combine(tokens, top_k, hidden, dtype, dxs, dxs_ld, row_of_slot, nullptr, dx, dx_ld, "dxs", "dx", stream);
}

extern "C" ns_status ns_moe_combine(int64_t tokens, int32_t top_k, int32_t hidden, ns_dtype dtype, const void *y,
                                    int64_t y_ld, const int32_t *row_of_slot, const float *weights, void *out,
                                    int64_t out_ld, void *stream) {
    if (misaligned(weights, 4)) return fail(NS_ERR_INVALID_ARG, "weights not 4-byte aligned");
    return combine(tokens, top_k, hidden, dtype, y, y_ld, row_of_slot, weights, out, out_ld, "y", "out", stream);
}

extern "C" ns_status ns_moe_combine_backward(int64_t tokens, int32_t top_k, int32_t hidden, ns_dtype dtype,
                                             const void *dout, int64_t dout_ld, const void *y, int64_t y_ld,
                                             const int32_t *row_of_slot, const float *weights, void *dy,
                                             int64_t dy_ld, float *dweights, void *stream) {
    int es;
    if (ns_status s = check_call(tokens, top_k, hidden, dtype, &es)) return s;
    if (ns_status s = check_rows("dout", dout, tokens, hidden, dout_ld, es)) return s;
    if (ns_status s = check_rows("y", y, tokens * top_k, hidden, y_ld, es)) return s;
    if (ns_status s = check_rows("dy", dy, tokens * top_k, hidden, dy_ld, es)) return s;
    if (ns_status s = check_map(tokens * top_k, row_of_slot)) return s;
    if (tokens > 0 && (!weights || !dweights)) return fail(NS_ERR_INVALID_ARG, "weights and dweights are required");
    if (misaligned(weights, 4) || misaligned(dweights, 4))
        return fail(NS_ERR_INVALID_ARG, "weights or dweights not 4-byte aligned");
    if (tokens == 0) return NS_OK;
    RowArgs a{};
    a.x = dout;
    a.x_ld = dout_ld;
    a.y = y;
    a.y_ld = y_ld;
    a.rows = dy;
    a.rows_ld = dy_ld;
    a.w = weights;
    a.dw = dweights;
    fill(a, tokens, top_k, hidden, es, row_of_slot);
    // At least two rounds of units a thread, spread evenly over at most 512 threads: a workgroup's sums and barriers
    // then cost less beside its rows (385 units, 3 choices: 192 threads 25 us, 448 32; 896 units, 8 choices: 448
    // threads 385 us, 256 393, 64 401).
    const int32_t rounds = a.units <= 64 ? 1 : std::max(2, (a.units + 511) / 512);
    const unsigned threads = (unsigned)std::max(1, ((a.units + rounds - 1) / rounds + 63) / 64) * 64;
    const dim3 grid(row_grid((uint32_t)tokens));
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, as_stream(stream), a); };
    auto pick = [&](auto t) {
        typedef decltype(t) T;
        if (past_cache(a, es, 2 * top_k + 1))
            top_k <= 4 ? go(moe_combine_backward_kernel<T, 4, true>) : go(moe_combine_backward_kernel<T, 8, true>);
        else
            top_k <= 4 ? go(moe_combine_backward_kernel<T, 4, false>) : go(moe_combine_backward_kernel<T, 8, false>);
    };
    if (dtype == NS_BF16) pick((__bf16)0.f);
    else pick(0.f);
    NSQ_HIP(hipGetLastError());
    return NS_OK;
}
