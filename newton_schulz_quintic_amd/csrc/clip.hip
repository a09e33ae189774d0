// The norm of many gradients together, and their clipping on the way into the
// momentum:
//   norm = sqrt(sum over tensors of sum g^2),
//   c = min(1, max_norm / (norm + eps)),  out = beta m + c g.
//
// Squares are added in 64 bits, which hold the square of any fp32 value and cost
// nothing here (one conversion and one fma for 2 or 4 bytes read); a workgroup's
// sums go to the workspace and one workgroup adds those in order, so the same
// gradients give the same bits.
//
// The tensors of a call are cut into chunks, numbered through, and every workgroup
// takes a run of chunks: it looks its first tensor up once and walks on from
// there. Up to kInline tensors travel in the kernel's arguments; the table of a
// longer list is written to the workspace first, kInline tensors a launch (about
// 2 us each), so that a captured call keeps nothing on the host.
//
// Bound by memory: the norm reads each gradient once, the clipping reads gradient
// (and momentum) and writes the output. In place with c = 1 and beta = 0 nothing
// has to be written, and nothing is read or written. The 28 matrices of four layers
// (hidden 4096, FFN 14336; 872 million values, bf16 gradients, fp32 momenta): norm 289
// us (6.0 TB/s), clipping 1655 us (5.3 TB/s). 26 norms' weights of up to 4096 values:
// 6.5 and 4.5 us, of which the launches and the chain of sums are the most.

#include <algorithm>

#include "elems.h"

namespace nsq {
namespace {

constexpr int kThreads = 256;
constexpr int kSoloThreads = 1024;
constexpr int kInline = 96;
constexpr int kMaxTensors = 1 << 20;
// As many workgroups as are resident at once (8 a CU).
constexpr int kMaxBlocks = 2048;
// Up to this many bytes of gradients one workgroup takes the whole norm: one launch in place of two (0.1 MB 4.9 us, 9.2
// with two; 0.3 MB 9.3 and 9.1).
constexpr int64_t kSoloBytes = 256 << 10;

struct Entry {
    const char *g, *m;
    char *o;
    int64_t count;
    int32_t first;      // number of its first chunk
    int16_t kind;       // bit 0: the gradient is fp32, bit 1: output and momentum are
    int16_t lg;         // log2 of a chunk's elements
};
static_assert(sizeof(Entry) == 40, "Entry layout");

struct ClipArgs {
    Entry inline_table[kInline];   // first: the kernels read it at the start of their argument segment
    const Entry *table;            // or, for a longer list, in the workspace
    int32_t n, chunks;
    double *partial;
    float *norm;
    double *sum_sq;
    const float *norm_in;
    float max_norm, eps, beta;
};
static_assert(sizeof(ClipArgs) <= 4096, "kernel arguments");

struct TableArgs {
    Entry part[kInline];
    Entry *to;
    int32_t n;
};

__global__ __launch_bounds__(kThreads) void grad_table_kernel(TableArgs a) {
    // eight bytes a thread, from the argument segment
    const uint64_t NSQ_CONST *from = (const uint64_t NSQ_CONST *)__builtin_amdgcn_kernarg_segment_ptr();
    uint64_t *to = reinterpret_cast<uint64_t *>(a.to);
    for (int i = threadIdx.x; i < a.n * (int)(sizeof(Entry) / 8); i += kThreads) to[i] = from[i];
}

__device__ inline const Entry NSQ_CONST *table_of(const ClipArgs &a) {
    if (a.table) return (const Entry NSQ_CONST *)a.table;
    return (const Entry NSQ_CONST *)__builtin_amdgcn_kernarg_segment_ptr();
}

__device__ inline Entry entry(const Entry NSQ_CONST *t) { return {t->g, t->m, t->o, t->count, t->first, t->kind, t->lg}; }

// The last entry whose first chunk is at most c.
__device__ inline int find(const Entry NSQ_CONST *t, int n, int c) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t[mid].first <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Calls f(entry, first element, end) for the chunks of one part of `parts`.
template <typename F>
__device__ inline void each_chunk(const ClipArgs &a, int part, int parts, const F &f) {
    const Entry NSQ_CONST *t = table_of(a);
    const int from = (int)((int64_t)a.chunks * part / parts);
    const int to = (int)((int64_t)a.chunks * (part + 1) / parts);
    if (from >= to) return;
    int at = find(t, a.n, from);
    Entry e = entry(t + at);
    int next = at + 1 < a.n ? t[at + 1].first : a.chunks;
    for (int c = from; c < to; ++c) {
        while (c >= next) {   // tensors without elements have no chunk
            ++at;
            e = entry(t + at);
            next = at + 1 < a.n ? t[at + 1].first : a.chunks;
        }
        const int64_t begin = (int64_t)(c - e.first) << e.lg;
        f(e, begin, min(begin + ((int64_t)1 << e.lg), e.count));
    }
}

// Sums of squares -------------------------------------------------------------

// Adds the squares of elements [begin, end), a chunk, dealt to `WIDTH` lanes.
template <typename T, int WIDTH>
__device__ inline void add_squares(const T *g, int64_t begin, int64_t end, int lane, double &sum) {
    constexpr int V = Vec16<T>::N, AT_ONCE = WIDTH == 64 ? 8 : 2;
    const int whole = (int)(end - begin) / V;
    const T *p = g + begin;
    const int tail = whole * V + lane;   // fewer than V, so lanes 0 .. V - 1
    const float last = tail < end - begin ? (float)p[tail] : 0.f;
    for (int i = lane; i < whole; i += AT_ONCE * WIDTH) {
        typename Vec16<T>::raw v[AT_ONCE];
#pragma unroll
        for (int n = 0; n < AT_ONCE; ++n) v[n] = load_vec(p + (i + n * WIDTH < whole ? i + n * WIDTH : i) * V);
#pragma unroll
        for (int n = 0; n < AT_ONCE; ++n) {
            if (n && i + n * WIDTH >= whole) break;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const double x = elem<T>(v[n], k);
                sum = __builtin_fma(x, x, sum);
            }
        }
    }
    sum = __builtin_fma((double)last, (double)last, sum);
}

template <int THREADS>
__device__ inline double block_sum(double v) {
    __shared__ double part[THREADS / 64];
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.0;
    for (int i = 0; i < THREADS / 64; ++i) s += part[i];
    return s;
}

__device__ inline void write_norm(const ClipArgs &a, double sum) {
    if (a.norm) *a.norm = (float)sqrt(sum);
    if (a.sum_sq) *a.sum_sq = sum;
}

// SOLO: one workgroup for everything, a run of chunks to each wave, and it writes the norm itself.
template <bool SOLO>
__global__ __launch_bounds__(SOLO ? kSoloThreads : kThreads) void grad_sum_kernel(ClipArgs a) {
    constexpr int THREADS = SOLO ? kSoloThreads : kThreads, WIDTH = SOLO ? 64 : kThreads;
    const int lane = threadIdx.x % WIDTH;
    const int part = SOLO ? __builtin_amdgcn_readfirstlane(threadIdx.x / 64) : blockIdx.x;
    double sum = 0.0;
    each_chunk(a, part, SOLO ? kSoloThreads / 64 : gridDim.x, [&](const Entry &e, int64_t begin, int64_t end) {
        if (e.kind & 1) add_squares<float, WIDTH>(reinterpret_cast<const float *>(e.g), begin, end, lane, sum);
        else add_squares<__bf16, WIDTH>(reinterpret_cast<const __bf16 *>(e.g), begin, end, lane, sum);
    });
    sum = block_sum<THREADS>(sum);
    if (threadIdx.x) return;
    if constexpr (SOLO) write_norm(a, sum);
    else a.partial[blockIdx.x] = sum;
}

__global__ __launch_bounds__(kThreads) void grad_join_kernel(ClipArgs a, int blocks) {
    double sum = 0.0;
#pragma unroll
    for (int k = 0; k < kMaxBlocks / kThreads; ++k) {
        const int i = k * kThreads + threadIdx.x;
        if (i < blocks) sum += a.partial[i];
    }
    sum = block_sum<kThreads>(sum);
    if (threadIdx.x == 0) write_norm(a, sum);
}

// Clipping ----------------------------------------------------------------------

// out = beta m + c g of elements [begin, end): eight elements a thread where both are bf16, else four.
template <typename G, typename O, bool MOM, bool NT>
__device__ inline void clip_run(const Entry &e, int64_t begin, int64_t end, float c, float beta) {
    constexpr int V = sizeof(G) == 2 && sizeof(O) == 2 ? 8 : 4;
    const G *g = reinterpret_cast<const G *>(e.g);
    const O *m = reinterpret_cast<const O *>(e.m);
    O *o = reinterpret_cast<O *>(e.o);
    const int64_t whole = (end - begin) / V;
    for (int64_t i = threadIdx.x; i < whole; i += 2 * kThreads) {
        const bool two = i + kThreads < whole;
        const int64_t at = begin + i * V, bt = two ? at + kThreads * V : at;
        const auto g0 = Elems<G, V>::template load<NT>(g + at), g1 = Elems<G, V>::template load<NT>(g + bt);
        typename Elems<O, V>::raw m0, m1;
        if constexpr (MOM) m0 = Elems<O, V>::template load<NT>(m + at), m1 = Elems<O, V>::template load<NT>(m + bt);
        float x[V], y[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            x[k] = c * Elems<G, V>::at(g0, k);
            y[k] = c * Elems<G, V>::at(g1, k);
            if constexpr (MOM) x[k] += beta * Elems<O, V>::at(m0, k), y[k] += beta * Elems<O, V>::at(m1, k);
        }
        Elems<O, V>::template store<NT>(o + at, x);
        if (two) Elems<O, V>::template store<NT>(o + bt, y);
    }
    const int64_t tail = begin + whole * V + threadIdx.x;
    if (tail < end) {
        float x = c * (float)g[tail];
        if constexpr (MOM) x += beta * (float)m[tail];
        o[tail] = (O)x;
    }
}

template <bool MOM, bool NT>
__global__ __launch_bounds__(kThreads) void grad_clip_kernel(ClipArgs a) {
    float c = 1.f;
    if (a.norm_in) {
        const float r = a.max_norm / (*a.norm_in + a.eps);
        c = r >= 1.f ? 1.f : r;   // a NaN stays
    }
    each_chunk(a, blockIdx.x, gridDim.x, [&](const Entry &e, int64_t begin, int64_t end) {
        if (!MOM && c == 1.f && e.g == e.o) return;   // in place and unchanged
        switch (e.kind) {
            case 0: return clip_run<__bf16, __bf16, MOM, NT>(e, begin, end, c, a.beta);
            case 1: return clip_run<float, __bf16, MOM, NT>(e, begin, end, c, a.beta);
            case 2: return clip_run<__bf16, float, MOM, NT>(e, begin, end, c, a.beta);
            default: return clip_run<float, float, MOM, NT>(e, begin, end, c, a.beta);
        }
    });
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

constexpr size_t kPartialBytes = kMaxBlocks * sizeof(double);

size_t table_bytes(int32_t n) { return n > kInline ? ((size_t)n * sizeof(Entry) + 255) / 256 * 256 : 0; }

struct ClipCall {
    ClipArgs a{};
    int64_t bytes = 0;   // read and written
    double grad_bytes = 0;
};

ns_status check_tensor(const char *what, int32_t i, const void *p, int64_t count, int32_t dtype) {
    if (!dtype_bytes(dtype)) return fail(NS_ERR_DTYPE, "%s %d: dtype %d is not NS_BF16 or NS_F32", what, i, dtype);
    if (count && !p) return fail(NS_ERR_INVALID_ARG, "%s %d is NULL", what, i);
    if (misaligned(p, dtype_bytes(dtype))) return fail(NS_ERR_INVALID_ARG, "%s %d not aligned to its type", what, i);
    return NS_OK;
}

// Checks a list and lays out its table: in the arguments, or (more than kInline
// tensors) later in the workspace. Chunks of 2048 elements, 4096 where all are bf16.
ns_status check_list(int32_t n, const int64_t *counts, const void *const *grads, const int32_t *grad_dtypes,
                     const void *const *momenta, void *const *outs, const int32_t *out_dtypes, bool momentum,
                     void *workspace, size_t workspace_bytes) {
    if (n < 0 || n > kMaxTensors) return fail(NS_ERR_INVALID_ARG, "n = %d outside [0, %d]", n, kMaxTensors);
    if (n && (!counts || !grads || !grad_dtypes)) return fail(NS_ERR_INVALID_ARG, "counts, grads and grad_dtypes are required");
    if (n && outs && !out_dtypes) return fail(NS_ERR_INVALID_ARG, "out_dtypes is NULL");
    if (n && momentum && !momenta) return fail(NS_ERR_INVALID_ARG, "momenta is NULL");
    int64_t chunks = 0;
    for (int32_t i = 0; i < n; ++i) {
        if (counts[i] < 0) return fail(NS_ERR_INVALID_ARG, "counts[%d] < 0", i);
        if (counts[i] > (int64_t(1) << 41)) return fail(NS_ERR_OVERFLOW, "counts[%d] above 2^41", i);
        if (ns_status s = check_tensor("gradient", i, grads[i], counts[i], grad_dtypes[i])) return s;
        if (outs) {
            if (ns_status s = check_tensor("output", i, outs[i], counts[i], out_dtypes[i])) return s;
            if (momentum)
                if (ns_status s = check_tensor("momentum", i, momenta[i], counts[i], out_dtypes[i])) return s;
            if (counts[i] && outs[i] == grads[i] && out_dtypes[i] != grad_dtypes[i])
                return fail(NS_ERR_INVALID_ARG, "output %d is its gradient in another type", i);
        }
        chunks += (counts[i] + 2047) / 2048;
    }
    if (chunks >= INT32_MAX) return fail(NS_ERR_OVERFLOW, "more than 2^42 elements in all");
    const size_t need = table_bytes(n) + kPartialBytes;
    if (n && (!workspace || workspace_bytes < need))
        return fail(NS_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : 0, need);
    if (misaligned(workspace, 256)) return fail(NS_ERR_INVALID_ARG, "workspace not 256-byte aligned");
    return NS_OK;
}

// Lays out the table of a checked list, in the arguments or by launches into the workspace.
ns_status lay_out(int32_t n, const int64_t *counts, const void *const *grads, const int32_t *grad_dtypes,
                  const void *const *momenta, void *const *outs, const int32_t *out_dtypes, bool momentum,
                  void *workspace, hipStream_t st, ClipCall *c) {
    ClipArgs &a = c->a;
    a.partial = reinterpret_cast<double *>(workspace);
    Entry *table = reinterpret_cast<Entry *>(reinterpret_cast<char *>(workspace) + kPartialBytes);
    a.table = n > kInline ? table : nullptr;
    a.n = n;
    TableArgs part;
    int64_t chunks = 0;
    for (int32_t i = 0; i < n; ++i) {
        Entry &e = n > kInline ? part.part[i % kInline] : a.inline_table[i];
        const bool gf = grad_dtypes[i] == NS_F32, of = outs && out_dtypes[i] == NS_F32;
        e.g = reinterpret_cast<const char *>(grads[i]);
        e.m = momentum ? reinterpret_cast<const char *>(momenta[i]) : nullptr;
        e.o = outs ? reinterpret_cast<char *>(outs[i]) : nullptr;
        e.count = counts[i];
        e.first = (int32_t)chunks;
        e.kind = (int16_t)((gf ? 1 : 0) | (of ? 2 : 0));
        e.lg = gf || of ? 11 : 12;
        chunks += (counts[i] + ((int64_t)1 << e.lg) - 1) >> e.lg;
        c->grad_bytes += (double)counts[i] * (gf ? 4 : 2);
        c->bytes += counts[i] * ((gf ? 4 : 2) + (outs ? (of ? 4 : 2) * (momentum ? 2 : 1) : 0));
        if (n > kInline && (i + 1 == n || i % kInline == kInline - 1)) {
            part.n = i % kInline + 1;
            part.to = table + (i - i % kInline);
            hipLaunchKernelGGL(grad_table_kernel, dim3(1), dim3(kThreads), 0, st, part);
            NSQ_HIP(hipGetLastError());
        }
    }
    a.chunks = (int32_t)chunks;
    return NS_OK;
}

}  // namespace
}  // namespace nsq

using namespace nsq;

extern "C" ns_status ns_grad_workspace_bytes(int32_t n, size_t *bytes) {
    if (!bytes) return fail(NS_ERR_INVALID_ARG, "bytes is NULL");
    if (n < 0 || n > kMaxTensors) return fail(NS_ERR_INVALID_ARG, "n = %d outside [0, %d]", n, kMaxTensors);
    *bytes = table_bytes(n) + kPartialBytes;
    return NS_OK;
}

extern "C" ns_status ns_grad_norm(int32_t n, const int64_t *counts, const void *const *grads, const int32_t *grad_dtypes,
                                  float *norm, double *sum_sq, void *workspace, size_t workspace_bytes, void *stream) {
    if (ns_status s = check_list(n, counts, grads, grad_dtypes, nullptr, nullptr, nullptr, false, workspace, workspace_bytes))
        return s;
    if (!norm && !sum_sq) return fail(NS_ERR_INVALID_ARG, "norm or sum_sq is required");
    if (misaligned(norm, 4) || misaligned(sum_sq, 8)) return fail(NS_ERR_INVALID_ARG, "norm or sum_sq not aligned to its type");
    ClipCall c;
    hipStream_t st = as_stream(stream);
    if (ns_status s = lay_out(n, counts, grads, grad_dtypes, nullptr, nullptr, nullptr, false, workspace, st, &c)) return s;
    c.a.norm = norm;
    c.a.sum_sq = sum_sq;
    if (c.grad_bytes <= kSoloBytes) {
        hipLaunchKernelGGL(grad_sum_kernel<true>, dim3(1), dim3(kSoloThreads), 0, st, c.a);
    } else {
        const int blocks = std::min(c.a.chunks, kMaxBlocks);
        hipLaunchKernelGGL(grad_sum_kernel<false>, dim3(blocks), dim3(kThreads), 0, st, c.a);
        NSQ_HIP(hipGetLastError());
        hipLaunchKernelGGL(grad_join_kernel, dim3(1), dim3(kThreads), 0, st, c.a, blocks);
    }
    NSQ_HIP(hipGetLastError());
    return NS_OK;
}

extern "C" ns_status ns_grad_clip(int32_t n, const int64_t *counts, const void *const *grads, const int32_t *grad_dtypes,
                                  const void *const *momenta, void *const *outs, const int32_t *out_dtypes,
                                  const float *norm, float max_norm, float eps, float beta, void *workspace,
                                  size_t workspace_bytes, void *stream) {
    const bool momentum = beta != 0.f;
    if (!(beta >= -3.4e38f && beta <= 3.4e38f)) return fail(NS_ERR_INVALID_ARG, "beta must be finite");
    if (n > 0 && !outs) return fail(NS_ERR_INVALID_ARG, "outs is NULL");
    if (ns_status s = check_list(n, counts, grads, grad_dtypes, momenta, outs, out_dtypes, momentum, workspace, workspace_bytes))
        return s;
    if (norm) {
        if (misaligned(norm, 4)) return fail(NS_ERR_INVALID_ARG, "norm not 4-byte aligned");
        if (!(max_norm >= 0.f)) return fail(NS_ERR_INVALID_ARG, "max_norm must be >= 0");
        if (!(eps >= 0.f) || eps > 3.4e38f) return fail(NS_ERR_INVALID_ARG, "eps must be finite and >= 0");
    }
    ClipCall c;
    hipStream_t st = as_stream(stream);
    if (ns_status s = lay_out(n, counts, grads, grad_dtypes, momenta, outs, out_dtypes, momentum, workspace, st, &c)) return s;
    c.a.norm_in = norm;
    c.a.max_norm = max_norm;
    c.a.eps = eps;
    c.a.beta = beta;
    const int blocks = std::min(c.a.chunks, kMaxBlocks);
    if (!blocks) return NS_OK;
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(blocks), dim3(kThreads), 0, st, c.a); };
    // More than the last-level cache holds goes past it: 0.41 GB in 64 tensors 84 us, 90 without.
    const bool past = c.bytes > kMallBytes;
    if (momentum) past ? go(grad_clip_kernel<true, true>) : go(grad_clip_kernel<true, false>);
    else past ? go(grad_clip_kernel<false, true>) : go(grad_clip_kernel<false, false>);
    NSQ_HIP(hipGetLastError());
    return NS_OK;
}
