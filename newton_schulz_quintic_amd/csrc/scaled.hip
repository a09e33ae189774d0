// 8-bit matrix products with a power-of-two scale for each block of 128 along the
// reduction, and the quantization that makes their operands.
//
// A value v of a block is held as e4m3(v / 2^e), with e the smallest whole number
// for which the block's largest magnitude over 2^e is at most 448 (e4m3's
// largest), and e + 127 in one byte. Dividing by a power of two is exact, so a
// value is rounded once. Product, for a block index kb and its 128 values of k:
//   out[m, n] = sum over kb of 2^(sa[m, kb] - 127) 2^(sb[n, kb] - 127) sum over k of a[m, k] b[n, k].
// bf16 outputs: the scales go into the matrix instruction
// (v_mfma_scale_f32_16x16x128_f8f6f4), which takes such a byte for each row of both
// operands: a block of 128 is one instruction, its sum is added to the fp32
// accumulator scaled, and no value is touched outside it.
// fp32 outputs: the 8-bit instructions (all three shapes alike) align the products
// of a block to the largest and drop bits below some 2^-13 of it; measured against
// 64 bits, sums come out 1.4e-5 of their rms off where the values of a block are
// normally distributed, 7e-5 where they spread over 2^12. Next to bf16's rounding
// (1.7e-3) that is nothing; where fp32 is asked for it is not. There the values are
// widened to bf16, scale included (one conversion for two values, exact within bf16's
// normal range: from blocks that hold only values under 5e-36 it can lose some), and go
// through v_mfma_f32_16x16x32_bf16, whose sums are as good as fp32 adds (2e-8 to
// 1e-7 here), at half the peak.

#include <algorithm>

#include "elems.h"

namespace nsq {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
#define NSQ_LDS __attribute__((address_space(3)))

constexpr int kBlock = 128;        // values of one scale
constexpr int kMaxGroups = 1024;
constexpr int kNumXcd = 8;
constexpr int64_t kMaxRows = int64_t(1) << 30, kMaxCols = 1 << 22;

__device__ inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Groups of rows ---------------------------------------------------------------

// Row group e is offsets[e] .. offsets[e + 1], cut to [0, rows).
__device__ inline int edge(const int32_t *offsets, int e, int rows) { return min(max(offsets[e], 0), rows); }

// The groups' rows in blocks of `unit`, numbered through: the group, its rows and the
// place in it of block target_of(total) (group -1: there is no such block), or with
// BY_GROUP the number of group `target`'s first block. A wave's lanes take a run of
// groups each, so this is a short chain of loads and one scan. Edges out of order give
// wrong blocks, but none outside the rows (a lane's sum is cut before the scan could
// overflow).
struct GroupBlock {
    int group, index, total, begin, end;
};
template <bool BY_GROUP, class F>
__device__ inline GroupBlock find_block(const int32_t *offsets, int groups, int rows, int unit, const F &target_of) {
    const int lane = threadIdx.x & 63, per = (groups + 63) / 64;
    const int from = min(lane * per, groups), to = min(from + per, groups);
    int sum = 0;
    for (int e = from; e < to; ++e) sum = min(sum + (max(edge(offsets, e + 1, rows) - edge(offsets, e, rows), 0) + unit - 1) / unit, 1 << 24);
    int upto = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(upto, d);
        if (lane >= d) upto += v;
    }
    GroupBlock r;
    r.total = uniform(__shfl(upto, 63));
    const int target = target_of(r.total);
    const bool mine = BY_GROUP ? target >= from && target < to : target >= upto - sum && target < upto;
    int group = -1, index = 0, begin = 0, end = 0;
    if (mine) {
        int before = upto - sum;
        for (int e = from; e < to; ++e) {
            const int lo = edge(offsets, e, rows), hi = max(edge(offsets, e + 1, rows), lo), n = (hi - lo + unit - 1) / unit;
            if (BY_GROUP ? e == target : target < before + n) {
                group = e;
                index = BY_GROUP ? before : target - before;
                begin = lo;
                end = hi;
                break;
            }
            before += n;
        }
    }
    const uint64_t who = __ballot(mine);
    const int at = who ? __ffsll((unsigned long long)who) - 1 : 0;
    r.group = who ? __builtin_amdgcn_readlane(group, at) : -1;
    r.index = __builtin_amdgcn_readlane(index, at);
    r.begin = __builtin_amdgcn_readlane(begin, at);
    r.end = __builtin_amdgcn_readlane(end, at);
    return r;
}

// ---------------------------------------------------------------------------
// quantization
// ---------------------------------------------------------------------------

struct QuantArgs {
    const char *x;
    uint8_t *q, *s, *qt, *st;
    const int32_t *offsets;
    int64_t x_ld, x_batch, q_ld, q_batch, s_batch, qt_ld, qt_batch, st_batch;
    int rows, cols, groups;
    int nb, nbt;          // blocks of a row of q, of qt
};

// The exponent's byte for a block's largest magnitude, and the scale itself.
__device__ inline int scale_byte(float largest) {
    const uint32_t b = __builtin_bit_cast(uint32_t, largest);
    const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFF) > 0x600000);   // 448 = 1.75 x 2^8
    return largest > 0.f ? max(e, -126) + 127 : 127;
}
__device__ inline float scale_of(uint32_t byte) { return __builtin_bit_cast(float, (byte & 255) << 23); }

// Eight consecutive elements of a row. Those that reach past its end are loaded from
// its last eight and shifted into place by trim(), so that no load waits in a branch
// (14589 x 335 bf16, both ways: 16.0 us with loads one by one, 12.2). Magnitudes are
// taken of the finite ones: where any is not (a wave finds out at once), `strange`
// forms leave those out and turn infinities into NaN, which e4m3 has. Conversion
// divides by the scale and rounds to nearest even, two values an instruction.
template <typename T> struct Eight;
template <> struct Eight<__bf16> {
    uint32_t p[4];   // pairs
    __device__ inline void load(const __bf16 *row, int c, int cols) {
        if (cols >= 8) {
            typedef uint32_t u4 __attribute__((ext_vector_type(4)));
            const u4 v = __builtin_bit_cast(u4, load_vec(row + min(c, cols - 8)));
#pragma unroll
            for (int k = 0; k < 4; ++k) p[k] = v[k];
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint16_t *q = reinterpret_cast<const uint16_t *>(row);
                const uint32_t lo = c + 2 * k < cols ? q[c + 2 * k] : 0, hi = c + 2 * k + 1 < cols ? q[c + 2 * k + 1] : 0;
                p[k] = lo | hi << 16;
            }
        }
    }
    __device__ inline void trim(int c, int cols) {
        const int by = cols >= 8 ? c - (cols - 8) : 0;
        if (by <= 0) return;
        if (by & 4) p[0] = p[2], p[1] = p[3], p[2] = p[3] = 0;
        if (by & 2) p[0] = p[1], p[1] = p[2], p[2] = p[3], p[3] = 0;
        if (by & 1) {
#pragma unroll
            for (int k = 0; k < 4; ++k) p[k] = p[k] >> 16 | (k < 3 ? p[k + 1] << 16 : 0);
        }
        if (by >= 8) clear();
    }
    __device__ inline void clear() { p[0] = p[1] = p[2] = p[3] = 0; }
    typedef uint16_t pair __attribute__((ext_vector_type(2)));
    // the pair's magnitudes as 16-bit integers, which order as the values do
    __device__ inline pair size(int k, bool strange) const {
        pair m = __builtin_bit_cast(pair, p[k] & 0x7FFF7FFFu);
        if (strange) m = pair{(uint16_t)(m.x >= 0x7F80 ? 0 : m.x), (uint16_t)(m.y >= 0x7F80 ? 0 : m.y)};
        return m;
    }
    __device__ inline bool odd() const {
        const pair m = __builtin_elementwise_max(__builtin_elementwise_max(size(0, false), size(1, false)),
                                                 __builtin_elementwise_max(size(2, false), size(3, false)));
        return max(m.x, m.y) >= 0x7F80;
    }
    __device__ inline void mend() {   // infinities to NaN
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if ((p[k] & 0x7FFFu) == 0x7F80u) p[k] |= 0x7Fu;
            if ((p[k] & 0x7FFF0000u) == 0x7F800000u) p[k] |= 0x7F0000u;
        }
    }
    __device__ inline float largest(bool strange) const {
        const pair m = __builtin_elementwise_max(__builtin_elementwise_max(size(0, strange), size(1, strange)),
                                                 __builtin_elementwise_max(size(2, strange), size(3, strange)));
        return __builtin_bit_cast(float, (uint32_t)max(m.x, m.y) << 16);
    }
    static __device__ inline uint32_t four(uint32_t a, uint32_t b, float scale) {
        typedef short s2 __attribute__((ext_vector_type(2)));
        s2 v = {0, 0};
        v = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(v, __builtin_bit_cast(bf16x2, a), scale, false);
        v = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(v, __builtin_bit_cast(bf16x2, b), scale, true);
        return __builtin_bit_cast(uint32_t, v);
    }
    __device__ inline uint2 bytes(float scale) const { return {four(p[0], p[1], scale), four(p[2], p[3], scale)}; }
    // largest magnitudes of the columns of eight rows, and column k's bytes
    static __device__ inline void columns(const Eight (&v)[8], bool strange, float (&m)[8]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            pair c = v[0].size(k, strange);
#pragma unroll
            for (int i = 1; i < 8; ++i) c = __builtin_elementwise_max(c, v[i].size(k, strange));
            m[2 * k] = __builtin_bit_cast(float, (uint32_t)c.x << 16);
            m[2 * k + 1] = __builtin_bit_cast(float, (uint32_t)c.y << 16);
        }
    }
    static __device__ inline uint2 column(const Eight (&v)[8], int k, float scale) {
        uint32_t two[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            two[i] = __builtin_amdgcn_perm(v[2 * i + 1].p[k / 2], v[2 * i].p[k / 2], k & 1 ? 0x07060302 : 0x05040100);
        return {four(two[0], two[1], scale), four(two[2], two[3], scale)};
    }
};
template <> struct Eight<float> {
    float v[8];
    __device__ inline void load(const float *row, int c, int cols) {
        if (cols >= 8) {
            const int at = min(c, cols - 8);
            const auto lo = load_vec(row + at), hi = load_vec(row + at + 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = lo[k], v[4 + k] = hi[k];
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = c + k < cols ? row[c + k] : 0.f;
        }
    }
    __device__ inline void trim(int c, int cols) {
        const int by = cols >= 8 ? c - (cols - 8) : 0;
        if (by <= 0) return;
#pragma unroll
        for (int step = 4; step; step >>= 1)
            if (by & step) {
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = k + step < 8 ? v[k + step] : 0.f;
            }
        if (by >= 8) clear();
    }
    __device__ inline void clear() {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = 0.f;
    }
    __device__ inline float size(int k, bool strange) const {
        const float m = fabsf(v[k]);
        return !strange || m <= 3.402823466e38f ? m : 0.f;
    }
    __device__ inline bool odd() const {
        float m = 0.f;   // 0 x (infinity or NaN) is NaN
#pragma unroll
        for (int k = 0; k < 8; ++k) m = fmaf(0.f, v[k], m);
        return m != m;
    }
    __device__ inline void mend() {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (!(fabsf(v[k]) <= 3.402823466e38f)) v[k] = __builtin_nanf("");
    }
    __device__ inline float largest(bool strange) const {
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) m = fmaxf(m, size(k, strange));
        return m;
    }
    static __device__ inline uint32_t four(float a, float b, float c, float d, float scale) {
        typedef short s2 __attribute__((ext_vector_type(2)));
        s2 r = {0, 0};
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, a, b, scale, false);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c, d, scale, true);
        return __builtin_bit_cast(uint32_t, r);
    }
    __device__ inline uint2 bytes(float scale) const {
        return {four(v[0], v[1], v[2], v[3], scale), four(v[4], v[5], v[6], v[7], scale)};
    }
    static __device__ inline void columns(const Eight (&v)[8], bool strange, float (&m)[8]) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            m[k] = v[0].size(k, strange);
#pragma unroll
            for (int i = 1; i < 8; ++i) m[k] = fmaxf(m[k], v[i].size(k, strange));
        }
    }
    static __device__ inline uint2 column(const Eight (&v)[8], int k, float scale) {
        return {four(v[0].v[k], v[1].v[k], v[2].v[k], v[3].v[k], scale), four(v[4].v[k], v[5].v[k], v[6].v[k], v[7].v[k], scale)};
    }
};

__device__ inline float max16(float v) {   // over 16 neighbouring lanes
    return lanes_join<0, 4>(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ inline float max_rows(float v) {   // over the wave's four rows of 16 lanes
    uint32_t x = __builtin_bit_cast(uint32_t, v);
    const auto a = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    x = max(a[0], a[1]);   // magnitudes order as their bits
    const auto b = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return __builtin_bit_cast(float, max(b[0], b[1]));
}

// Rows only: 16 lanes take a block of 128 values, AT_ONCE blocks at a time. 8192 x
// 4096 bf16 18.3 us, 65536 x 7168 249 us (5.5 and 5.7 TB/s: memory).
template <typename T, int AT_ONCE>
__global__ __launch_bounds__(256) void quant_rows_kernel(QuantArgs a) {
    const int64_t units = (int64_t)a.rows * a.nb;
    const int lane = threadIdx.x & 15;
    const int64_t first = (int64_t)blockIdx.x * 16 * AT_ONCE + (threadIdx.x >> 4);
    Eight<T> v[AT_ONCE];
    int64_t row[AT_ONCE];
    int kb[AT_ONCE];
    bool odd = false;
#pragma unroll
    for (int n = 0; n < AT_ONCE; ++n) {
        const int64_t u = min(first + 16 * n, units - 1);
        row[n] = units >> 32 ? u / a.nb : (uint32_t)u / (uint32_t)a.nb;
        kb[n] = (int)(u - row[n] * a.nb);
        v[n].load(reinterpret_cast<const T *>(a.x) + row[n] * a.x_ld, kb[n] * kBlock + lane * 8, a.cols);
    }
#pragma unroll
    for (int n = 0; n < AT_ONCE; ++n) {
        v[n].trim(kb[n] * kBlock + lane * 8, a.cols);
        odd |= v[n].odd();
    }
    const bool strange = __any(odd);
    if (strange) {
#pragma unroll
        for (int n = 0; n < AT_ONCE; ++n) v[n].mend();
    }
#pragma unroll
    for (int n = 0; n < AT_ONCE; ++n) {
        const int byte = scale_byte(max16(v[n].largest(strange)));
        if (first + 16 * n >= units) return;
        *reinterpret_cast<uint2 *>(a.q + row[n] * a.q_ld + kb[n] * kBlock + lane * 8) = v[n].bytes(scale_of(byte));
        if (lane == 0) a.s[row[n] * a.nb + kb[n]] = (uint8_t)byte;
    }
}

// A tile of 128 x 128: a thread holds 8 x 8 values of it. SQUARE: one scale for
// the tile, for q and for qt; else one for each row (q) and one for each column (qt).
// The transpose goes through LDS, eight bytes (of a column) at a time: unit u of
// column c at u ^ (c / 8 & 14), which spreads a wave's writes over the banks. 14336 x
// 4096 bf16 in squares, both ways 40 us (5.8 TB/s); 8192 x 14336, both ways by row and
// column 95-110 us (4.3-4.9 TB/s), the transpose alone of 8192 x 4096 19 us (5.3). Loads
// past the cache took 101 us for the second and 258 in place of 247 for 16384 x 16384.
template <typename T, bool SQUARE>
__global__ __launch_bounds__(256) void quant_tile_kernel(QuantArgs a) {
    __shared__ __attribute__((aligned(16))) float part[4][kBlock];
    __shared__ __attribute__((aligned(16))) uint8_t turned[kBlock * kBlock];
    const int cb = blockIdx.x;
    const int lane = threadIdx.x & 15, down = threadIdx.x >> 4, wave = threadIdx.x >> 6;
    // rows [r0, end) go to columns t0 and on of qt
    int r0 = blockIdx.y * kBlock, end = min(r0 + kBlock, a.rows), t0 = r0;
    bool turn = a.qt != nullptr;
    if (a.offsets) {
        const GroupBlock g = find_block<false>(a.offsets, a.groups, a.rows, kBlock, [](int) { return (int)blockIdx.y; });
        if (g.group >= 0) {
            r0 = g.begin + g.index * kBlock;
            end = min(r0 + kBlock, g.end);
            turn = turn && t0 < a.nbt * kBlock;
        } else {   // rows in front of the first group, and those behind the last: they have no place in qt
            const int first = edge(a.offsets, 0, a.rows), front = (first + kBlock - 1) / kBlock, i = (int)blockIdx.y - g.total;
            r0 = i < front ? i * kBlock : edge(a.offsets, a.groups, a.rows) + (i - front) * kBlock;
            end = min(r0 + kBlock, i < front ? first : a.rows);
            turn = false;
            if (r0 >= end || !a.q) return;
        }
    }
    const T *x = reinterpret_cast<const T *>(a.x) + blockIdx.z * a.x_batch;
    const int c0 = cb * kBlock + lane * 8;
    Eight<T> v[8];
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + down * 8 + i;
        if (r < end) v[i].load(x + (int64_t)r * a.x_ld, c0, a.cols);
        else v[i].clear();
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i].trim(c0, a.cols);
        odd |= v[i].odd();
    }
    const bool strange = __any(odd);
    if (strange) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i].mend();
    }
    float square = 1.f;
    if constexpr (SQUARE) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, v[i].largest(strange));
        m = wave_max(m);
        if ((threadIdx.x & 63) == 0) part[0][wave] = m;
        __syncthreads();
        const int byte = scale_byte(fmaxf(fmaxf(part[0][0], part[0][1]), fmaxf(part[0][2], part[0][3])));
        square = scale_of(byte);
        if (threadIdx.x == 0) {
            if (a.s) a.s[blockIdx.z * a.s_batch + (int64_t)blockIdx.y * a.nb + cb] = (uint8_t)byte;
            if (a.st) a.st[blockIdx.z * a.st_batch + (int64_t)cb * a.nbt + blockIdx.y] = (uint8_t)byte;
        }
    }
    if (a.q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = r0 + down * 8 + i;
            float scale = square;
            if constexpr (!SQUARE) {
                const int b = scale_byte(max16(v[i].largest(strange)));
                scale = scale_of(b);
                if (lane == 0 && r < end) a.s[(int64_t)r * a.nb + cb] = (uint8_t)b;
            }
            if (r < end) *reinterpret_cast<uint2 *>(a.q + blockIdx.z * a.q_batch + r * a.q_ld + c0) = v[i].bytes(scale);
        }
    }
    if (!turn) return;
    float scale[8];
    if constexpr (SQUARE) {
#pragma unroll
        for (int k = 0; k < 8; ++k) scale[k] = square;
    } else {
        float m[8];
        Eight<T>::columns(v, strange, m);
#pragma unroll
        for (int k = 0; k < 8; ++k) m[k] = max_rows(m[k]);
        if ((threadIdx.x & 63) < 16) {
#pragma unroll
            for (int k = 0; k < 8; ++k) part[wave][lane * 8 + k] = m[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int c = lane * 8 + k;
            const int b = scale_byte(fmaxf(fmaxf(part[0][c], part[1][c]), fmaxf(part[2][c], part[3][c])));
            scale[k] = scale_of(b);
            if (down == 0 && cb * kBlock + c < a.cols) a.st[(int64_t)(cb * kBlock + c) * a.nbt + t0 / kBlock] = (uint8_t)b;
        }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        *reinterpret_cast<uint2 *>(turned + (lane * 8 + k) * kBlock + (down ^ (lane & 14)) * 8) = Eight<T>::column(v, k, scale[k]);
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int col = p * 32 + (threadIdx.x >> 3), piece = (threadIdx.x & 7) * 16;
        if (cb * kBlock + col >= a.cols) continue;
        const uint4 out = *reinterpret_cast<const uint4 *>(turned + col * kBlock + (piece ^ ((col >> 3 & 14) * 8)));
        *reinterpret_cast<uint4 *>(a.qt + blockIdx.z * a.qt_batch + (int64_t)(cb * kBlock + col) * a.qt_ld + t0 + piece) = out;
    }
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------

enum Grouping { kDense = 0, kRows = 1, kReduce = 2 };

struct MatArgs {
    const uint8_t *a, *as, *b, *bs;
    char *out;
    const int32_t *offsets;
    int64_t lda, ldb, ldo, b_batch, bs_batch, out_batch;
    int m, n, nkb;                 // rows of a, rows of b, blocks along the reduction
    int groups, rows;              // rows: what the groups divide (a's rows, or kReduce: tokens)
    int b_square, out_f32;
    int tiles_m, tiles_n;
    float *partial;                // with several splits of the reduction: [split][group][m][n]
    int splits;
};

// Tile of BM x BN computed by WM x WN waves; stages of one block (128 bytes a row) of both operands in two LDS buffers.
template <int BM_, int BN_, int WM_, int WN_> struct Tile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
    static constexpr int NM = BM / WM / 16, NN = BN / WN / 16;
    static constexpr int PANEL_A = BM * kBlock, PANEL_B = BN * kBlock, STAGE = PANEL_A + PANEL_B;
    static constexpr int LOADS_A = BM / WAVES / 8, LOADS_B = BN / WAVES / 8;   // 8 rows a wave load
};

// Panel row r sits at r * 128 bytes, its 16-byte chunk c at slot c ^ swz(r): the 16
// lanes of a fragment read (16 rows, one chunk each) hit distinct banks.
__device__ inline int swz(int r) { return (r >> 1) & 7; }

// Eight e4m3 values, bytes of two words, times a power of two, as bf16.
__device__ inline bf16x8 widen8(int lo, int hi, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

template <int N> __device__ inline void wait_vmcnt() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
}

// Workgroup id -> tile such that an XCD's workgroups (ids congruent mod 8) get a contiguous run.
__device__ inline int xcd_remap(int b, int g) {
    const int xcd = b % kNumXcd, local = b / kNumXcd, per = g / kNumXcd, rem = g % kNumXcd;
    return xcd < rem ? xcd * (per + 1) + local : rem * (per + 1) + (xcd - rem) * per + local;
}

// Tiles in runs of up to 8 rows of tiles, columns of tiles outside, so that neighbours share panels.
__device__ inline void place(int t, int tiles_m, int tiles_n, int *tm, int *tn) {
    constexpr int RUN = 8;
    const int band = t / (RUN * tiles_n), in = t - band * RUN * tiles_n;
    const int height = min(RUN, tiles_m - band * RUN);
    *tm = band * RUN + in % height;
    *tn = in / height;
}

// A workgroup's tile: rows [row0, row_end) of a (the tile's first row and the end of its
// group's), rows col0 .. of b, blocks [kb0, kb0 + nk) of the reduction.
struct Spot {
    int group, row0, row_end, col0, kb0, nk;
    bool any;
};
template <int GROUPING, int BM, int BN>
__device__ inline Spot locate(const MatArgs &p) {
    Spot s = {0, 0, p.m, 0, 0, p.nkb, true};
    int tm, tn;
    if constexpr (GROUPING == kRows) {
        int t = 0, all = 0;   // this workgroup's tile, the number of tiles
        const GroupBlock g = find_block<false>(p.offsets, p.groups, p.rows, BM, [&](int total) {
            all = min(total, (int)gridDim.x / p.tiles_n) * p.tiles_n;
            t = xcd_remap(blockIdx.x, max(all, 1));
            return (int)blockIdx.x < all ? t / p.tiles_n : -1;
        });
        s.any = (int)blockIdx.x < all && g.group >= 0;
        if (!s.any) return s;
        const int first = t / p.tiles_n - g.index;   // the group's first row of tiles
        s.group = g.group;
        s.row_end = g.end;
        place(t - first * p.tiles_n, (g.end - g.begin + BM - 1) / BM, p.tiles_n, &tm, &tn);
        s.row0 = g.begin + tm * BM;
    } else {
        const int per = p.tiles_m * p.tiles_n;
        const int t = xcd_remap(blockIdx.x, gridDim.x);
        s.group = t / per;
        place(t - s.group * per, p.tiles_m, p.tiles_n, &tm, &tn);
        s.row0 = tm * BM;
        if constexpr (GROUPING == kReduce) {
            const GroupBlock g = find_block<true>(p.offsets, p.groups, p.rows, kBlock, [&](int) { return s.group; });
            const int rows = g.end - g.begin;
            s.kb0 = g.index;
            s.nk = max(0, min((rows + kBlock - 1) / kBlock, p.nkb - s.kb0));
        }
    }
    s.col0 = tn * BN;
    return s;
}

// Scale words: the bytes of blocks 4 j .. 4 j + 3 of one row (nk of them in all). The
// last word of a row is loaded from four bytes before the row's end, never past it,
// and shifted by `tail_bits` when it is used. Rows at `base` + row[i].
__device__ inline int word_at(int j, int nk) { return min(4 * j, nk - 4); }
__device__ inline int tail_bits(int j, int nk) { return min(8 * (4 * j - word_at(j, nk)), 31); }
template <int N>
__device__ inline void load_words(const uint8_t *base, const int (&row)[N], int j, int nk, uint32_t (&w)[N]) {
    typedef uint32_t word_u __attribute__((aligned(1)));
    const int at = word_at(j, nk);
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = *reinterpret_cast<const word_u *>(base + (uint32_t)(row[i] + at));
}
// The first words, also of rows of fewer than four blocks.
template <int N>
__device__ inline void first_words(const uint8_t *base, const int (&row)[N], int nk, uint32_t (&w)[N]) {
    if (nk >= 4) return load_words(base, row, 0, nk, w);
    uint32_t b[3][N];
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) b[k][i] = base[(uint32_t)(row[i] + min(k, nk - 1))];
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = b[0][i] | b[1][i] << 8 | b[2][i] << 16;
}

// acc += the products of a block of 128 of 16 rows each, b's first; scales are the words' low bytes.
template <bool WIDE>
__device__ inline f32x4 multiply(i32x8 b, i32x8 a, f32x4 acc, uint32_t sb, uint32_t sa) {
    if constexpr (WIDE) {
#pragma unroll
        for (int g = 0; g < 4; ++g)
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(b[2 * g], b[2 * g + 1], scale_of(sb)),
                                                          widen8(a[2 * g], a[2 * g + 1], scale_of(sa)), acc, 0, 0, 0);
        return acc;
    } else {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, acc, 0, 0, 0, (int)sb, 0, (int)sa);
    }
}

// Up to four consecutive values of a row of the output.
template <bool WIDE>
__device__ inline void store4(char *out, int64_t at, f32x4 x, int left) {
    typedef typename std::conditional<WIDE, float, __bf16>::type O;
    O *to = reinterpret_cast<O *>(out) + at;
    float v[4] = {x[0], x[1], x[2], x[3]};
    if (left >= 4) return Elems<O, 4>::store(to, v);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (k < left) to[k] = (O)v[k];
}

// 128 x 128 a workgroup of four waves, two workgroups a CU, a block's loads under the
// block before. 4096 x 4096 -> 2048 bf16 37 us (1840 TFLOP/s). WIDE: fp32 output
// through bf16 products: 14336 x 8192 -> 4096 852 us (1130 TFLOP/s; 1205 on another
// GPU; a bf16 library product of 8192^3 1421). Two conversions stand beside each matrix
// instruction there and share its issue slots: instructions alone reach 1870 TFLOP/s,
// with their conversions 1410. 256 x 256 tiles of eight waves (1185), 128 x 256 (1220)
// and 256 x 128 (1096, 1205 for this) were no better. With one workgroup a CU a block
// takes some 0.6 us (bf16), with two stages of loads under way as with four.
template <int GROUPING, bool WIDE, class C>
__device__ __forceinline__ void scaled_tile(const MatArgs &p, char *lds) {
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), wm = wave / C::WN, wn = wave % C::WN;
    const Spot at = locate<GROUPING, C::BM, C::BN>(p);
    if (!at.any) return;
    const int row0 = at.row0, row_end = at.row_end, col0 = at.col0, group = at.group;
    // this workgroup's part of the reduction
    const int skip = at.nk * (int)blockIdx.y / p.splits, nk = at.nk * ((int)blockIdx.y + 1) / p.splits - skip;
    const int kb0 = at.kb0 + skip;
    const uint8_t *pa = p.a + row0 * p.lda + (int64_t)kb0 * kBlock;
    const uint8_t *pb = p.b + (GROUPING == kRows ? group * p.b_batch : 0) + col0 * p.ldb + (int64_t)kb0 * kBlock;
    const uint8_t *psb = p.bs + (GROUPING == kRows ? group * p.bs_batch : 0) + (int64_t)(p.b_square ? col0 / kBlock : col0) * p.nkb + kb0;
    // rows past the tile's last one are read as that one: their results are not stored
    const int ra = row_end - row0 - 1, rb = p.n - col0 - 1;
    const __amdgpu_buffer_rsrc_t rsa = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(pa), (short)0, -1, 0x00020000);
    const __amdgpu_buffer_rsrc_t rsb = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(pb), (short)0, -1, 0x00020000);
    int off_a[C::LOADS_A], off_b[C::LOADS_B];
#pragma unroll
    for (int i = 0; i < C::LOADS_A; ++i) {
        const int r = (wave * C::LOADS_A + i) * 8 + (lane >> 3);
        off_a[i] = min(r, ra) * (int)p.lda + (((lane & 7) ^ swz(r)) << 4);
    }
#pragma unroll
    for (int i = 0; i < C::LOADS_B; ++i) {
        const int r = (wave * C::LOADS_B + i) * 8 + (lane >> 3);
        off_b[i] = min(r, rb) * (int)p.ldb + (((lane & 7) ^ swz(r)) << 4);
    }
    const auto load_stage = [&](int kb, int buf) {
        char *base = lds + buf * C::STAGE;
#pragma unroll
        for (int i = 0; i < C::LOADS_A; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsa, (NSQ_LDS void *)(base + (wave * C::LOADS_A + i) * 1024), 16, off_a[i],
                                                     kb * kBlock, 0, 0);
#pragma unroll
        for (int i = 0; i < C::LOADS_B; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsb, (NSQ_LDS void *)(base + C::PANEL_A + (wave * C::LOADS_B + i) * 1024),
                                                     16, off_b[i], kb * kBlock, 0, 0);
    };
    // scale rows of this lane's fragments
    static_assert(C::BN % kBlock == 0, "whole square blocks");
    const uint8_t *psa = p.as + (int64_t)row0 * p.nkb + kb0;
    int sa_row[C::NM], sb_row[C::NN];
#pragma unroll
    for (int i = 0; i < C::NM; ++i) sa_row[i] = min((wm * C::NM + i) * 16 + (lane & 15), ra) * p.nkb;
#pragma unroll
    for (int j = 0; j < C::NN; ++j) {
        const int r = min((wn * C::NN + j) * 16 + (lane & 15), rb);
        sb_row[j] = (p.b_square ? r / kBlock : r) * p.nkb;
    }
    uint32_t sa[C::NM], sb[C::NN], next_a[C::NM], next_b[C::NN];
    f32x4 acc[C::NN][C::NM];
#pragma unroll
    for (int j = 0; j < C::NN; ++j)
#pragma unroll
        for (int i = 0; i < C::NM; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int frag = (lane & 15) * kBlock, fsw = swz(lane & 15);
    const int c0 = ((lane >> 4) ^ fsw) << 4, c1 = ((4 + (lane >> 4)) ^ fsw) << 4;
    const auto read = [&](const char *panel, int block) {
        const char *q = panel + block * 16 * kBlock + frag;
        const i32x4 lo = *reinterpret_cast<const i32x4 *>(q + c0), hi = *reinterpret_cast<const i32x4 *>(q + c1);
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    if (nk > 0) {
        first_words(psa, sa_row, nk, next_a);
        first_words(psb, sb_row, nk, next_b);
        load_stage(0, 0);
    }
    for (int kb = 0; kb < nk; ++kb) {
        if ((kb & 3) == 0) {   // four blocks' scales at a time, loaded four blocks ahead
#pragma unroll
            for (int i = 0; i < C::NM; ++i) sa[i] = next_a[i] >> (kb ? tail_bits(kb >> 2, nk) : 0);
#pragma unroll
            for (int j = 0; j < C::NN; ++j) sb[j] = next_b[j] >> (kb ? tail_bits(kb >> 2, nk) : 0);
            if (kb + 4 < nk) {
                load_words(psa, sa_row, (kb >> 2) + 1, nk, next_a);
                load_words(psb, sb_row, (kb >> 2) + 1, nk, next_b);
            }
        }
        wait_vmcnt<0>();
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (kb + 1 < nk) load_stage(kb + 1, (kb + 1) & 1);
        const char *panel_a = lds + (kb & 1) * C::STAGE + wm * C::NM * 16 * kBlock;
        const char *panel_b = lds + (kb & 1) * C::STAGE + C::PANEL_A + wn * C::NN * 16 * kBlock;
        // b first: a lane then holds four consecutive columns of one row
        if constexpr (WIDE) {
            bf16x8 fb[C::NN][4];
#pragma unroll
            for (int j = 0; j < C::NN; ++j) {
                const i32x8 f = read(panel_b, j);
#pragma unroll
                for (int g = 0; g < 4; ++g) fb[j][g] = widen8(f[2 * g], f[2 * g + 1], scale_of(sb[j]));
            }
#pragma unroll
            for (int i = 0; i < C::NM; ++i) {
                const i32x8 f = read(panel_a, i);
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const bf16x8 fa = widen8(f[2 * g], f[2 * g + 1], scale_of(sa[i]));
#pragma unroll
                    for (int j = 0; j < C::NN; ++j)
                        acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j][g], fa, acc[j][i], 0, 0, 0);
                }
            }
        } else {
            i32x8 fb[C::NN];
#pragma unroll
            for (int j = 0; j < C::NN; ++j) fb[j] = read(panel_b, j);
#pragma unroll
            for (int i = 0; i < C::NM; ++i) {
                const i32x8 fa = read(panel_a, i);
#pragma unroll
                for (int j = 0; j < C::NN; ++j)
                    acc[j][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[j], fa, acc[j][i], 0, 0, 0, (int)sb[j], 0, (int)sa[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < C::NM; ++i) sa[i] >>= 8;
#pragma unroll
        for (int j = 0; j < C::NN; ++j) sb[j] >>= 8;
    }
    // lane l of block (j, i): row l % 16 of block i, columns 4 (l / 16) .. + 4 of block j
    char *out = p.out + (GROUPING == kReduce ? group * p.out_batch * (WIDE ? 4 : 2) : 0);
    const int64_t part = (GROUPING == kReduce ? (int64_t)blockIdx.y * p.groups + group : blockIdx.y) * p.m * p.n;
#pragma unroll
    for (int i = 0; i < C::NM; ++i) {
        const int r = (wm * C::NM + i) * 16 + (lane & 15);
        if (r > ra) continue;
#pragma unroll
        for (int j = 0; j < C::NN; ++j) {
            const int c = col0 + (wn * C::NN + j) * 16 + 4 * (lane >> 4);
            if (p.splits > 1) store4<true>(reinterpret_cast<char *>(p.partial + part), (int64_t)(row0 + r) * p.n + c, acc[j][i], p.n - c);
            else store4<WIDE>(out, (row0 + r) * p.ldo + c, acc[j][i], p.n - c);
        }
    }
}

// Adds the splits' sums in order: four values of a row a thread. (A split to each wave of a workgroup and a sum over
// LDS took 1 us less for 32 splits of 256 x 256 values, 2 to 3 us more for few splits of more.)
template <int GROUPING, typename O>
__global__ __launch_bounds__(256) void scaled_join_kernel(MatArgs p) {
    const int parts = GROUPING == kReduce ? p.groups : 1;
    const int64_t all = (int64_t)parts * p.m * p.n;
    const int per = (p.n + 3) / 4;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = i / per;   // over all groups
    const int c = (int)(i - row * per) * 4;
    if (row >= (int64_t)parts * p.m) return;
    if (GROUPING == kRows && (row < edge(p.offsets, 0, p.rows) || row >= edge(p.offsets, p.groups, p.rows))) return;
    const int64_t at = row * p.n + c, group = row / p.m;
    O *out = reinterpret_cast<O *>(p.out) + group * p.out_batch + (row - group * p.m) * p.ldo + c;
    if (c + 4 <= p.n) {
        float v[4] = {};
#pragma unroll 4
        for (int s = 0; s < p.splits; ++s) {
            const auto x = load_vec(p.partial + s * all + at);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] += x[k];
        }
        Elems<O, 4>::store(out, v);
    } else {
        for (int k = 0; c + k < p.n; ++k) {
            float v = 0.f;
            for (int s = 0; s < p.splits; ++s) v += p.partial[s * all + at + k];
            out[k] = (O)v;
        }
    }
}

template <int GROUPING, bool WIDE, class C>
__global__ __launch_bounds__(C::THREADS) void scaled_tile_kernel(MatArgs p) {
    __shared__ __attribute__((aligned(16))) char lds[2 * C::STAGE];
    scaled_tile<GROUPING, WIDE, C>(p, lds);
}

// --- few rows ---------------------------------------------------------------------
// Up to 32 rows, as of tokens being decoded: bound by b's bytes, so every CU has to
// be reading. A workgroup takes NB blocks of 16 rows of b and all of a (MB blocks of
// 16 rows), its eight waves a run of blocks of the reduction each, straight from memory
// to registers (a wave's two loads of a block bring 128 bytes of each row); the
// waves' sums meet in LDS. a comes from the caches NB times less often than with
// one block of b. 16 x 4096 -> 14336 bf16 13 us (4.5 TB/s; what a CU can have under way
// at once is the bound, 27 bytes a ns), 16 x 8192 -> 20000 32 us, one row 4096 -> 4096 8.
constexpr int kRowsThreads = 512;
template <bool WIDE, int MB, int NB>
__global__ __launch_bounds__(kRowsThreads) void scaled_rows_kernel(MatArgs p) {
    // 16 waves: 16 x 4096 -> 1024 6.7 -> 6.8 us, 16 x 14336 -> 4096 17.7 -> 19.7, 32 x 6144 -> 2048 12.4 -> 15.4
    constexpr int W = kRowsThreads / 64;
    // blocks of the reduction whose loads a wave has under way together (four: 16 x 6144 -> 6144 15.4 -> 19.0 us)
    constexpr int AT_ONCE = MB + NB <= 4 ? 2 : 1;
    __shared__ f32x4 part[W][MB * NB][64];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), low = lane & 15;
    const int col0 = blockIdx.x * 16 * NB;
    const int k0 = p.nkb * wave / W, k1 = p.nkb * (wave + 1) / W;
    const uint8_t *a[MB], *sa[MB], *b[NB], *sb[NB];
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const int r = min(i * 16 + low, p.m - 1);
        a[i] = p.a + r * p.lda + (lane >> 4) * 16;
        sa[i] = p.as + (int64_t)r * p.nkb;
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        const int r = min(col0 + j * 16 + low, p.n - 1);
        b[j] = p.b + r * p.ldb + (lane >> 4) * 16;
        sb[j] = p.bs + (int64_t)(p.b_square ? r / kBlock : r) * p.nkb;
    }
    f32x4 acc[NB][MB];
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < MB; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int k = k0; k < k1; k += AT_ONCE) {
        i32x4 fb[AT_ONCE][NB][2], fa[AT_ONCE][MB][2];
        uint32_t wb[AT_ONCE][NB], wa[AT_ONCE][MB];
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
            const int at = min(k + u, k1 - 1);
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                fb[u][j][0] = *reinterpret_cast<const i32x4 *>(b[j] + (int64_t)at * kBlock);
                fb[u][j][1] = *reinterpret_cast<const i32x4 *>(b[j] + (int64_t)at * kBlock + 64);
                wb[u][j] = sb[j][at];
            }
#pragma unroll
            for (int i = 0; i < MB; ++i) {
                fa[u][i][0] = *reinterpret_cast<const i32x4 *>(a[i] + (int64_t)at * kBlock);
                fa[u][i][1] = *reinterpret_cast<const i32x4 *>(a[i] + (int64_t)at * kBlock + 64);
                wa[u][i] = sa[i][at];
            }
        }
        __builtin_amdgcn_sched_barrier(0);   // every load before the first product
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
            if (k + u >= k1) break;
#pragma unroll
            for (int j = 0; j < NB; ++j)
#pragma unroll
                for (int i = 0; i < MB; ++i)
                    acc[j][i] = multiply<WIDE>(__builtin_shufflevector(fb[u][j][0], fb[u][j][1], 0, 1, 2, 3, 4, 5, 6, 7),
                                               __builtin_shufflevector(fa[u][i][0], fa[u][i][1], 0, 1, 2, 3, 4, 5, 6, 7),
                                               acc[j][i], wb[u][j], wa[u][i]);
        }
    }
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < MB; ++i) part[wave][j * MB + i][lane] = acc[j][i];
    __syncthreads();
#pragma unroll
    for (int q = wave; q < MB * NB; q += W) {
        const int r = q % MB * 16 + low, c = col0 + q / MB * 16 + 4 * (lane >> 4);
        f32x4 sum = part[0][q][lane];
#pragma unroll
        for (int w = 1; w < W; ++w) sum += part[w][q][lane];
        if (r < p.m) store4<WIDE>(p.out, (int64_t)r * p.ldo + c, sum, p.n - c);
    }
}

// --- 256 x 256 tiles on four waves, accumulators in fixed registers -------------
// For bf16 outputs of calls with enough tiles to fill the GPU. Four waves of 128 x
// 128, one a SIMD, hold their 8 x 8 blocks of 16 x 16 in the AGPRs a0..a255 (the
// register allocator moves a tile of that size about inside the loop), and every
// MFMA is an inline-asm statement on its block's registers (acc_scaled.h). A block
// of 128 k is one stage, 32 KB a panel. The next stage's B fragments (64 registers)
// are read at the start of a stage, A fragments pass through four register sets as
// they are used. LDS holds three A panels and two B panels; with a barrier once the
// next B is read and one once this A is, panels three stages on are loaded as soon
// as their place is free, and have two (A) and 1.5 (B) stages to land
// (scaled_stage.inc). Stages past the last one are loaded and read as the last one
// and not used, so that the loop has one form.
// Measured: 8192 x 4096 -> 14336 385-410 us (2340-2500 TFLOP/s), 8192 x 14336 -> 4096
// 347 (2770), 8192^3 428 (2570): 80-84 % of the library's unscaled 8-bit product on the
// same GPU. A stage takes 1.39 us on all CUs (3.1 PFLOP/s; instructions alone, on
// random values, 3.77 at the clock that their power leaves) and a tile 7 us beside its
// stages, most of it the outputs of 256 tiles that end together. Timed for what the
// loads cost: 8192 x 14336 -> 4096 339 us, 320 with every load an L2 hit, 288 with none. Other orders of
// loads, reads and barriers within a stage were within 2 %, one barrier a stage 8 %
// slower; a workgroup that goes from tile to tile and stores from its registers took
// 3 % less at these sizes and 7 to 17 % more with rows at odd places or few tiles.
#include "acc_pinned.h"
#include "acc_scaled.h"

constexpr int kQuadThreads = 256, kQuadTile = 256;
constexpr int kQuadPanel = kQuadTile * kBlock;
constexpr int kQuadLds = 5 * kQuadPanel;
constexpr int kQuadPitch = kQuadTile * 2 + 16;   // of the output tile in LDS: rows on different banks

__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

template <int GROUPING, bool SQUARE>
__device__ __forceinline__ void scaled_quad(const MatArgs &__restrict__ p, char *lds) {
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), wm = wave >> 1, wn = wave & 1;
    const Spot at = locate<GROUPING, kQuadTile, kQuadTile>(p);
    if (!at.any) return;
    const int ra_last = at.row_end - at.row0 - 1, rb_last = p.n - at.col0 - 1, nk = at.nk;
    const uint8_t *pa = p.a + at.row0 * p.lda + (int64_t)at.kb0 * kBlock;
    const uint8_t *pb = p.b + (GROUPING == kRows ? at.group * p.b_batch : 0) + at.col0 * p.ldb + (int64_t)at.kb0 * kBlock;
    // a wave's 128 columns have one square block's scales, or each its own
    constexpr int NSB = SQUARE ? 1 : 8;
    const uint8_t *psa = p.as + (int64_t)at.row0 * p.nkb + at.kb0;
    const uint8_t *psb = p.bs + (GROUPING == kRows ? at.group * p.bs_batch : 0) +
                         (int64_t)(SQUARE ? at.col0 / kBlock : at.col0) * p.nkb + at.kb0;
    const __amdgpu_buffer_rsrc_t rsa = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(pa), (short)0, -1, 0x00020000);
    const __amdgpu_buffer_rsrc_t rsb = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(pb), (short)0, -1, 0x00020000);
    // Load n of a panel brings 8 rows: n < 4 the first halves of the two wave rows (rows 0 .. 63 and 128 .. 191), n >= 4 the others.
    const auto load_row = [&](int n) { return (wave >> 1) * 128 + (n >> 2) * 64 + ((wave & 1) * 4 + (n & 3)) * 8; };
    int off_a[8], off_b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = load_row(i) + (lane >> 3), chunk = ((lane & 7) ^ swz(r)) << 4;
        off_a[i] = min(r, ra_last) * (int)p.lda + chunk;
        off_b[i] = min(r, rb_last) * (int)p.ldb + chunk;
    }
    // this lane's rows in a's and b's scales
    struct Places {
        int a[8], b[NSB];
    };
    const auto places = [&]() {
        Places w;
        int l = lane & 15;
        asm volatile("" : "+v"(l));   // found again for each use: kept, they would take 16 registers
#pragma unroll
        for (int i = 0; i < 8; ++i) w.a[i] = min(wm * 128 + i * 16 + l, ra_last) * p.nkb;
#pragma unroll
        for (int i = 0; i < NSB; ++i) w.b[i] = (SQUARE ? min(wn, rb_last / kBlock) : min(wn * 128 + i * 16 + l, rb_last)) * p.nkb;
        return w;
    };
    char *const panel_b = lds + 3 * kQuadPanel;
    const auto load_a = [&](int n, int kb, int ring) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsa, (NSQ_LDS void *)(lds + ring * kQuadPanel + load_row(n) * kBlock), 16, off_a[n],
                                                 uniform(min(kb, nk - 1) * kBlock), 0, 0);
    };
    const auto load_b = [&](int n, int kb) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsb, (NSQ_LDS void *)(panel_b + (kb & 1) * kQuadPanel + load_row(n) * kBlock), 16,
                                                 off_b[n], uniform(min(kb, nk - 1) * kBlock), 0, 0);
    };
    const int fsw = swz(lane & 15), c0 = ((lane >> 4) ^ fsw) << 4, c1 = ((4 + (lane >> 4)) ^ fsw) << 4;
    const int frag_a = (wm * 128 + (lane & 15)) * kBlock, frag_b = (wn * 128 + (lane & 15)) * kBlock;
    const auto read = [&](const char *row, int block) {
        const i32x4 lo = *reinterpret_cast<const i32x4 *>(row + block * 16 * kBlock + c0);
        const i32x4 hi = *reinterpret_cast<const i32x4 *>(row + block * 16 * kBlock + c1);
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    if (GROUPING != kReduce || nk > 0) {   // only a group of rows may be empty
#pragma unroll
        for (int n = 0; n < 8; ++n) load_a(n, 0, 0), load_b(n, 0);
        uint32_t sa[8], sb_word[NSB], next_a[8], next_b[NSB];
        {
            const Places w = places();
            first_words(psa, w.a, nk, sa);
            first_words(psb, w.b, nk, sb_word);
#pragma unroll
            for (int i = 0; i < 8; ++i) next_a[i] = sa[i];
#pragma unroll
            for (int j = 0; j < NSB; ++j) next_b[j] = sb_word[j];
            if (nk > 4) {
                load_words(psa, w.a, 1, nk, next_a);
                load_words(psb, w.b, 1, nk, next_b);
            }
        }
#pragma unroll
        for (int n = 0; n < 8; ++n) load_b(n, 1);
#pragma unroll
        for (int n = 0; n < 8; ++n) load_a(n, 1, 1);
        pinned::zero();
        wait_vmcnt<8>();   // all but A's stage 1
        lds_barrier();
        i32x8 FA[4], FB[2][8];
#pragma unroll
        for (int j = 0; j < 8; ++j) FB[0][j] = read(panel_b + frag_b, j);
        FA[0] = read(lds + frag_a, 0);
        FA[1] = read(lds + frag_a, 1);
        FA[2] = read(lds + frag_a, 2);
        lds_barrier();   // every wave has stage 0's B fragments
#pragma unroll
        for (int n = 0; n < 8; ++n) load_b(n, 2);
#pragma unroll
        for (int n = 0; n < 8; ++n) load_a(n, 2, 2);
        int ring = 0;   // where stage kb's A panel is, and stage kb + 3's will be
        const auto stage = [&](auto par, int kb) {
            constexpr int PAR = decltype(par)::value;
            const int then = ring == 2 ? 0 : ring + 1;
            const char *now_a = lds + ring * kQuadPanel + frag_a, *then_a = lds + then * kQuadPanel + frag_a;
            const char *next_panel_b = panel_b + (PAR ^ 1) * kQuadPanel + frag_b;
            const auto sb = [&](int j) { return sb_word[SQUARE ? 0 : j]; };
            const auto ra = [&](int slot, int i) { FA[slot] = read(now_a, i); };
            const auto rna = [&](int slot, int i) { FA[slot] = read(then_a, i); };
            const auto rb = [&](int slot, int j) { FB[slot][j] = read(next_panel_b, j); };
            const auto la = [&](int n) { load_a(n, kb + 3, ring); };
            const auto lb = [&](int n) { load_b(n, kb + 3); };
#include "scaled_stage.inc"
            if ((kb & 3) == 3) {
#pragma unroll
                for (int i = 0; i < 8; ++i) sa[i] = next_a[i] >> tail_bits((kb + 1) >> 2, nk);
#pragma unroll
                for (int j = 0; j < NSB; ++j) sb_word[j] = next_b[j] >> tail_bits((kb + 1) >> 2, nk);
                if (kb + 5 < nk) {
                    const Places w = places();
                    load_words(psa, w.a, (kb + 5) >> 2, nk, next_a);
                    load_words(psb, w.b, (kb + 5) >> 2, nk, next_b);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) sa[i] >>= 8;
#pragma unroll
                for (int j = 0; j < NSB; ++j) sb_word[j] >>= 8;
            }
            ring = then;
        };
        int kb = 0;
        for (; kb + 1 < nk; kb += 2) {
            stage(std::integral_constant<int, 0>{}, kb);
            stage(std::integral_constant<int, 1>{}, kb + 1);
        }
        if (kb < nk) stage(std::integral_constant<int, 0>{}, kb);
        wait_vmcnt<0>();   // loads past the last stage
        pinned::drain();
    } else {
        pinned::zero();
    }
    lds_barrier();
    // Block q = 8 i + j: lane l has row l % 16 of row block i, columns 4 (l / 16) .. + 4 of column block j. The tile
    // goes through LDS and leaves in whole rows.
    typedef uint16_t h4 __attribute__((ext_vector_type(4)));
    pinned::each_block([&](auto qc, f32x4 v) {
        constexpr int i = decltype(qc)::value >> 3, j = decltype(qc)::value & 7;
        h4 h;
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = __builtin_bit_cast(uint16_t, (__bf16)v[k]);
        *reinterpret_cast<h4 *>(lds + (wm * 128 + i * 16 + (lane & 15)) * kQuadPitch + (wn * 128 + j * 16 + 4 * (lane >> 4)) * 2) = h;
    });
    lds_barrier();
    __bf16 *out = reinterpret_cast<__bf16 *>(p.out) + (GROUPING == kReduce ? at.group * p.out_batch : 0);
    const int c = (threadIdx.x & 31) * 8, rows = min(ra_last + 1, kQuadTile);
    typedef Elems<__bf16, 8> Out;
    __bf16 *to = out + (int64_t)at.row0 * p.ldo + at.col0 + c;
    // Stored past the caches, whose room a's and b's panels have use for: 256 groups of 256 rows, 7168 -> 2048 1035 -> 989
    // us, 32768 x 1024 -> 4096 171 -> 162.
    if (rows == kQuadTile && at.col0 + kQuadTile <= p.n) {
#pragma unroll 8
        for (int i = 0; i < 32; ++i) {
            const int r = i * 8 + (threadIdx.x >> 5);
            __builtin_nontemporal_store(*reinterpret_cast<const Out::raw *>(lds + r * kQuadPitch + c * 2),
                                        reinterpret_cast<Out::raw_u *>(to + r * p.ldo));
        }
        return;
    }
    for (int r = threadIdx.x >> 5; r < rows; r += 8) {
        const Out::raw v = *reinterpret_cast<const Out::raw *>(lds + r * kQuadPitch + c * 2);
        if (at.col0 + c + 8 <= p.n) {
            *reinterpret_cast<Out::raw_u *>(to + r * p.ldo) = v;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (at.col0 + c + k < p.n) to[r * p.ldo + k] = __builtin_bit_cast(__bf16, (uint16_t)v[k]);
        }
    }
}

template <int GROUPING, bool SQUARE>
__global__ __launch_bounds__(kQuadThreads, 1) void scaled_quad_kernel(MatArgs p) {
    __shared__ __attribute__((aligned(16))) char lds[kQuadLds];
    scaled_quad<GROUPING, SQUARE>(p, lds);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

// Whether scaled_rows_kernel takes a dense call. It has no second launch and no more workgroups than n gives; a long
// reduction over few columns, and over most with a second block of rows, is better cut into parts (splits_of). Cold
// weights, this kernel against the parts: 16 x 4096 -> 14336 15.1, 18.1 us; 16 x 8192 -> 4096 12.1, 14.1; 16 x 14336 ->
// 1024 19, 11.9; 32 x 4096 -> 14336 17.8, 19.5; 32 x 8192 -> 4096 17.1, 15.2; 32 x 14336 -> 4096 24.6, 18.8; 32 x 8192 ->
// 28672 46.8, 66.
bool few_rows(int64_t m, int64_t n, int64_t nkb) {
    return m <= 16 ? nkb <= 64 || n > 2048 : m <= 32 && (nkb <= 48 || n > 16384);
}

// Into how many parts the reduction is cut where 128-tiles are too few for the GPU: two workgroups a CU, and at least
// four blocks each (a workgroup takes some 0.6 us a block for bf16, 1 us for fp32, however many stages of loads are under
// way; the second launch 3 us and the parts' traffic). Without and with: 128 x 14336 -> 4096 82, 25 us; 256 x 65536 -> 256
// (fp32) 561, 28; 1024 x 8192 -> 1024 (fp32) 74, 31; 512 x 2048 -> 512 14, 11; but 1024 x 2048 -> 1024 14, 18. One tile
// for most CUs is cut in two where the reduction is long: 768 x 8192 -> 4096 49, 42 us; 896 x 14336 -> 4096 81, 67; but
// 896 x 4096 -> 4096 28, 32. With groups of rows there are at most m / 128 + groups tiles of rows, and no more than rows:
// 2 rows of 4 groups, 7808 -> 320 (fp32) 66, 13 us. Over groups of rows the longest group counts, taken as twice the average.
int splits_of(int64_t m, int64_t n, int64_t nkb, int32_t groups, int32_t reduce) {
    int64_t tiles = blocks_of(m) * blocks_of(n), depth = nkb;
    if (reduce) tiles *= groups, depth = 2 * nkb / groups;
    else if (groups) tiles = std::min(m, m / kBlock + groups) * blocks_of(n);
    else if (few_rows(m, n, nkb)) return 1;
    if (tiles == 0 || tiles > 256 || depth < (tiles >= 192 ? 64 : tiles > 48 ? 24 : 16)) return 1;
    return (int)std::max<int64_t>(1, std::min<int64_t>({depth / 4, 512 / tiles, 32}));
}
size_t partial_bytes(int64_t m, int64_t n, int64_t nkb, int32_t groups, int32_t reduce) {
    const int splits = splits_of(m, n, nkb, groups, reduce);
    return splits > 1 ? (size_t)splits * (reduce ? groups : 1) * m * n * sizeof(float) : 0;
}

// 256-tiles or 128-tiles, for bf16: by the rounds that each takes, in us at a depth of 4096 (measured within 3 us of this
// for 500 to 1300 small tiles). 512 of the small tiles are resident at once; a whole round of them takes 35 us, a last one
// of few 22 and up to 13 more. A round of 256 large ones takes 54 however few they are. With small, with large tiles: 2048
// x 4096 -> 4096 37, 51 us; -> 4352 60, 53; -> 8192 70, 56; -> 8300 93, 110; 64 x 4096 -> 70000 76, 105; 8192 x 4096 ->
// 14336 490, 393. Groups of rows are taken as equal: 64 groups of 128 rows, 4096 -> 4096 241, 279 us; of 187 365, 293.
// Other depths are not weighed (32000 x 640 -> 7744 234 us, floor 100).
bool quad_tiles(int64_t m, int64_t n, int32_t groups, int32_t reduce) {
    const int64_t copies = std::max(groups, 1), rows = groups && !reduce ? (m + groups - 1) / groups : m;
    const int64_t small = copies * blocks_of(rows) * blocks_of(n);
    const int64_t large = copies * ((rows + kQuadTile - 1) / kQuadTile) * ((n + kQuadTile - 1) / kQuadTile);
    const int64_t last = small % 512;
    return (large + 255) / 256 * 54 < small / 512 * 35 + (last ? 22 + last * 13 / 512 : 0);
}

// Whether one launch takes `groups` workgroups of `threads` along an axis: fewer than 2^32 threads.
ns_status check_grid(int64_t groups, int64_t threads) {
    if (groups > UINT32_MAX / threads) return fail(NS_ERR_OVERFLOW, "%lld workgroups are more than a launch takes", (long long)groups);
    return NS_OK;
}

// e4m3 rows: 16-byte aligned, whole blocks.
ns_status check_bytes(const char *name, const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t batch, int64_t batch_stride) {
    if (!p) return fail(NS_ERR_INVALID_ARG, "%s is NULL", name);
    if (misaligned(p, 16)) return fail(NS_ERR_INVALID_ARG, "%s not 16-byte aligned", name);
    if (ld < cols || ld % 16 || ld > (int64_t(1) << 22))
        return fail(NS_ERR_INVALID_ARG, "%s: rows %lld apart (a multiple of 16, at least %lld, at most 2^22)", name, (long long)ld,
                    (long long)cols);
    if (batch > 1 && (batch_stride < 0 || batch_stride % 16)) return fail(NS_ERR_INVALID_ARG, "%s: batch stride not a multiple of 16", name);
    if (batch > 1 && too_far(batch, batch_stride)) return fail(NS_ERR_OVERFLOW, "%s: offsets overflow", name);
    return NS_OK;
}

// Outputs: whether any two of `count` matrices of rows x cols values, `ld` and `stride` apart, share a place. Matrices may lie
// behind each other or between each other's rows. (cols <= ld; a matrix g further on has its row i where this one has row
// i + q, and r values behind it.)
bool overlap(int64_t count, int64_t stride, int64_t rows, int64_t ld, int64_t cols) {
    const int64_t extent = (rows - 1) * ld + cols;
    if (stride >= extent) return false;
    for (int64_t g = 1; g < count && g * stride < extent; ++g) {
        const int64_t q = g * stride / ld, r = g * stride % ld;
        if (r < cols || (q + 1 < rows && ld - r < cols)) return true;
    }
    return false;
}

// Blocks of 16 rows of b to a workgroup of scaled_rows_kernel. A CU brings some 27 bytes a ns to its registers, of a
// as of b, and a call ends with its busiest CU.
int row_blocks(int64_t n, int mb) {
    int best = 1;
    int64_t least = INT64_MAX;
    for (int nb = 1; nb <= 8; ++nb) {
        const int64_t groups = (n + 16 * nb - 1) / (16 * nb), cost = (groups + 255) / 256 * (nb + mb);
        if (cost < least) least = cost, best = nb;
    }
    return best;
}

ns_status launch_rows(const MatArgs &p, hipStream_t st) {
    const int mb = p.m <= 16 ? 1 : 2, nb = row_blocks(p.n, mb);
    const int64_t workgroups = ((int64_t)p.n + 16 * nb - 1) / (16 * nb);
    if (ns_status s = check_grid(workgroups, kRowsThreads)) return s;
    const dim3 grid((unsigned)workgroups);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(kRowsThreads), 0, st, p); };
    auto pick = [&](auto wide, auto mb) {
        constexpr bool WIDE = decltype(wide)::value;
        constexpr int MB = decltype(mb)::value;
        switch (nb) {
            case 1: return go(scaled_rows_kernel<WIDE, MB, 1>);
            case 2: return go(scaled_rows_kernel<WIDE, MB, 2>);
            case 3: return go(scaled_rows_kernel<WIDE, MB, 3>);
            case 4: return go(scaled_rows_kernel<WIDE, MB, 4>);
            case 5: return go(scaled_rows_kernel<WIDE, MB, 5>);
            case 6: return go(scaled_rows_kernel<WIDE, MB, 6>);
            case 7: return go(scaled_rows_kernel<WIDE, MB, 7>);
            default: return go(scaled_rows_kernel<WIDE, MB, 8>);
        }
    };
    typedef std::integral_constant<int, 1> One;
    typedef std::integral_constant<int, 2> Two;
    if (p.out_f32) mb == 1 ? pick(std::true_type{}, One{}) : pick(std::true_type{}, Two{});
    else mb == 1 ? pick(std::false_type{}, One{}) : pick(std::false_type{}, Two{});
    NSQ_HIP(hipGetLastError());
    return NS_OK;
}

template <int GROUPING> ns_status launch_tile(const MatArgs &p, int64_t grid, hipStream_t st) {
    typedef Tile<128, 128, 2, 2> T;
    const dim3 blocks((unsigned)grid, p.splits), threads(T::THREADS);
    if (p.out_f32) hipLaunchKernelGGL((scaled_tile_kernel<GROUPING, true, T>), blocks, threads, 0, st, p);
    else hipLaunchKernelGGL((scaled_tile_kernel<GROUPING, false, T>), blocks, threads, 0, st, p);
    NSQ_HIP(hipGetLastError());
    if (p.splits > 1) {
        const int64_t join_threads = (int64_t)(GROUPING == kReduce ? p.groups : 1) * p.m * ((p.n + 3) / 4);
        const dim3 join((unsigned)((join_threads + 255) / 256));
        if (p.out_f32) hipLaunchKernelGGL((scaled_join_kernel<GROUPING, float>), join, dim3(256), 0, st, p);
        else hipLaunchKernelGGL((scaled_join_kernel<GROUPING, __bf16>), join, dim3(256), 0, st, p);
        NSQ_HIP(hipGetLastError());
    }
    return NS_OK;
}

}  // namespace
}  // namespace nsq

using namespace nsq;

extern "C" ns_status ns_quantize(int64_t batch, int64_t rows, int64_t cols, ns_dtype dtype, const void *x, int64_t x_ld,
                                 int64_t x_batch, int32_t block_rows, const int32_t *offsets, int32_t groups, void *q,
                                 int64_t q_ld, int64_t q_batch, uint8_t *scales, void *qt, int64_t qt_ld, int64_t qt_batch,
                                 uint8_t *scales_t, void *stream) {
    const int es = dtype_bytes(dtype);
    if (!es) return fail(NS_ERR_DTYPE, "dtype %d is not NS_BF16 or NS_F32", dtype);
    if (batch < 0 || batch > 65535) return fail(NS_ERR_INVALID_ARG, "batch outside [0, 65535]");
    if (rows < 0 || rows > kMaxRows) return fail(NS_ERR_INVALID_ARG, "rows outside [0, 2^30]");
    if (cols < 1 || cols > kMaxCols) return fail(NS_ERR_INVALID_ARG, "cols outside [1, 2^22]");
    if (block_rows != 1 && block_rows != kBlock) return fail(NS_ERR_INVALID_ARG, "block_rows must be 1 or 128");
    if (block_rows == 1 && batch > 1) return fail(NS_ERR_INVALID_ARG, "a batch needs block_rows = 128");
    if (!batch || !rows) return NS_OK;   // no address is looked at: empty tensors have none
    if (!q != !scales || !qt != !scales_t || (!q && !qt))
        return fail(NS_ERR_INVALID_ARG, "q and scales, or qt and scales_t, or both pairs are required");
    if (!x) return fail(NS_ERR_INVALID_ARG, "x is NULL");
    if (misaligned(x, es)) return fail(NS_ERR_INVALID_ARG, "x not aligned to its type");
    if (x_ld < 0 || (batch > 1 && x_batch < 0)) return fail(NS_ERR_INVALID_ARG, "negative stride");
    if (too_far(rows, x_ld) || too_far(batch, x_batch) || rows * (double)x_ld + batch * (double)x_batch > 4.6e18 / es)
        return fail(NS_ERR_OVERFLOW, "x: offsets overflow");
    const int64_t nb = blocks_of(cols);
    int64_t nbt = blocks_of(rows);
    if (offsets) {
        if (block_rows != 1) return fail(NS_ERR_INVALID_ARG, "offsets need block_rows = 1");
        if (groups < 1 || groups > kMaxGroups) return fail(NS_ERR_INVALID_ARG, "groups = %d outside [1, %d]", groups, kMaxGroups);
        if (misaligned(offsets, 4)) return fail(NS_ERR_INVALID_ARG, "offsets not 4-byte aligned");
        nbt = rows / kBlock + groups;
    }
    if (q)
        if (ns_status s = check_bytes("q", q, rows, nb * kBlock, q_ld, batch, q_batch)) return s;
    if (qt)
        if (ns_status s = check_bytes("qt", qt, cols, nbt * kBlock, qt_ld, batch, qt_batch)) return s;
    if ((q && overlap(batch, q_batch, rows, q_ld, nb * kBlock)) || (qt && overlap(batch, qt_batch, cols, qt_ld, nbt * kBlock)))
        return fail(NS_ERR_INVALID_ARG, "matrices of q or of qt overlap");
    QuantArgs a{};
    a.x = reinterpret_cast<const char *>(x);
    a.x_ld = x_ld;
    a.x_batch = x_batch;
    a.q = reinterpret_cast<uint8_t *>(q);
    a.q_ld = q_ld;
    a.q_batch = q_batch;
    a.s = scales;
    a.s_batch = blocks_of(rows) * nb;
    a.qt = reinterpret_cast<uint8_t *>(qt);
    a.qt_ld = qt_ld;
    a.qt_batch = qt_batch;
    a.st = scales_t;
    a.st_batch = nb * nbt;
    a.offsets = qt ? offsets : nullptr;
    a.groups = groups;
    a.rows = (int)rows;
    a.cols = (int)cols;
    a.nb = (int)nb;
    a.nbt = (int)nbt;
    hipStream_t st = as_stream(stream);
    if (block_rows == 1 && !qt) {
        const int64_t units = rows * nb;
        // One block a group of lanes, four in large calls: 2048 x 4096 bf16 6.6 and 7.0 us, 8192 x 4096 18.4 both, 65536
        // x 7168 259 and 248.
        const bool few = units < 16 * 4 * 4096;
        const int64_t grid = (units + (few ? 16 : 64) - 1) / (few ? 16 : 64);
        if (ns_status s = check_grid(grid, 256)) return s;
        auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(256), 0, st, a); };
        if (dtype == NS_BF16) few ? go(quant_rows_kernel<__bf16, 1>) : go(quant_rows_kernel<__bf16, 4>);
        else few ? go(quant_rows_kernel<float, 1>) : go(quant_rows_kernel<float, 4>);
    } else {
        // for q with groups two rows of tiles more: the rows in front of the first and behind the last are two runs more to round up
        const int64_t down = a.offsets && q ? nbt + 2 : nbt;
        if (down > 65535) return fail(NS_ERR_OVERFLOW, "rows too many for qt or square blocks");
        const dim3 grid((unsigned)nb, (unsigned)down, (unsigned)batch);
        auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, a); };
        if (dtype == NS_BF16) block_rows == 1 ? go(quant_tile_kernel<__bf16, false>) : go(quant_tile_kernel<__bf16, true>);
        else block_rows == 1 ? go(quant_tile_kernel<float, false>) : go(quant_tile_kernel<float, true>);
    }
    NSQ_HIP(hipGetLastError());
    return NS_OK;
}

extern "C" ns_status ns_scaled_matmul_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t groups, size_t *bytes) {
    if (!bytes) return fail(NS_ERR_INVALID_ARG, "bytes is NULL");
    if (m < 0 || m > kMaxRows || n < 0 || n > kMaxRows) return fail(NS_ERR_INVALID_ARG, "m or n outside [0, 2^30]");
    if (k < 0 || k % kBlock || k > kMaxCols) return fail(NS_ERR_INVALID_ARG, "k must be a multiple of 128 up to 2^22");
    if (groups < 0 || groups > kMaxGroups) return fail(NS_ERR_INVALID_ARG, "groups = %d outside [0, %d]", groups, kMaxGroups);
    *bytes = partial_bytes(m, n, k / kBlock, groups, 0);
    if (groups) *bytes = std::max(*bytes, partial_bytes(m, n, k / kBlock, groups, 1));
    return NS_OK;
}

extern "C" ns_status ns_scaled_matmul(int64_t m, int64_t n, int64_t k, const void *a, int64_t a_ld, const uint8_t *a_scales,
                                      const void *b, int64_t b_ld, int64_t b_batch, const uint8_t *b_scales,
                                      int32_t b_block_rows, const int32_t *offsets, int32_t groups, int32_t reduce,
                                      int64_t rows, ns_dtype out_dtype, void *out, int64_t out_ld, int64_t out_batch,
                                      void *workspace, size_t workspace_bytes, void *stream) {
    const int es = dtype_bytes(out_dtype);
    if (!es) return fail(NS_ERR_DTYPE, "out_dtype %d is not NS_BF16 or NS_F32", out_dtype);
    size_t need;
    if (ns_status s = ns_scaled_matmul_workspace_bytes(m, n, k, groups, &need)) return s;
    if (b_block_rows != 1 && b_block_rows != kBlock) return fail(NS_ERR_INVALID_ARG, "b_block_rows must be 1 or 128");
    if (reduce != 0 && reduce != 1) return fail(NS_ERR_INVALID_ARG, "reduce must be 0 or 1");
    if (!offsets != !groups) return fail(NS_ERR_INVALID_ARG, "offsets and groups go together");
    if (reduce && !offsets) return fail(NS_ERR_INVALID_ARG, "reduce needs offsets");
    if (misaligned(offsets, 4)) return fail(NS_ERR_INVALID_ARG, "offsets not 4-byte aligned");
    if (need && (!workspace || workspace_bytes < need))
        return fail(NS_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : 0, need);
    if (misaligned(workspace, 256)) return fail(NS_ERR_INVALID_ARG, "workspace not 256-byte aligned");
    if (!m || !n) return NS_OK;
    if (!out || misaligned(out, es)) return fail(NS_ERR_INVALID_ARG, "out is NULL or not aligned to its type");
    if (out_ld < n || too_far(m, out_ld) || m * (double)out_ld > 1e18 || (reduce && groups > 1 && (out_batch < 0 || too_far(groups, out_batch * es))))
        return fail(NS_ERR_INVALID_ARG, "out: bad strides");
    if (reduce && overlap(groups, out_batch, m, out_ld, n)) return fail(NS_ERR_INVALID_ARG, "the groups' products overlap in out");
    if (k) {
        if (ns_status s = check_bytes("a", a, m, k, a_ld, 1, 0)) return s;
        if (ns_status s = check_bytes("b", b, n, k, b_ld, offsets && !reduce ? groups : 1, b_batch)) return s;
        if (!a_scales || !b_scales) return fail(NS_ERR_INVALID_ARG, "a_scales and b_scales are required");
    }
    if (reduce && (rows < 0 || rows / kBlock + groups < 0 || k < (rows / kBlock) * kBlock))
        return fail(NS_ERR_INVALID_ARG, "rows = %lld do not fit k", (long long)rows);
    MatArgs p{};
    p.a = reinterpret_cast<const uint8_t *>(a);
    p.as = a_scales;
    p.b = reinterpret_cast<const uint8_t *>(b);
    p.bs = b_scales;
    p.out = reinterpret_cast<char *>(out);
    p.offsets = offsets;
    p.lda = a_ld;
    p.ldb = b_ld;
    p.ldo = out_ld;
    p.b_batch = b_batch;
    p.m = (int)m;
    p.n = (int)n;
    p.nkb = (int)(k / kBlock);
    p.bs_batch = (b_block_rows == 1 ? n : blocks_of(n)) * p.nkb;
    p.out_batch = out_batch;
    p.groups = groups;
    p.rows = (int)(reduce ? rows : m);
    p.b_square = b_block_rows == kBlock;
    p.out_f32 = out_dtype == NS_F32;
    hipStream_t st = as_stream(stream);
    if (!offsets && few_rows(m, n, p.nkb)) return launch_rows(p, st);
    if (!p.out_f32 && k && !(reduce && p.b_square) && quad_tiles(m, n, groups, reduce)) {
        p.tiles_m = (int)((m + kQuadTile - 1) / kQuadTile);
        p.tiles_n = (int)((n + kQuadTile - 1) / kQuadTile);
        int64_t quads = (int64_t)p.tiles_m * p.tiles_n;
        if (offsets && !reduce) quads = (m / kQuadTile + groups) * p.tiles_n;
        if (reduce) quads *= groups;
        if (ns_status s = check_grid(quads, kQuadThreads)) return s;
        auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3((unsigned)quads), dim3(kQuadThreads), 0, st, p); };
        if (!offsets) p.b_square ? go(scaled_quad_kernel<kDense, true>) : go(scaled_quad_kernel<kDense, false>);
        else if (!reduce) p.b_square ? go(scaled_quad_kernel<kRows, true>) : go(scaled_quad_kernel<kRows, false>);
        else go(scaled_quad_kernel<kReduce, false>);
        NSQ_HIP(hipGetLastError());
        return NS_OK;
    }
    p.tiles_m = (int)blocks_of(m);
    p.tiles_n = (int)blocks_of(n);
    int64_t grid = (int64_t)p.tiles_m * p.tiles_n;
    if (offsets && !reduce) grid = std::min(m, m / kBlock + groups) * p.tiles_n;
    if (reduce) grid *= groups;
    p.splits = splits_of(m, n, p.nkb, groups, reduce);
    p.partial = reinterpret_cast<float *>(workspace);
    if (ns_status s = check_grid(grid, 256)) return s;
    if (!offsets) return launch_tile<kDense>(p, grid, st);
    return reduce ? launch_tile<kReduce>(p, grid, st) : launch_tile<kRows>(p, grid, st);
}
