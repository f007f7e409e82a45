// The operators between a decode step's quantized projections: rotary positions,
// appending keys and values to a paged 8-bit cache, and the attention over it
// (sm_100a).
//
// The cache.  Pages of P tokens; codes e4m3 [page][head][token][D], so that one
// head's part of a page is one contiguous tile; scales binary32
// [page][head][P / 16], one per block of 16 tokens and head, always a power of
// two 2^e with e in [-40, 40].  A floating code with power-of-two scales lets a
// block grow: when an appended token raises e by k, the earlier codes are
// multiplied by 2^-k, which is exact but for results below the code's least
// normal number, so tokens appended one by one end as a prompt appended at once but
// for such codes (integer codes would round again at every rise).  Keys also differ in size from
// channel to channel, where a floating code keeps the same relative error.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "awq_device.cuh"

namespace awq {
namespace kv {

constexpr unsigned kDevErrBadIndex = 16u;   // a page, position or length outside its array
constexpr int kBlock = 16;                  // tokens that share a scale
constexpr int kEMin = -40, kEMax = 40;      // exponents of the scales

enum : int { kF32 = 0, kF16 = 1, kBF16 = 2 };

struct Cache {
    uint8_t *codes[2];     // keys, values
    float *scales[2];
    int64_t n_pages;
    int page, heads, dim;  // tokens per page, heads, head dimension
};
struct Batch {
    const int32_t *seq_lens;   // [n_seqs] tokens in the cache, the new ones included
    const int32_t *cu;         // [n_seqs + 1] rows of the new tokens, or NULL: row b is sequence b's
    const int32_t *pages;      // [n_seqs][ld_pages]
    int64_t ld_pages, max_pages;
    int n_seqs;
};
struct Rows {
    const void *data;
    int64_t ld_tok, ld_head;
    int heads, dtype;
};
struct Rope {
    const float2 *table;       // [n_pos][rot / 2] cosine, sine
    int64_t n_pos;
    int rot, interleaved;
};

// New tokens of sequence b: rows [row0, row0 + n) at positions [start, start + n).
struct Seq {
    int row0, n;
    int64_t start;             // may be negative: those rows have no place in the cache
    int64_t len;               // start + n
};
// A sequence with more new tokens than `most` is an error: it is reported and has none.
__device__ __forceinline__ Seq seq_info(const Batch &B, int b, int64_t T, int most = 0x7fffffff) {
    Seq s;
    int64_t r0 = b, r1 = b + 1;
    if (B.cu) {
        r0 = B.cu[b];
        r1 = B.cu[b + 1];
    }
    if (r0 < 0) r0 = 0;
    if (r0 > T) r0 = T;
    if (r1 > T) r1 = T;
    s.row0 = (int)r0;
    s.n = r1 > r0 ? (int)(r1 - r0) : 0;
    if (s.n > most) {
        atomicOr(&g_dev_error, kDevErrBadIndex);
        s.n = 0;
    }
    const int64_t len = B.seq_lens[b];
    s.len = len < 0 ? 0 : len;
    s.start = s.len - s.n;
    return s;
}
// The sequence of row t (the last b with cu[b] <= t); -1 if it has none.
__device__ __forceinline__ int seq_of_row(const Batch &B, int64_t t) {
    if (!B.cu) return t < B.n_seqs ? (int)t : -1;
    int lo = 0, hi = B.n_seqs;             // cu[lo] <= t < cu[hi]
    if (t < B.cu[0] || t >= B.cu[hi]) return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (B.cu[mid] <= t) lo = mid; else hi = mid;
    }
    return lo;
}
// The page of `position`, or -1 (raising the error flag) if the table has none
// there or names one outside the pool.
__device__ __forceinline__ int64_t page_of(const Batch &B, const Cache &C, int b, int64_t position) {
    const int64_t i = position / C.page;
    if (i >= B.max_pages) {
        atomicOr(&g_dev_error, kDevErrBadIndex);
        return -1;
    }
    const int64_t p = B.pages[(int64_t)b * B.ld_pages + i];
    if (p < 0 || p >= C.n_pages) {
        atomicOr(&g_dev_error, kDevErrBadIndex);
        return -1;
    }
    return p;
}

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }
__device__ __forceinline__ int exponent_of(float scale) {      // of a power of two
    const int e = ((__float_as_int(scale) >> 23) & 255) - 127;
    return e < kEMin ? kEMin : (e > kEMax ? kEMax : e);
}
// The least e in [kEMin, kEMax] with amax <= 448 * 2^e (amax finite, >= 0):
// 448 = 1.75 * 2^8, so e = exponent(amax) - 8, one more if its fraction is above 1.75.
__device__ __forceinline__ int exponent_for(float amax) {
    const int bits = __float_as_int(amax);
    const int e = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
    return e < kEMin ? kEMin : (e > kEMax ? kEMax : e);
}

// ----- 1 / 2 / 4 / 8 neighbouring elements of a row, as binary32 -------------
template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f(float v) { return v; }
template <> __device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f(float v) { return v; }
template <> __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }

template <int BYTES> struct Word;
template <> struct Word<4> { using type = uint32_t; };
template <> struct Word<8> { using type = uint2; };
template <> struct Word<16> { using type = uint4; };

template <typename T, int N>
__device__ __forceinline__ void load_n(const T *p, float (&v)[N]) {
    constexpr int B = sizeof(T) * N < 16 ? sizeof(T) * N : 16, M = B / sizeof(T);
    using W = typename Word<B>::type;
    W w[N / M];
#pragma unroll
    for (int i = 0; i < N / M; ++i) w[i] = reinterpret_cast<const W *>(p)[i];
    const T *t = reinterpret_cast<const T *>(w);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = to_f(t[i]);
}
template <typename T, int N>
__device__ __forceinline__ void store_n(T *p, const float (&v)[N]) {
    constexpr int B = sizeof(T) * N < 16 ? sizeof(T) * N : 16, M = B / sizeof(T);
    using W = typename Word<B>::type;
    W w[N / M];
    T *t = reinterpret_cast<T *>(w);
#pragma unroll
    for (int i = 0; i < N; ++i) t[i] = from_f<T>(v[i]);
#pragma unroll
    for (int i = 0; i < N / M; ++i) reinterpret_cast<W *>(p)[i] = w[i];
}

// N elements as they lie in memory, to be taken apart later (fewer registers while they are on their way).
template <typename T, int N> struct Raw {
    static constexpr int B = sizeof(T) * N < 16 ? sizeof(T) * N : 16, M = sizeof(T) * N / B;
    typename Word<B>::type w[M];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < M; ++i) w[i] = reinterpret_cast<const typename Word<B>::type *>(p)[i];
    }
    __device__ __forceinline__ void take(float (&v)[N]) const {
        const T *t = reinterpret_cast<const T *>(w);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = to_f(t[i]);
    }
};

// ---------------------------------------------------------------------------
// The table of cosines and sines.  Angles pos * f_i and the frequencies
// f_i = base^(-2 i / rot), in binary64: at position 10^5 a binary32 angle is off
// by 4e-3.  Only the table's entries are rounded, once, to binary32.
//   linear  f / factor                     ntk  base * factor^(rot / (rot - 2))
//   yarn    f (1 - w) + f / factor * w, w the ramp between the pairs that turn
//           beta_fast and beta_slow times over the original context
// ---------------------------------------------------------------------------
struct TableArgs {
    float2 *table;
    int64_t n_pos;
    int half;                  // rot / 2
    double log_base, inv_factor, ramp_lo, ramp_hi, magnitude;
};
__global__ void __launch_bounds__(256) rope_table_kernel(const TableArgs A) {
    const int64_t n = A.n_pos * A.half;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t pos = i / A.half;
        const int p = (int)(i - pos * A.half);
        double f = exp(-A.log_base * ((double)p / A.half));
        double w = (p - A.ramp_lo) / (A.ramp_hi - A.ramp_lo);
        w = w < 0.0 ? 0.0 : (w > 1.0 ? 1.0 : w);
        f = f * (1.0 - w) + f * A.inv_factor * w;
        double s, c;
        sincos((double)pos * f, &s, &c);
        A.table[i] = make_float2((float)(c * A.magnitude), (float)(s * A.magnitude));
    }
}

// One pair: y1 = RN(RN(x1 c) - RN(x2 s)), y2 = RN(RN(x2 c) + RN(x1 s)); the
// roundings are pinned, so every kernel that rotates gives the same bits.
__device__ __forceinline__ float2 rotate(float x1, float x2, float2 cs) {
    return make_float2(__fsub_rn(__fmul_rn(x1, cs.x), __fmul_rn(x2, cs.y)),
                       __fadd_rn(__fmul_rn(x2, cs.x), __fmul_rn(x1, cs.y)));
}

// ---------------------------------------------------------------------------
// Rotary positions of rows [T][heads][dim].  Bound by the bytes of x and y.  A block
// of 128 threads takes a token, then the next one of its share, whose position is on
// its way meanwhile; a thread keeps to one place of the head -- 8 neighbouring
// elements, with their 8 partners in the half layout, or one pair where alignment or
// sizes do not allow 16-byte accesses -- loads its cosines and sines once and goes over
// the heads, two (half) or four (interleaved) on their way at a time, the first before the
// position is known.  Registers (64 at most, so 1024 threads an SM) matter more than loads
// in flight: 16384 tokens of 32 heads of 128, half of it turned, bf16, took 203 us with 128
// registers and a block a token, 69 with 64, 53 with blocks that stay (5.2 TB/s; the copy
// rate is 6.6).
// ---------------------------------------------------------------------------
struct RopeArgs {
    Rows x, y;
    int64_t T;
    int dim, inverse;
    const int32_t *positions;
    Rope r;
};
template <int N>
__device__ __forceinline__ void load_cs(const float2 *row, float sign, float2 (&cs)[N]) {
    const float4 *p = reinterpret_cast<const float4 *>(row);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const float4 v = p[i];
        cs[2 * i] = make_float2(v.x, v.y * sign);
        cs[2 * i + 1] = make_float2(v.z, v.w * sign);
    }
}
// Places of a head's row: [rot / 16] paired eights (half layout) or [rot / 8] of four pairs
// (interleaved), then [(dim - rot) / 8] eights to copy; without 16-byte accesses dim / 2 pairs.
__host__ __device__ __forceinline__ int rope_items(int dim, int rot, bool interleaved) {
    return interleaved ? dim / 8 : rot / 16 + (dim - rot) / 8;
}
// One head's place, in: MODE 0 eights to copy, 1 four pairs, 2 paired eights.
template <int MODE, typename TO, typename RX, typename CS>
__device__ __forceinline__ void rope_place(const RX &ra, const RX &rb, TO *y, int half, const CS &cs) {
    float a[8], b[8];
    ra.take(a);
    if (MODE == 2) rb.take(b);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (MODE == 2) {
            const float2 z = rotate(a[j], b[j], cs[j]);
            a[j] = z.x;
            b[j] = z.y;
        } else if (MODE == 1 && !(j & 1)) {
            const float2 z = rotate(a[j], a[j + 1], cs[j / 2]);
            a[j] = z.x;
            a[j + 1] = z.y;
        }
    }
    store_n(y, a);
    if (MODE == 2) store_n(y + half, b);
}
// All heads of one token, by `threads` threads of which this is number `tid`.  `position` is called once, after the
// first heads' loads are out; it gives the table's row or NULL (nothing is written).
template <bool INTER, typename TI, typename TO, typename POS>
__device__ __forceinline__ void rope_token(const TI *x, int64_t ldx, TO *y, int64_t ldy, const Rope &r, float sign, int dim,
                                           int heads, int tid, int threads, POS position) {
    const int half = r.rot >> 1, per = rope_items(dim, r.rot, INTER);
    const int wide = per < threads ? per : threads, step = threads / wide, h0 = tid / wide;
    if (h0 >= step) return;
    constexpr int U = INTER ? 4 : 2;                               // heads on their way at a time: 32 elements
    const float2 *row = nullptr;
    for (int j = tid % wide; j < per; j += wide) {
        const bool turn = (INTER ? 8 : 16) * j < r.rot;
        const int d = INTER || turn ? 8 * j : r.rot + 8 * (j - (r.rot >> 4));
        const bool two = !INTER && turn;
        float2 cs[INTER ? 4 : 8];
        for (int h = h0; h < heads; h += U * step) {
            Raw<TI, 8> a[U], b[INTER ? 1 : U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (h + u * step < heads) {
                    a[u].load(x + (h + u * step) * ldx + d);
                    if (two) b[INTER ? 0 : u].load(x + (h + u * step) * ldx + d + half);
                }
            if (h == h0) {
                if (!row) row = position();
                if (!row) return;
                if (turn) load_cs(row + (INTER ? 4 : 8) * j, sign, cs);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (h + u * step < heads) {
                    TO *to = y + (h + u * step) * ldy + d;
                    if (!turn) rope_place<0>(a[u], a[u], to, half, cs);
                    else rope_place<INTER ? 1 : 2>(a[u], b[INTER ? 0 : u], to, half, cs);
                }
        }
    }
}
// The same a pair at a time, for rows of any alignment, head_dim and rot; types and layout looked at as it goes.
__device__ __forceinline__ float load_any(const void *p, int dtype, int64_t i) {
    return dtype == kF32   ? static_cast<const float *>(p)[i]
           : dtype == kF16 ? __half2float(static_cast<const __half *>(p)[i])
                           : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}
__device__ __forceinline__ void store_any(void *p, int dtype, int64_t i, float v) {
    if (dtype == kF32) static_cast<float *>(p)[i] = v;
    else if (dtype == kF16) static_cast<__half *>(p)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}
__device__ __noinline__ void rope_token_any(const Rows x, const Rows y, int64_t t, const Rope r, const float2 *row, float sign,
                                            int dim, int tid, int threads) {
    const int half = r.rot >> 1;
    for (int i = tid; i < dim / 2 * x.heads; i += threads) {
        const int h = i / (dim / 2), j = i - h * (dim / 2);
        const bool apart = j < half && !r.interleaved;
        const int d1 = apart ? j : 2 * j, d2 = apart ? j + half : 2 * j + 1;
        const int64_t from = t * x.ld_tok + h * x.ld_head, to = t * y.ld_tok + h * y.ld_head;
        float2 z = make_float2(load_any(x.data, x.dtype, from + d1), load_any(x.data, x.dtype, from + d2));
        if (j < half) z = rotate(z.x, z.y, make_float2(row[j].x, row[j].y * sign));
        store_any(const_cast<void *>(y.data), y.dtype, to + d1, z.x);
        store_any(const_cast<void *>(y.data), y.dtype, to + d2, z.y);
    }
}
__device__ __forceinline__ const float2 *rope_row(const RopeArgs &A, int64_t pos) {
    if (pos >= 0 && pos < A.r.n_pos) return A.r.table + pos * (A.r.rot >> 1);
    atomicOr(&g_dev_error, kDevErrBadIndex);
    return nullptr;
}
__global__ void __launch_bounds__(128, 8) rope_any_kernel(const RopeArgs A) {
    griddep_launch_dependents();
    griddep_wait();
    for (int64_t t = blockIdx.x; t < A.T; t += gridDim.x)
        if (const float2 *row = rope_row(A, A.positions[t]))
            rope_token_any(A.x, A.y, t, A.r, row, A.inverse ? -1.0f : 1.0f, A.dim, threadIdx.x, blockDim.x);
}
template <typename TI, typename TO, bool INTER>
__global__ void __launch_bounds__(128, 8) rope_kernel(const RopeArgs A) {
    griddep_launch_dependents();
    griddep_wait();
    int64_t next = A.positions[blockIdx.x];
    for (int64_t t = blockIdx.x; t < A.T; t += gridDim.x) {
        const int64_t pos = next;
        if (t + gridDim.x < A.T) next = A.positions[t + gridDim.x];
        rope_token<INTER>(static_cast<const TI *>(A.x.data) + t * A.x.ld_tok, A.x.ld_head,
                          static_cast<TO *>(const_cast<void *>(A.y.data)) + t * A.y.ld_tok, A.y.ld_head, A.r,
                          A.inverse ? -1.0f : 1.0f, A.dim, A.x.heads, threadIdx.x, blockDim.x,
                          [&]() -> const float2 * { return rope_row(A, pos); });
    }
}

// ---------------------------------------------------------------------------
// Append.  A team of warps per (block of 16 positions that gets new tokens, head): four
// warps of four rows of keys and values each, which stay in registers, so k and v are
// read once, the block's exponents are known before any code is written, and no two teams
// touch the same block; one warp and one row where every sequence has one new token.
// Seven prompts, 8 + 32 heads, 345 MB: 87 us on the device (4.0 TB/s), 119 with the queries
// rotated after the appends; 256 single tokens, 8 + 64 heads: 6.5 us; one: 3.6.  The prompts are
// bound by instructions beside waits for loads: 61 % of the issue slots and 45 % of the ALUs,
// HBM at 44 %, 22 warps an SM that wait for their rows longer than for anything else (nothing of
// a team's next item is on its way meanwhile).  Decode is latency: lengths, page, rows, old scale.
// Rows are dealt to blocks of threads in chunks: the rows of a chunk that open a
// block (its leaders) are found by a ballot, and (leader, head) items go round the teams.
// Other blocks of threads of the same launch rotate the queries.
// ---------------------------------------------------------------------------
struct AppendArgs {
    Cache C;
    Batch B;
    int64_t T;
    Rows kv[2], q, q_out;
    Rope r;                    // table NULL: no rotation
    int64_t appends;           // blocks of threads that append: `parts` for a chunk of rows
    int parts;
    int q_rows;                // rows of queries of each of the others, at most 32
};
constexpr int kAppendThreads = 256;

__device__ __forceinline__ int64_t last_position(const Batch &B, const Cache &C, const Rope &r) {
    int64_t end = B.max_pages * C.page;
    if (r.table && r.n_pos < end) end = r.n_pos;
    return end;
}
// Elements [d0, d0 + N) of a row, v, rotated one by one: for tables whose pairs do not lie side by side in a lane.
template <typename TI, int N>
__device__ __forceinline__ void rotate_apart(const TI *x, const float2 *row, const Rope &r, int d0, float (&v)[N]) {
    const int half = r.rot >> 1;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int d = d0 + j;
        if (d >= r.rot) continue;
        const bool hi = r.interleaved ? d & 1 : d >= half;
        const int other = r.interleaved ? d ^ 1 : (hi ? d - half : d + half);
        const float o = to_f(x[other]);
        const float2 cs = row[r.interleaved ? d >> 1 : (hi ? d - half : d)];
        v[j] = hi ? rotate(o, v[j], cs).y : rotate(v[j], o, cs).x;
    }
}
__device__ __forceinline__ uint16_t e4m3x2(float a, float b) {     // a in the low byte
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 from_e4m3x2(uint16_t v) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(v, __NV_E4M3);
    return __half22float2(__half2(h));
}
// Codes of one lane's N values in units of 2^e; what is not finite becomes NaN.
template <int N>
__device__ __forceinline__ void store_codes(uint8_t *p, const float (&v)[N], float inv) {
    uint16_t w[N / 2];
#pragma unroll
    for (int j = 0; j < N; j += 2) {
        const float a = isfinite(v[j]) ? v[j] * inv : __int_as_float(0x7fffffff);
        const float b = isfinite(v[j + 1]) ? v[j + 1] * inv : __int_as_float(0x7fffffff);
        w[j / 2] = e4m3x2(a, b);
    }
    if (N == 4) *reinterpret_cast<uint32_t *>(p) = w[0] | ((uint32_t)w[N / 2 - 1] << 16);
    else *reinterpret_cast<uint16_t *>(p) = w[0];
}

// One item: keys and values of one head and block.  TEAM warps (this is number `member`) with kBlock / TEAM rows
// each, or one with one row.  `page` is the block's, `share` [2][4].
template <typename TI, int D, int TEAM, bool INTER>
__device__ __forceinline__ void append_block(const AppendArgs &A, int64_t len, int64_t end, int64_t page, int64_t pos,
                                             int64_t row, int head, int member, int team, float *share) {
    constexpr int N = D / 32, OWN = TEAM == 1 ? 1 : kBlock / TEAM;
    const int lane = threadIdx.x & 31, d0 = lane * N, k0 = member * OWN;
    const int off = (int)(pos % kBlock);                           // rows of the block from before
    int n = kBlock - off;
    if (len - pos < n) n = (int)(len - pos);
    if (end - pos < n) n = (int)(end - pos);
    const int64_t tile = (page * A.C.heads + head) * A.C.page + pos % A.C.page;     // first row written
    const TI *x[2];
#pragma unroll
    for (int w = 0; w < 2; ++w)
        x[w] = static_cast<const TI *>(A.kv[w].data) + (row + k0) * A.kv[w].ld_tok + head * A.kv[w].ld_head;
    // all loads first: rows of values and keys, the keys' partners where they are neighbours (half layout), cosines and sines
    const int half = A.r.rot >> 1, lo = INTER ? d0 >> 1 : (d0 < half ? d0 : d0 - half);
    const bool near = INTER ? A.r.rot % N == 0 : half % N == 0 && half % 2 == 0, turn = A.r.table && d0 < A.r.rot;
    const bool pair = !INTER && near && turn;
    Raw<TI, N> rv[OWN], rk[OWN], ro[OWN];
#pragma unroll
    for (int i = 0; i < OWN; ++i)
        if (k0 + i < n) {
            rv[i].load(x[1] + i * A.kv[1].ld_tok + d0);
            rk[i].load(x[0] + i * A.kv[0].ld_tok + d0);
            if (pair) ro[i].load(x[0] + i * A.kv[0].ld_tok + (d0 < half ? d0 + half : d0 - half));
        }
    int e_old[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) e_old[w] = off ? exponent_of(A.C.scales[w][tile / kBlock]) : kEMin;
    float v[2][OWN][N], amax[2] = {0.0f, 0.0f};
    const float2 *table = A.r.table + (pos + k0) * half + lo;
    if (near && turn) {
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            float2 cs[N];
            if (k0 + i < n) {
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (!INTER || j < N / 2) cs[j] = table[i * half + j];
            }
            rk[i].take(v[0][i]);
            if (INTER) {
#pragma unroll
                for (int j = 0; j < N; j += 2) {
                    const float2 z = rotate(v[0][i][j], v[0][i][j + 1], cs[j / 2]);
                    v[0][i][j] = z.x;
                    v[0][i][j + 1] = z.y;
                }
            } else {
                float o[N];
                ro[i].take(o);
#pragma unroll
                for (int j = 0; j < N; ++j)
                    v[0][i][j] = d0 < half ? rotate(v[0][i][j], o[j], cs[j]).x : rotate(o[j], v[0][i][j], cs[j]).y;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            rk[i].take(v[0][i]);
            if (turn && k0 + i < n) rotate_apart<TI, N>(x[0] + i * A.kv[0].ld_tok, A.r.table + (pos + k0 + i) * half, A.r, d0, v[0][i]);
        }
    }
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        rv[i].take(v[1][i]);
        if (k0 + i < n) {
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (isfinite(v[w][i][j])) amax[w] = fmaxf(amax[w], fabsf(v[w][i][j]));
        }
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) amax[w] = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax[w])));
    if (TEAM > 1) {
        if (lane < 2) share[4 * lane + member] = lane ? amax[1] : amax[0];
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(32 * TEAM) : "memory");       // every warp has read the old scales, too
#pragma unroll
        for (int w = 0; w < 2; ++w)
            amax[w] = fmaxf(fmaxf(share[4 * w], share[4 * w + 1]), fmaxf(share[4 * w + 2], share[4 * w + 3]));
    } else {
        __syncwarp();
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        uint8_t *codes = A.C.codes[w] + tile * D + d0;
        int e = exponent_for(amax[w]);
        if (e > e_old[w]) {
            const float f = pow2(e_old[w] - e);
            for (int i = 1 + member; i <= off; i += TEAM) {        // the codes from before, in the new scale
                uint8_t *p = codes - i * D;
                uint16_t c[N / 2];
#pragma unroll
                for (int j = 0; j < N / 2; ++j) {
                    const float2 o = from_e4m3x2(reinterpret_cast<const uint16_t *>(p)[j]);
                    c[j] = e4m3x2(o.x * f, o.y * f);
                }
#pragma unroll
                for (int j = 0; j < N / 2; ++j) reinterpret_cast<uint16_t *>(p)[j] = c[j];
            }
        } else {
            e = e_old[w];
        }
        if (lane == 0 && member == 0) A.C.scales[w][tile / kBlock] = pow2(e);
        const float inv = pow2(-e);
#pragma unroll
        for (int i = 0; i < OWN; ++i)
            if (k0 + i < n) store_codes<N>(codes + (k0 + i) * D, v[w][i], inv);
    }
}

// Position of row t, -1 if it has none that the tables cover.
__device__ __forceinline__ int64_t position_of(const AppendArgs &A, int64_t t, int64_t end) {
    if (t >= A.T) return -1;
    const int b = seq_of_row(A.B, t);
    if (b < 0) return -1;
    const Seq s = seq_info(A.B, b, A.T);
    const int64_t pos = s.start + (t - s.row0);
    return pos < end ? pos : -1;
}

template <typename TI, typename TO, int D, int TEAM, bool INTER>
__global__ void __launch_bounds__(kAppendThreads, 3) kv_append_kernel(const AppendArgs A) {
    constexpr int CHUNK = TEAM == 1 ? 1 : 16, WARPS = kAppendThreads / 32, TEAMS = WARPS / TEAM;
    __shared__ float share[TEAMS][2][8];
    griddep_launch_dependents();
    griddep_wait();
    const int64_t end = last_position(A.B, A.C, A.r);
    // the blocks that append lie evenly between those that rotate queries: the ones wait, the others stream
    const int64_t before = blockIdx.x * A.appends / gridDim.x;
    if (before == (blockIdx.x + 1) * A.appends / gridDim.x) {
        // queries: the rows' positions are looked up by the lanes of every warp at once; a lone row takes all threads
        const int lane = threadIdx.x & 31;
        const int64_t row0 = (blockIdx.x - before) * A.q_rows;
        const int64_t mine = lane < A.q_rows ? position_of(A, row0 + lane, end) : -1;
        const int threads = A.q_rows == 1 ? kAppendThreads : kAppendThreads / 2;
        const bool vec = A.r.rot % (INTER ? 8 : 16) == 0;
        for (int i = threadIdx.x / threads; i < A.q_rows; i += kAppendThreads / threads) {
            const int64_t pos = __shfl_sync(0xffffffffu, mine, i), t = row0 + i;
            if (pos >= 0) {
                const float2 *table = A.r.table + pos * (A.r.rot >> 1);
                const int tid = threadIdx.x % threads;
                if (vec)
                    rope_token<INTER>(static_cast<const TI *>(A.q.data) + t * A.q.ld_tok, A.q.ld_head,
                                      static_cast<TO *>(const_cast<void *>(A.q_out.data)) + t * A.q_out.ld_tok, A.q_out.ld_head,
                                      A.r, 1.0f, D, A.q.heads, tid, threads, [&]() { return table; });
                else
                    rope_token_any(A.q, A.q_out, t, A.r, table, 1.0f, D, tid, threads);
            }
            __syncwarp();
        }
        return;
    }
    const int64_t at = before / A.parts;
    // the chunk's rows: lane i looks at row chunk0 + i (every warp does the same)
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int part = (int)(before % A.parts);
    const int64_t row = at * CHUNK + lane;
    int64_t pos = 0, len = 0, page = -1;
    bool lead = false;
    if (lane < CHUNK && row < A.T) {
        const int b = seq_of_row(A.B, row);
        if (b >= 0) {
            const Seq s = seq_info(A.B, b, A.T);
            len = s.len;
            pos = s.start + (row - s.row0);
            const int64_t first = s.start > 0 ? s.start : 0;
            lead = pos >= first && pos < end && (pos == first || pos % kBlock == 0);
            if (pos >= end && threadIdx.x < 32) atomicOr(&g_dev_error, kDevErrBadIndex);
            if (lead) page = page_of(A.B, A.C, b, pos);
            lead = lead && page >= 0;
        }
    }
    const unsigned leads = __ballot_sync(0xffffffffu, lead);
    const int items = __popc(leads) * A.C.heads, team = warp / TEAM;
    int turn = 0;
    for (int it = part * TEAMS + team; it < items; it += A.parts * TEAMS, turn ^= 1) {
        const int k = it / A.C.heads, head = it - k * A.C.heads;
        unsigned rest = leads;
        for (int i = 0; i < k; ++i) rest &= rest - 1;
        const int src = __ffs(rest) - 1;                           // the lane of leader k
        append_block<TI, D, TEAM, INTER>(A, __shfl_sync(0xffffffffu, len, src), end, __shfl_sync(0xffffffffu, page, src),
                                  __shfl_sync(0xffffffffu, pos, src), __shfl_sync(0xffffffffu, row, src), head,
                                  warp % TEAM, team, share[team][turn]);
    }
}

}  // namespace kv
}  // namespace awq
