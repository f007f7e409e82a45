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
// normal number, so tokens appended one by one end as a prompt appended at once
// (integer codes would round again at every rise).  Keys also differ in size from
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
// Rotary positions of rows [T][heads][dim].  Bound by the bytes of x and y; the
// table's row of a token is read once per head from L1.  One block per token;
// a thread moves 8 neighbouring elements (16 with their partners in the half
// layout), or one pair where alignment or sizes do not allow 16-byte accesses.
// ---------------------------------------------------------------------------
struct RopeArgs {
    Rows x, y;
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
// Item `i` of one head's row: rows of items are [rot / 16] of paired eights
// (half layout) or [rot / 8] of four pairs (interleaved), then [(dim - rot) / 8] eights.
template <typename TI, typename TO>
__device__ __forceinline__ void rope_item(const TI *x, TO *y, const float2 *row, const Rope &r, float sign, int i) {
    const int half = r.rot >> 1;
    if (r.interleaved) {
        float v[8];
        load_n(x + 8 * i, v);
        if (8 * i < r.rot) {
            float2 cs[4];
            load_cs(row + 4 * i, sign, cs);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 z = rotate(v[2 * j], v[2 * j + 1], cs[j]);
                v[2 * j] = z.x;
                v[2 * j + 1] = z.y;
            }
        }
        store_n(y + 8 * i, v);
    } else if (16 * i < r.rot) {
        float a[8], b[8];
        float2 cs[8];
        load_n(x + 8 * i, a);
        load_n(x + half + 8 * i, b);
        load_cs(row + 8 * i, sign, cs);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 z = rotate(a[j], b[j], cs[j]);
            a[j] = z.x;
            b[j] = z.y;
        }
        store_n(y + 8 * i, a);
        store_n(y + half + 8 * i, b);
    } else {
        const int d = r.rot + 8 * (i - (r.rot >> 4));
        float v[8];
        load_n(x + d, v);
        store_n(y + d, v);
    }
}
__host__ __device__ __forceinline__ int rope_items(int dim, int rot, bool interleaved) {
    return interleaved ? dim / 8 : rot / 16 + (dim - rot) / 8;
}
// Pair `i` of dim / 2, any alignment.
template <typename TI, typename TO>
__device__ __forceinline__ void rope_pair(const TI *x, TO *y, const float2 *row, const Rope &r, float sign, int i) {
    const int half = r.rot >> 1;
    int d1 = 2 * i, d2 = 2 * i + 1;
    if (!r.interleaved && i < half) {
        d1 = i;
        d2 = i + half;
    }
    float2 z = make_float2(to_f(x[d1]), to_f(x[d2]));
    if (i < half) {
        float2 cs = row[i];
        cs.y *= sign;
        z = rotate(z.x, z.y, cs);
    }
    y[d1] = from_f<TO>(z.x);
    y[d2] = from_f<TO>(z.y);
}
template <typename TI, typename TO, bool VEC>
__global__ void __launch_bounds__(256) rope_kernel(const RopeArgs A) {
    const int64_t t = blockIdx.x;
    const int64_t pos = A.positions[t];
    if (pos < 0 || pos >= A.r.n_pos) {
        if (threadIdx.x == 0) atomicOr(&g_dev_error, kDevErrBadIndex);
        return;
    }
    const float2 *row = A.r.table + pos * (A.r.rot >> 1);
    const float sign = A.inverse ? -1.0f : 1.0f;
    const TI *x = static_cast<const TI *>(A.x.data) + t * A.x.ld_tok;
    TO *y = static_cast<TO *>(const_cast<void *>(A.y.data)) + t * A.y.ld_tok;
    const int per = VEC ? rope_items(A.dim, A.r.rot, A.r.interleaved) : A.dim / 2;
    for (int i = threadIdx.x; i < per * A.x.heads; i += blockDim.x) {
        const int h = i / per, j = i - h * per;
        if (VEC) rope_item(x + h * A.x.ld_head, y + h * A.y.ld_head, row, A.r, sign, j);
        else rope_pair(x + h * A.x.ld_head, y + h * A.y.ld_head, row, A.r, sign, j);
    }
}

// ---------------------------------------------------------------------------
// Append.  One warp per (block of 16 positions that gets new tokens, head, keys
// or values): all new rows of the block are held in registers (16 x D / 32 values
// a lane), so k and v are read once, the block's exponent is known before any
// code is written, and no two warps touch the same block.  Bound by the bytes of
// k and v; in decode (one row a block) by latency.
// Rows are dealt to blocks of threads in chunks: the rows of a chunk that open a
// block (its leaders) are found by a ballot, and (leader, head, k / v) items go
// round the warps.  A second range of the grid rotates the queries.
// ---------------------------------------------------------------------------
struct AppendArgs {
    Cache C;
    Batch B;
    int64_t T;
    Rows kv[2], q, q_out;
    Rope r;                    // table NULL: no rotation
    int chunk;                 // rows per block of threads: 1 or 16
    int64_t chunks;            // blocks in x that append; those past them rotate queries
};
constexpr int kAppendThreads = 256;

__device__ __forceinline__ int64_t last_position(const Batch &B, const Cache &C, const Rope &r) {
    int64_t end = B.max_pages * C.page;
    if (r.table && r.n_pos < end) end = r.n_pos;
    return end;
}
// Elements [d0, d0 + N) of the rotated row (N = D / 32 a lane).
template <typename TI, int N>
__device__ __forceinline__ void rotated(const TI *x, const float2 *row, const Rope &r, int d0, float (&v)[N]) {
    load_n(x + d0, v);
    if (!row) return;
    const int half = r.rot >> 1;
    if (r.interleaved) {
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            if (d0 + j >= r.rot) continue;
            const float2 z = rotate(v[j], v[j + 1], row[(d0 + j) >> 1]);
            v[j] = z.x;
            v[j + 1] = z.y;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int d = d0 + j;
            if (d >= r.rot) continue;
            const bool hi = d >= half;
            const float other = to_f(x[hi ? d - half : d + half]);
            const float2 cs = row[hi ? d - half : d];
            v[j] = hi ? rotate(other, v[j], cs).y : rotate(v[j], other, cs).x;
        }
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

template <typename TI, int D>
__device__ __forceinline__ void append_block(const AppendArgs &A, const Seq &s, int b, int64_t pos, int64_t row,
                                             int head, int which) {
    constexpr int N = D / 32;
    const int lane = threadIdx.x & 31, d0 = lane * N;
    const int64_t end = last_position(A.B, A.C, A.r);
    const int off = (int)(pos % kBlock);                           // rows of the block from before
    const int64_t page = page_of(A.B, A.C, b, pos);
    if (page < 0) return;
    int n = kBlock - off;
    if (s.len - pos < n) n = (int)(s.len - pos);
    if (end - pos < n) n = (int)(end - pos);
    const Rows &R = A.kv[which];
    const TI *x = static_cast<const TI *>(R.data) + row * R.ld_tok + head * R.ld_head;
    const int half = A.r.rot >> 1;
    const bool turn = which == 0 && A.r.table != nullptr;
    float v[kBlock][N];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < kBlock; ++i)
        if (i < n) rotated<TI, N>(x + i * R.ld_tok, turn ? A.r.table + (pos + i) * half : nullptr, A.r, d0, v[i]);
#pragma unroll
    for (int i = 0; i < kBlock; ++i)
        if (i < n) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (isfinite(v[i][j])) amax = fmaxf(amax, fabsf(v[i][j]));
        }
    int e = exponent_for(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax))));
    const int64_t tile = (page * A.C.heads + head) * A.C.page + pos % A.C.page;     // first row written
    float *scale = A.C.scales[which] + tile / kBlock;
    uint8_t *codes = A.C.codes[which] + tile * D + d0;
    if (off) {
        const int e_old = exponent_of(*scale);
        if (e > e_old) {
            const float f = pow2(e_old - e);
            for (int i = 1; i <= off; ++i) {
                uint8_t *p = codes - i * D;
                uint16_t w[N / 2];
#pragma unroll
                for (int j = 0; j < N / 2; ++j) {
                    const float2 o = from_e4m3x2(reinterpret_cast<const uint16_t *>(p)[j]);
                    w[j] = e4m3x2(o.x * f, o.y * f);
                }
#pragma unroll
                for (int j = 0; j < N / 2; ++j) reinterpret_cast<uint16_t *>(p)[j] = w[j];
            }
        } else {
            e = e_old;
        }
        __syncwarp();                                              // every lane has read the old scale
    }
    if (lane == 0) *scale = pow2(e);
    const float inv = pow2(-e);
#pragma unroll
    for (int i = 0; i < kBlock; ++i)
        if (i < n) store_codes<N>(codes + i * D, v[i], inv);
}

template <typename TI, typename TO, int D>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendArgs A) {
    const int64_t end = last_position(A.B, A.C, A.r);
    if (blockIdx.x >= A.chunks) {                                  // queries: one row a block
        const int64_t t = blockIdx.x - A.chunks;
        const int b = seq_of_row(A.B, t);
        if (b < 0) return;
        const Seq s = seq_info(A.B, b, A.T);
        const int64_t pos = s.start + (t - s.row0);
        if (pos < 0 || pos >= end) return;
        const float2 *row = A.r.table + pos * (A.r.rot >> 1);
        const TI *x = static_cast<const TI *>(A.q.data) + t * A.q.ld_tok;
        TO *y = static_cast<TO *>(const_cast<void *>(A.q_out.data)) + t * A.q_out.ld_tok;
        const bool vec = A.r.interleaved ? A.r.rot % 8 == 0 : A.r.rot % 16 == 0;
        const int per = vec ? rope_items(D, A.r.rot, A.r.interleaved) : D / 2;
        for (int i = blockIdx.y * kAppendThreads + threadIdx.x; i < per * A.q.heads; i += gridDim.y * kAppendThreads) {
            const int h = i / per, j = i - h * per;
            if (vec) rope_item(x + h * A.q.ld_head, y + h * A.q_out.ld_head, row, A.r, 1.0f, j);
            else rope_pair(x + h * A.q.ld_head, y + h * A.q_out.ld_head, row, A.r, 1.0f, j);
        }
        return;
    }
    // the chunk's rows: lane i looks at row chunk0 + i (every warp does the same)
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x * (int64_t)A.chunk + lane;
    int b = -1;
    int64_t pos = 0;
    Seq s = {};
    bool lead = false;
    if (lane < A.chunk && row < A.T) {
        b = seq_of_row(A.B, row);
        if (b >= 0) {
            s = seq_info(A.B, b, A.T);
            pos = s.start + (row - s.row0);
            const int64_t first = s.start > 0 ? s.start : 0;
            lead = pos >= first && pos < end && (pos == first || pos % kBlock == 0);
            if (pos >= end && threadIdx.x < 32) atomicOr(&g_dev_error, kDevErrBadIndex);
        }
    }
    const unsigned leads = __ballot_sync(0xffffffffu, lead);
    const int per = 2 * A.C.heads, items = __popc(leads) * per;
    const int warps = kAppendThreads / 32;
    for (int it = blockIdx.y * warps + warp; it < items; it += gridDim.y * warps) {
        const int k = it / per, hv = it - k * per;
        const int src = __fns(leads, 0, k + 1);                    // the lane of leader k
        Seq ss;
        ss.len = __shfl_sync(0xffffffffu, s.len, src);
        const int bb = __shfl_sync(0xffffffffu, b, src);
        const int64_t pp = __shfl_sync(0xffffffffu, pos, src);
        const int64_t rr = __shfl_sync(0xffffffffu, row, src);
        append_block<TI, D>(A, ss, bb, pp, rr, hv >> 1, hv & 1);
    }
}

}  // namespace kv
}  // namespace awq
