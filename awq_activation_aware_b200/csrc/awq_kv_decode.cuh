// Attention over the paged 8-bit cache for few query rows per key head: single
// tokens and short drafts (sm_100a).  See awq_kv.cuh for the cache.
//
// A step reads every key and value once and does 4 * rows operations per byte, so
// HBM bounds it: rows <= 16 keep the tensor cores far from their rate, and what
// matters is that the codes stream without a pause and that the instructions to
// turn them into operands fit beside the stream (an SM takes in 27 bytes a clock).
//
//  * Work.  A unit is 64 keys of one (sequence, key head, tile of 8 or 16 query rows); a
//    row is (new token, query head of the key head's group), so a group shares each
//    key.  The units of a launch, in order, are cut into equal contiguous ranges,
//    one per block of threads (two or three blocks an SM), whatever the lengths: a ragged
//    batch and one long sequence fill the machine alike.  Lengths are read on the
//    device.  A segment (the units of one sequence, head and row tile) that crosses
//    a cut leaves partial results, summed in order by a second kernel: the result
//    does not depend on timing.
//  * Stream.  One warp feeds a ring of stages by TMA, one box per page (64 keys at
//    most), 128-byte rows swizzled (64-byte rows for D = 64), and the blocks' scales
//    by 4-byte asynchronous copies.  Four warps consume: warp w owns keys
//    16 w .. 16 w + 15 of each stage, one block of scales.
//  * Products (mma m16n8k16, fp16 operands, binary32 sums), both with the codes as
//    the 16-row operand: S^T = K Q^T and O^T = V^T P^T, so 8 query rows cost half of
//    what 16 do and hold half the registers.  The codes are exact in fp16, and any
//    order of the contracted index will do: a lane takes 16 neighbouring codes of a
//    key in one 16-byte load and the fragments' k indices are whatever those are;
//    the query fragments are loaded to match.  For the second product a lane takes 16
//    codes of four keys; pairs of keys are interleaved by byte permutes, and the
//    probabilities change lanes by a transposing 8 x 8 move.  Both load patterns are
//    free of bank conflicts under the TMA swizzle.
//  * Scales.  The key scale multiplies the score.  The value scale 2^e enters the
//    exponent: P' = 2^(x + e - m + 9), so P' stays in fp16's range whatever the
//    scales, and the row sum adds 2^-e P'.  m, a running reference per row, is some
//    earlier largest x + e; it is raised only when a value exceeds it by 2^6
//    (P' <= 2^15 < 65504), which one vote finds out: no reductions across lanes and
//    no rescaling of the accumulators in the ordinary step.
//  * Masks.  Keys past the sequence may hold anything: their scores become -inf and
//    their codes zero.  A NaN value in a key that some rows of a partly masked block
//    do not see is taken out of the product and put into the sums of the rows that do.
#pragma once

#include <type_traits>

#include "awq_kv.cuh"

namespace awq {
namespace kv {
namespace dec {

constexpr int TILE = 64;                   // keys per unit and stage
constexpr int WARPS = 4;                   // consumer warps
constexpr int THREADS = 32 * (WARPS + 1);
constexpr float kLift = 9.0f, kSlack = 6.0f;

// NT tiles of 8 query rows.
template <int D, int NT> struct Shape {
    static constexpr int ROWS = 8 * NT;
    static constexpr int BLOCKS = NT == 1 ? 3 : 2;         // resident per SM
    static constexpr int STAGE = 2 * TILE * D;             // keys, values
    static constexpr int STAGES = (NT == 1 ? 3 : 4) * (128 / D);
    static constexpr int PER = D / 8;                      // elements of a row that one lane holds
    static constexpr int LD = D + 36;                      // row of the merge area: 4 floats after every PER, 4 more
    static constexpr int OFF_SCALES = STAGES * STAGE;      // float [STAGES][8]
    static constexpr int OFF_BARS = OFF_SCALES + STAGES * 32;
    static constexpr int OFF_ML = OFF_BARS + STAGES * 16;  // float [WARPS][ROWS][2]
    static constexpr int OFF_O = OFF_ML + WARPS * ROWS * 8;
    static constexpr int BYTES = OFF_O + WARPS * ROWS * LD * 4 + 1024;   // + alignment
};

struct Meta {                              // a segment that starts in this block and ends in a later one
    int32_t b, head, rt, last;             // last: the block of its last unit; -1: no such segment
};
struct Args {
    Cache C;
    Batch B;
    int64_t T;
    Rows q, out;
    float scale_log2;
    int64_t window;
    float *lse;
    int group;                             // query heads per key head
    int rows;                              // query rows per tile: 8 or 16
    int box_rows;                          // keys per TMA box: min(page, 64)
    Meta *meta;                            // [grid]
    float *part_ml;                        // [grid][2][rows][2]: slot 0 ends a segment begun earlier, slot 1 starts one
    float *part_o;                         // [grid][2][rows][D]
    uint64_t timeout_ns;
};

// The units of sequence b: heads * rt * nt.
struct Span {
    Seq s;
    int lo, hi;                            // keys that exist and that some row may see
    int t0, nt, rt;
};
constexpr int64_t kMaxLen = 1 << 30;       // positions fit 32 bits with room to spare
__device__ __forceinline__ Span span_of(const Args &A, int b) {
    Span p;
    p.s = seq_info(A.B, b, A.T);
    int64_t cap = A.B.max_pages * A.C.page;
    if (cap > kMaxLen) cap = kMaxLen;
    p.hi = (int)(p.s.len < cap ? p.s.len : cap);
    const int64_t lo = A.window ? p.s.start + 1 - A.window : 0;
    p.lo = lo < 0 ? 0 : (lo > p.hi ? p.hi : (int)lo);
    p.t0 = p.lo / TILE;
    p.nt = (p.hi + TILE - 1) / TILE - p.t0;
    if (p.nt < 1) p.nt = 1;                // rows without keys still get their zeros
    p.rt = (int)(((int64_t)p.s.n * A.group + A.rows - 1) / A.rows);
    return p;
}
__device__ __forceinline__ int64_t units_of(const Args &A, int b) {
    const Span p = span_of(A, b);
    return (int64_t)A.C.heads * p.rt * p.nt;
}

// Where a block's range starts, found by all threads: sums of units over the
// sequences, a chunk of blockDim.x at a time.
struct Range {
    int64_t first, end;                    // units of this block
    int b;                                 // sequence of `first`
    int64_t base;                          // units before sequence b
    int64_t total;
    int64_t blocks;                        // blocks that have units: every one of them at least one
};
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *warp_sums, int64_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, v, i);
        if (lane >= i) v += o;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    int64_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < WARPS + 1; ++w) {
        if (w < warp) before += warp_sums[w];
        total += warp_sums[w];
    }
    return before + v;                     // inclusive
}
__device__ __forceinline__ Range find_range(const Args &A, int64_t *sums, int64_t *found) {
    Range r;
    const int n = A.B.n_seqs;
    int64_t total = 0, incl = 0, mine = 0;
    for (int b0 = 0; b0 < n; b0 += THREADS) {
        const int b = b0 + threadIdx.x;
        int64_t part;
        mine = b < n ? units_of(A, b) : 0;
        incl = block_scan(mine, sums, part);
        total += part;
    }
    r.total = total;
    r.blocks = total < gridDim.x ? total : gridDim.x;
    r.b = 0;
    r.base = r.first = r.end = 0;
    if ((int64_t)blockIdx.x >= r.blocks) return r;
    r.first = total * blockIdx.x / r.blocks;
    r.end = total * (blockIdx.x + 1) / r.blocks;
    int64_t base = 0;
    for (int b0 = 0; b0 < n; b0 += THREADS) {
        int64_t part = total;
        if (n > THREADS) {                 // otherwise the only chunk is still in registers
            const int b = b0 + threadIdx.x;
            mine = b < n ? units_of(A, b) : 0;
            incl = block_scan(mine, sums, part);
        }
        if (base + incl - mine <= r.first && r.first < base + incl) {
            found[0] = b0 + threadIdx.x;
            found[1] = base + incl - mine;
        }
        base += part;
        if (base > r.first) break;
    }
    __syncthreads();
    r.b = (int)found[0];
    r.base = found[1];
    return r;
}

// The block's place in its range: a run of tiles of one segment.
struct Cursor {
    int b, head, rt;
    Span p;
    int64_t seg0;                          // first unit of the segment
    int64_t u;                             // next unit
    __device__ __forceinline__ void start(const Args &A, const Range &r) {
        b = r.b;
        p = span_of(A, b);
        u = r.first;
        const int64_t i = (u - r.base) / p.nt;
        seg0 = r.base + i * p.nt;
        head = (int)(i / p.rt);
        rt = (int)(i % p.rt);
    }
    __device__ __forceinline__ int64_t seg_end() const { return seg0 + p.nt; }
    // to the segment that starts at seg_end() (there is one: it is below the range's end)
    __device__ __forceinline__ void next(const Args &A) {
        seg0 += p.nt;
        u = seg0;
        if (++rt < p.rt) return;
        rt = 0;
        if (++head < A.C.heads) return;
        head = 0;
        do {
            p = span_of(A, ++b);
        } while (p.rt == 0);
    }
};

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t cvt_lo(uint32_t w) {        // two codes to two fp16, exactly
    uint32_t d;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(d) : "r"(w));
    return d;
}
__device__ __forceinline__ uint32_t cvt_hi(uint32_t w) {
    uint32_t d;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(d) : "r"(w));
    return d;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {   // a in the low half
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
    return d;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
// The 8 x 8 matrix of 16-bit elements that a warp holds, row g in lanes 4 g .. 4 g + 3, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t w) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(w));
    return d;
}
// Bytes of a word that hold a NaN code (0x7f or 0xff): 0x80 in each, else 0.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * WARPS) : "memory"); }

// Query fragments (the 8-column operand) of row g of each tile: 16 neighbouring elements of
// chunk 2 c + i (D = 128) or c (D = 64) per i, as fp16.  bf16 rows are lifted by a power of two
// to fp16's upper range, exact for every element above 2^-28 of the row's largest; the return
// value takes it back.
template <typename TQ, int D>
__device__ __forceinline__ float load_query(const Args &A, const Cursor &cur, int row, uint32_t (&qf)[D / 16][2]) {
    const int lane = threadIdx.x & 31, c = lane & 3;
    constexpr int NI = D / 64;
    const int i = row / A.group, h = cur.head * A.group + row % A.group;
    uint32_t w[NI][8] = {};
    if (i < cur.p.s.n) {
        const TQ *q = static_cast<const TQ *>(A.q.data) + (int64_t)(cur.p.s.row0 + i) * A.q.ld_tok +
                      (int64_t)h * A.q.ld_head;
#pragma unroll
        for (int k = 0; k < NI; ++k) {
            const uint4 *p = reinterpret_cast<const uint4 *>(q + 16 * (NI * c + k));
            const uint4 v0 = p[0], v1 = p[1];
            w[k][0] = v0.x; w[k][1] = v0.y; w[k][2] = v0.z; w[k][3] = v0.w;
            w[k][4] = v1.x; w[k][5] = v1.y; w[k][6] = v1.z; w[k][7] = v1.w;
        }
    }
    float unscale = 1.0f;
    if (!std::is_same<TQ, __half>::value) {
        uint32_t top = 0;                                          // largest magnitude, as bf16 bits
#pragma unroll
        for (int k = 0; k < NI; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) top = max(top, max(w[k][j] & 0x7fffu, (w[k][j] >> 16) & 0x7fffu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = min(max((int)(top >> 7) - 127, -100), 126);        // 2^e <= largest < 2^(e + 1)
        const float f = pow2(14 - e);
        unscale = pow2(e - 14);
#pragma unroll
        for (int k = 0; k < NI; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                w[k][j] = pack_f16(__uint_as_float(w[k][j] << 16) * f, __uint_as_float(w[k][j] & 0xffff0000u) * f);
    }
#pragma unroll
    for (int k = 0; k < NI; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {                              // step (k, j): elements 4 j .. 4 j + 3 of the chunk
            qf[4 * k + j][0] = w[k][2 * j];
            qf[4 * k + j][1] = w[k][2 * j + 1];
        }
    return unscale;
}

// Byte offset of the 16-byte chunk of a swizzled row.
template <int D> __device__ __forceinline__ uint32_t chunk_at(uint32_t row, uint32_t chunk) {
    return D == 128 ? row * 128 + ((chunk ^ (row & 7)) << 4) : row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
}

template <typename TQ, int D, int NT>
__global__ void __launch_bounds__(THREADS, Shape<D, NT>::BLOCKS)
kv_decode_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v, const Args A) {
    using S = Shape<D, NT>;
    constexpr int ROWS = S::ROWS;
    extern __shared__ uint8_t raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    float *scales = reinterpret_cast<float *>(sm + S::OFF_SCALES);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + S::OFF_BARS), *empty = full + S::STAGES;
    __shared__ int64_t sums[WARPS + 1], found[2];
    __shared__ int abort_flag;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    if (threadIdx.x == 0) {
        abort_flag = 0;
        found[0] = found[1] = 0;
        for (int i = 0; i < S::STAGES; ++i) {
            mbar_init(full + i, 16);
            mbar_init(empty + i, WARPS);
        }
        fence_mbar_init();
        A.meta[blockIdx.x].last = -1;
    }
    griddep_launch_dependents();
    __syncthreads();
    const Range R = find_range(A, sums, found);
    if (R.first >= R.end) return;
    Cursor cur;
    cur.start(A, R);

    if (warp == WARPS) {
        // ---- the stream: lanes 0-7 a box of keys or values each, lanes 8-15 a block's scale each
        const int which = (lane >> 2) & 1, j = lane & 3;
        const int rows = lane < 8 ? A.box_rows : kBlock;           // keys this lane looks after
        const bool active = lane < 8 ? j < TILE / A.box_rows : lane < 16;
        const void *tmap = which ? &tmap_v : &tmap_k;
        auto page_at = [&](int64_t u) -> int64_t {                 // -1: nothing there; -2: a bad page
            const int pos = (cur.p.t0 + (int)(u - cur.seg0)) * TILE + j * rows;
            if (!active || pos >= cur.p.hi) return -1;
            const int64_t p = A.B.pages[(int64_t)cur.b * A.B.ld_pages + pos / A.C.page];
            return p < 0 || p >= A.C.n_pages ? -2 : p;
        };
        if (lane == 0 && cur.p.s.len > cur.p.hi) atomicOr(&g_dev_error, kDevErrBadIndex);
        int64_t page = page_at(cur.u);
        int stage = 0;
        uint32_t phase = 1;                                        // the first round finds the stages empty
        int64_t issued = 0;
        bool ok = true;
        for (int64_t u = R.first; u < R.end; ++u) {
            const int pos = (cur.p.t0 + (int)(u - cur.seg0)) * TILE + j * rows;
            const int64_t tile = (page * A.C.heads + cur.head) * A.C.page + pos % A.C.page;      // its first row
            const int64_t here = page;
            if (u + 1 < R.end) {                                   // the next page number is on its way meanwhile
                if (u + 1 == cur.seg_end()) {
                    cur.next(A);
                    if (lane == 0 && cur.p.s.len > cur.p.hi) atomicOr(&g_dev_error, kDevErrBadIndex);
                }
                page = page_at(u + 1);
            }
            ok = mbar_wait_warp(empty + stage, phase, &abort_flag, A.timeout_ns);
            if (!ok) break;
            if (lane < 8) {
                if (here >= 0) {
                    mbar_arrive_expect_tx(full + stage, rows * D);
                    tma_load_2d(sm + stage * S::STAGE + which * TILE * D + j * rows * D, tmap, 0, (int32_t)tile, full + stage);
                } else {
                    mbar_arrive(full + stage);
                }
            } else if (lane < 16) {
                float *dst = scales + stage * 8 + which * 4 + j;
                if (here >= 0) {
                    cp_async_4(dst, A.C.scales[which] + tile / kBlock);
                    cp_async_arrive_noinc(full + stage);
                } else {
                    *dst = -1.0f;                                  // no such block
                    if (here == -2) atomicOr(&g_dev_error, kDevErrBadIndex);
                    mbar_arrive(full + stage);
                }
            }
            __syncwarp();
            ++issued;
            if (++stage == S::STAGES) {
                stage = 0;
                phase ^= 1;
            }
        }
        if (!ok) {                                                 // given up: let the copies in flight land
            for (int k = 0; k < S::STAGES && k < issued; ++k) {
                const int64_t n = issued - 1 - k;
                uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait_hint(full + n % S::STAGES, (uint32_t)((n / S::STAGES) & 1), 20000u))
                    if (global_timer_ns() - t0 > A.timeout_ns) break;
            }
        }
        return;
    }

    // ---- consumers
    const int g = lane >> 2, c = lane & 3;
    constexpr int NJ = D / 16;                                     // 16-row tiles of the second product
    uint32_t qf[NT][D / 16][2];
    float rowf[NT][2], base[NT][2], l[NT][2], o[NT][NJ][4];        // base: m - kLift of rows 2 c, 2 c + 1 of a tile
    int pos_of[NT][2];                                             // their positions
    int all_lo = 0, all_hi = 0;                                    // keys that every row of the tile sees
    int stage = 0;
    uint32_t phase = 0;
    bool fresh = true, ok = true;
    for (int64_t u = R.first; u < R.end; ++u) {
        if (fresh) {
            fresh = false;
            const int n = cur.p.s.n, row0 = cur.rt * ROWS;
            int last = (row0 + ROWS - 1) / A.group;
            if (last >= n) last = n - 1;
            const int64_t p0 = cur.p.s.start + row0 / A.group + 1, p1 = cur.p.s.start + last + 1 - A.window;
            all_hi = p0 < 0 ? 0 : (p0 < cur.p.hi ? (int)p0 : cur.p.hi);
            all_lo = A.window && p1 > 0 ? (p1 < kMaxLen ? (int)p1 : (int)kMaxLen) : 0;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float unscale = load_query<TQ, D>(A, cur, row0 + 8 * t + g, qf[t]) * A.scale_log2;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    rowf[t][x] = __shfl_sync(0xffffffffu, unscale, 4 * (2 * c + x));       // from the lane that loaded the row
                    base[t][x] = -INFINITY;
                    l[t][x] = 0.0f;
                    int i = (row0 + 8 * t + 2 * c + x) / A.group;
                    if (i >= n) i = n - 1;                         // rows of nobody follow the last token
                    const int64_t at = cur.p.s.start + i;
                    pos_of[t][x] = at < kMaxLen ? (at < -1 ? -1 : (int)at) : (int)kMaxLen;
                }
#pragma unroll
                for (int j = 0; j < NJ; ++j) o[t][j][0] = o[t][j][1] = o[t][j][2] = o[t][j][3] = 0.0f;
            }
        }
        // a wait that ran out skips the keys but not the barriers below
        ok = ok && mbar_wait_warp(full + stage, phase, &abort_flag, A.timeout_ns);
        const int key0 = (cur.p.t0 + (int)(u - cur.seg0)) * TILE + 16 * warp;
        const int left = cur.p.hi - key0;                          // keys of the block that exist
        const float ks = scales[stage * 8 + warp], vs = scales[stage * 8 + 4 + warp];
        if (ok && left > 0 && ks >= 0.0f && vs >= 0.0f) {
            const uint32_t kt = smem_u32(sm + stage * S::STAGE), vt = kt + TILE * D;
            float s[NT][4];                                        // keys g (0, 1), g + 8 (2, 3) of rows 2 c, 2 c + 1
#pragma unroll
            for (int t = 0; t < NT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.0f;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const uint4 k0 = lds128(kt + chunk_at<D>(16 * warp + g, (D / 64) * c + i));
                const uint4 k1 = lds128(kt + chunk_at<D>(16 * warp + 8 + g, (D / 64) * c + i));
                const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t a[4] = {cvt_lo(w0[j]), cvt_lo(w1[j]), cvt_hi(w0[j]), cvt_hi(w1[j])};
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma_16816(s[t], a, qf[t][4 * i + j][0], qf[t][4 * i + j][1]);
                }
            }
            const int e = exponent_of(vs);
            const float ev = (float)e, inv_v = pow2(-e);
            const bool whole = key0 >= all_lo && key0 + 16 <= all_hi;
            // x + e; hidden keys -inf
            float top = -INFINITY;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float f0 = rowf[t][0] * ks, f1 = rowf[t][1] * ks;
                s[t][0] = __fmaf_rn(s[t][0], f0, ev);
                s[t][1] = __fmaf_rn(s[t][1], f1, ev);
                s[t][2] = __fmaf_rn(s[t][2], f0, ev);
                s[t][3] = __fmaf_rn(s[t][3], f1, ev);
                if (!whole) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int key = key0 + g + 8 * (k >> 1), at = pos_of[t][k & 1];
                        if (key > at || key >= cur.p.hi || (A.window && key <= at - A.window)) s[t][k] = -INFINITY;
                    }
                }
                // past base + kLift + kSlack? (a row without a reference: past -inf)
                top = fmaxf(top, fmaxf(fmaxf(s[t][0], s[t][2]) - base[t][0], fmaxf(s[t][1], s[t][3]) - base[t][1]));
            }
            if (__any_sync(0xffffffffu, top > kLift + kSlack)) {   // seldom: raise the references
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float mx = fmaxf(s[t][x], s[t][2 + x]);
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16)) - kLift;
                        const float f = mx > base[t][x] ? ex2(base[t][x] - mx) : 1.0f;
                        base[t][x] = fmaxf(mx, base[t][x]);
                        l[t][x] *= f;
#pragma unroll
                        for (int j = 0; j < NJ; ++j) {
                            o[t][j][x] *= f;
                            o[t][j][2 + x] *= f;
                        }
                    }
            }
            uint32_t pb[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float b0 = base[t][0] == -INFINITY ? 0.0f : base[t][0];
                const float b1 = base[t][1] == -INFINITY ? 0.0f : base[t][1];
#pragma unroll
                for (int k = 0; k < 4; ++k) s[t][k] = ex2(s[t][k] - (k & 1 ? b1 : b0));
                l[t][0] = __fmaf_rn(s[t][0] + s[t][2], inv_v, l[t][0]);
                l[t][1] = __fmaf_rn(s[t][1] + s[t][3], inv_v, l[t][1]);
                pb[t][0] = transpose8x8(pack_f16(s[t][0], s[t][1]));       // keys 2 c, 2 c + 1 of row g
                pb[t][1] = transpose8x8(pack_f16(s[t][2], s[t][3]));       // keys 2 c + 8, 2 c + 9
            }
            // values of keys 2 c, 2 c + 1, 2 c + 8, 2 c + 9: D / 8 codes of each
            uint32_t v[4][D / 32];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t row = 16 * warp + 2 * c + (k & 1) + 8 * (k >> 1);
                if constexpr (D == 128) {
                    const uint4 x = lds128(vt + chunk_at<D>(row, g));
                    v[k][0] = x.x; v[k][1] = x.y; v[k][2] = x.z; v[k][3] = x.w;
                } else {
                    const uint2 x = lds64(vt + chunk_at<D>(row, g >> 1) + (g & 1) * 8);
                    v[k][0] = x.x; v[k][1] = x.y;
                }
            }
            if (!whole) {
                // keys that do not exist: zeros.  NaN codes: zeros here, NaN in the sums of the rows that see them.
                uint32_t bad = 0;                                  // bit i: key i of the 16
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int key = 2 * c + (k & 1) + 8 * (k >> 1);
#pragma unroll
                    for (int w = 0; w < D / 32; ++w) {
                        if (key >= left) v[k][w] = 0;
                        const uint32_t n = nan_bytes(v[k][w]);
                        if (n) {
                            bad |= 1u << key;
                            v[k][w] &= ~((n >> 7) * 0xffu);
                        }
                    }
                }
                bad = __reduce_or_sync(0xffffffffu, bad);
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int i = g + 8 * (k >> 1), key = key0 + i, at = pos_of[t][k & 1];
                        if (((bad >> i) & 1) && key <= at && (!A.window || key > at - A.window)) l[t][k & 1] = NAN;
                    }
            }
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                const uint32_t x0 = __byte_perm(v[0][w], v[1][w], 0x5140), x1 = __byte_perm(v[0][w], v[1][w], 0x7362);
                const uint32_t y0 = __byte_perm(v[2][w], v[3][w], 0x5140), y1 = __byte_perm(v[2][w], v[3][w], 0x7362);
                const uint32_t a0[4] = {cvt_lo(x0), cvt_hi(x0), cvt_lo(y0), cvt_hi(y0)};   // elements 4 w, 4 w + 1
                const uint32_t a1[4] = {cvt_lo(x1), cvt_hi(x1), cvt_lo(y1), cvt_hi(y1)};   // elements 4 w + 2, 4 w + 3
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    mma_16816(o[t][2 * w], a0, pb[t][0], pb[t][1]);
                    mma_16816(o[t][2 * w + 1], a1, pb[t][0], pb[t][1]);
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + stage);
        if (++stage == S::STAGES) {
            stage = 0;
            phase ^= 1;
        }

        if (u + 1 < R.end && u + 1 < cur.seg_end()) continue;
        // ---- the segment, or this block's part of it, is done: join the four warps
        fresh = true;
        float *ml = reinterpret_cast<float *>(sm + S::OFF_ML), *oa = reinterpret_cast<float *>(sm + S::OFF_O);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float sum = l[t][x];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                const int r = warp * ROWS + 8 * t + 2 * c + x;
                if (g == 0) {
                    ml[2 * r] = base[t][x];
                    ml[2 * r + 1] = sum;
                }
                float *row = oa + r * S::LD + g * (S::PER + 4);
#pragma unroll
                for (int j = 0; j < NJ; j += 2)
                    *reinterpret_cast<float4 *>(row + 2 * j) =
                        make_float4(o[t][j][x], o[t][j][2 + x], o[t][j + 1][x], o[t][j + 1][2 + x]);
            }
        consumers_sync();
        const bool begins = cur.seg0 >= R.first, ends = cur.seg_end() <= R.end;
        const int tid = threadIdx.x;
        for (int i = tid; i < ROWS * D / 8; i += 32 * WARPS) {
            const int r = i / (D / 8), d = (i % (D / 8)) * 8;
            const int row = cur.rt * ROWS + r, tok = row / A.group, hq = cur.head * A.group + row % A.group;
            if (tok >= cur.p.s.n) continue;
            float mx = -INFINITY, L = 0.0f, v[8] = {};
#pragma unroll
            for (int w = 0; w < WARPS; ++w) mx = fmaxf(mx, ml[(w * ROWS + r) * 2]);
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float mw = ml[(w * ROWS + r) * 2], lw = ml[(w * ROWS + r) * 2 + 1];
                const float f = mw == -INFINITY ? 1.0f : ex2(mw - mx);      // without keys all is 0 (or NaN)
                L = __fmaf_rn(f, lw, L);
                const float4 *p = reinterpret_cast<const float4 *>(oa + (w * ROWS + r) * S::LD + d + 4 * (d / S::PER));
                const float4 x = p[0], y = p[1];
                v[0] = __fmaf_rn(f, x.x, v[0]); v[1] = __fmaf_rn(f, x.y, v[1]);
                v[2] = __fmaf_rn(f, x.z, v[2]); v[3] = __fmaf_rn(f, x.w, v[3]);
                v[4] = __fmaf_rn(f, y.x, v[4]); v[5] = __fmaf_rn(f, y.y, v[5]);
                v[6] = __fmaf_rn(f, y.z, v[6]); v[7] = __fmaf_rn(f, y.w, v[7]);
            }
            if (begins && ends) {
                const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] *= inv;
                store_n(static_cast<TQ *>(const_cast<void *>(A.out.data)) + (int64_t)(cur.p.s.row0 + tok) * A.out.ld_tok +
                            (int64_t)hq * A.out.ld_head + d, v);
                if (A.lse && d == 0)
                    A.lse[(int64_t)(cur.p.s.row0 + tok) * A.q.heads + hq] =
                        L == 0.0f ? -INFINITY : (mx + log2f(L)) * 0.6931471805599453f;
            } else {
                const int64_t slot = ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * ROWS + r;
                store_n(A.part_o + slot * D + d, v);
                if (d == 0) {
                    A.part_ml[slot * 2] = mx;
                    A.part_ml[slot * 2 + 1] = L;
                }
            }
        }
        if (begins && !ends && tid == 0) {
            // the block of the segment's last unit x: the last i with total i / blocks <= x
            A.meta[blockIdx.x] = {cur.b, cur.head, cur.rt, (int32_t)((cur.seg_end() * R.blocks - 1) / R.total)};
        }
        consumers_sync();
        if (u + 1 < R.end) cur.next(A);
    }
}

// One block of threads per (block of the first kernel, row): the segment that
// starts there, its parts summed in order.  Four warps take every fourth part.
template <typename TQ, int D>
__global__ void __launch_bounds__(128) kv_decode_join_kernel(const Args A) {
    constexpr int N = D / 32;
    const int ROWS = A.rows;
    __shared__ float sl[4], so[4][D];
    griddep_wait();
    const Meta M = A.meta[blockIdx.x];
    if (M.last < 0) return;
    const Seq s = seq_info(A.B, M.b, A.T);
    const int r = blockIdx.y, row = M.rt * ROWS + r, tok = row / A.group, hq = M.head * A.group + row % A.group;
    if (tok >= s.n) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int first = blockIdx.x;
    auto slot_of = [&](int i) { return ((int64_t)i * 2 + (i == first ? 1 : 0)) * ROWS + r; };
    // the largest maximum over all parts, then this warp's sums relative to it
    float mx = -INFINITY;
    for (int i = first + lane; i <= M.last; i += 32) mx = fmaxf(mx, A.part_ml[slot_of(i) * 2]);
#pragma unroll
    for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
    float L = 0.0f, v[N] = {};
#pragma unroll 4
    for (int i = first + warp; i <= M.last; i += 4) {
        const int64_t at = slot_of(i);
        const float2 p = *reinterpret_cast<const float2 *>(A.part_ml + at * 2);
        float x[N];
        load_n(A.part_o + at * D + lane * N, x);
        const float f = p.x == -INFINITY ? 1.0f : ex2(p.x - mx);
        L = __fmaf_rn(f, p.y, L);
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = __fmaf_rn(f, x[k], v[k]);
    }
    if (lane == 0) sl[warp] = L;
#pragma unroll
    for (int k = 0; k < N; ++k) so[warp][lane * N + k] = v[k];
    __syncthreads();
    if (warp) return;
    L = (sl[0] + sl[1]) + (sl[2] + sl[3]);
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int d = lane * N + k;
        v[k] = ((so[0][d] + so[1][d]) + (so[2][d] + so[3][d])) * inv;
    }
    store_n(static_cast<TQ *>(const_cast<void *>(A.out.data)) + (int64_t)(s.row0 + tok) * A.out.ld_tok +
                (int64_t)hq * A.out.ld_head + lane * N, v);
    if (A.lse && lane == 0)
        A.lse[(int64_t)(s.row0 + tok) * A.q.heads + hq] = L == 0.0f ? -INFINITY : (mx + log2f(L)) * 0.6931471805599453f;
}

}  // namespace dec
}  // namespace kv
}  // namespace awq
