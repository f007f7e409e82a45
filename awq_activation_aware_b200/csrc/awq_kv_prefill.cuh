// Attention over the paged 8-bit cache for many query rows per key head: prompts,
// chunks of prompts and longer drafts (sm_100a).  See awq_kv.cuh for the cache.
//
// The products bound it (tcgen05, fp16 operands, binary32 accumulators in tensor
// memory): 4 D operations a (row, key).  A block of threads owns 256 query rows, two
// tiles of 128, of one sequence and key head -- a row is (new token, query head of the
// key head's group), so a group shares each key -- and runs over the keys 128 at a time:
//
//   warps 0-3, 4-7   softmax of tile 0, tile 1: one row a thread.  Scores S from tensor
//                    memory, P' = 2^(x + e - base) as fp16 back into the columns S came
//                    from, the row's sum and reference in registers.
//   warps 8-11       codes to fp16 operands, exactly, in 128-byte-swizzled tiles in
//                    shared memory.  One conversion serves 256 rows.
//   warps 12, 13     issue the products of tile 0, tile 1: S = Q K^T from shared memory,
//                    O += P' V with P' from tensor memory and V [key][D] as it lies in
//                    the cache (the operand whose rows run along D).
//   warp 14          brings the codes by TMA, a box per page, and the scales.
//
// The scores of a row tile have two buffers of 64 keys: those of the next step are ready
// when a step's P' is, so the softmax warps never wait for their own products (with one
// buffer of 128 keys a tile went through softmax, products and back, 4900 clocks a turn
// of which the softmax was 2100).  Scales and
// references are those of the kernel for few rows (awq_kv_decode.cuh): the key scale
// multiplies the score, the value scale is an exponent, a row's reference is raised
// only when a score passes it by 2^6, and then its part of O is rescaled in tensor
// memory, after the products of the step before.
//
// With too few blocks of rows to fill the machine the keys are split over several
// blocks of threads, and a second kernel joins their parts in order.
//
// Measured (device, graphs of ten calls on one input): 8192 new tokens, 32 query heads
// over 8, dim 128: 624 us, 881 TFLOP/s (dim 64: 516 us, 533); 512 tokens after 16000, 64
// heads: 289 us, 943 TFLOP/s.  No single unit bounds it.  256 rows x 128 keys take 4800
// clocks, of which the tensor pipe is busy for 2670 (56 %; its operations alone are 2048:
// a product of 64 keys takes 49 clocks for 32, because it reads 128 rows of Q for 64 of K),
// shared memory for 3380 wavefronts (1024 Q, 1024 K and V, 1080 loads and stores, 256 TMA),
// the special functions 46 % and the ALUs 36 %.  The softmax of two warps a scheduler takes
// 2350 clocks by itself, 2720 with products beside.  What is left over is waiting: scores,
// softmax and products of a tile come one after the other, and two tiles and two score
// buffers do not cover all of it.
#pragma once

#include "awq_kv_decode.cuh"

namespace awq {
namespace kv {
namespace pre {

using dec::add_unless_finite;
using dec::cvt_hi;
using dec::cvt_lo;
using dec::ex2;
using dec::kLift;
using dec::kMaxLen;
using dec::kSlack;
using dec::nan_bytes;
using dec::pack_f16;

constexpr int ROWS = 256, TILE = 128;      // query rows of a block of threads, keys per converted tile
constexpr int STEP = 64;                   // keys per softmax step
constexpr int SOFT_WARPS = 8, CONV_WARP = 8, MMA_WARP = 12;
constexpr int THREADS = 32 * 16;          // warp 15 only gives its registers away
constexpr int SOFT_REGS = 176, CONV_REGS = 104, MMA_REGS = 56;     // of 128 a thread at launch
static_assert(2 * SOFT_REGS + CONV_REGS + MMA_REGS == 4 * 128, "the block's registers");
constexpr int LOAD_WARP = 14;
constexpr int SLOTS = 4;                   // tiles whose scales are kept
constexpr int RING = 3;                    // operands, and tiles of codes, on the way

template <int D> struct Shape {
    static constexpr int OPERAND = TILE * D * 2;           // one tile of Q, K or V as fp16
    static constexpr int CODES = TILE * D;                 // one tile of codes
    static constexpr int OFF_Q = 0, OFF_OP = 2 * OPERAND;  // operands: K and V of a tile in turn, RING of them
    static constexpr int OFF_RAW = OFF_OP + RING * OPERAND;        // codes as they come
    static constexpr int OFF_SC = OFF_RAW + RING * CODES;  // float4 [SLOTS][8]: key scale, e, 2^-e of a block's values
    static constexpr int OFF_NAN = OFF_SC + SLOTS * 8 * 16;        // byte [SLOTS][TILE]: the key's values hold a NaN
    static constexpr int OFF_BAR = OFF_NAN + SLOTS * TILE;
    static constexpr int OFF_HERE = OFF_BAR + 256;         // int [RING]: which blocks of the codes are there
    static constexpr int BYTES = OFF_HERE + 16 + 1024;     // + alignment
};

struct Args {
    Cache C;
    Batch B;
    int64_t T;
    Rows q, out;
    float scale_log2;
    int64_t window;
    float *lse;
    int group, splits, max_tokens;
    int box_rows;                          // keys per TMA box: min(page, TILE)
    float *part_ml;                        // [block][ROWS][2]
    float *part_o;                         // [block][ROWS][D]
    uint64_t timeout_ns;
};

// What a block of threads works on.  Blocks that have the most keys come first.
struct Item {
    Seq s;
    int b, head, split;
    int row0, rows;                        // first row, rows of the sequence and head
    int hi;                                // keys that exist for some row
    int t0, nt, ns;                        // first tile of keys, how many (of this split), and their steps
    int all_lo, all_hi;                    // keys that every row sees
    bool any;
};
__device__ __forceinline__ int clamp_pos(int64_t p) { return p < 0 ? 0 : (p < kMaxLen ? (int)p : (int)kMaxLen); }
__device__ __forceinline__ Item item_of(const Args &A, int64_t i) {
    Item w;
    w.split = (int)(i % A.splits);
    i /= A.splits;
    w.head = (int)(i % A.C.heads);
    i /= A.C.heads;
    w.b = (int)(i % A.B.n_seqs);
    const int64_t from_end = i / A.B.n_seqs;
    w.s = seq_info(A.B, w.b, A.T, A.max_tokens);
    w.rows = w.s.n * A.group;
    const int tiles = (w.rows + ROWS - 1) / ROWS;
    w.any = from_end < tiles;
    if (!w.any) return w;
    w.row0 = (int)(tiles - 1 - from_end) * ROWS;
    const int first = w.row0 / A.group;
    int last = (w.row0 + ROWS - 1) / A.group;
    if (last >= w.s.n) last = w.s.n - 1;
    int64_t cap = A.B.max_pages * A.C.page;
    if (cap > kMaxLen) cap = kMaxLen;
    if (w.s.len < cap) cap = w.s.len;
    const int64_t hi = w.s.start + last + 1, lo = A.window ? w.s.start + first + 1 - A.window : 0;
    w.hi = clamp_pos(hi < cap ? hi : cap);
    w.t0 = clamp_pos(lo) / TILE;
    int nt = (w.hi + TILE - 1) / TILE - w.t0;
    if (nt < 0) nt = 0;
    const int per = (nt + A.splits - 1) / A.splits;
    const int j0 = w.split * per;
    w.t0 += j0;
    w.nt = nt - j0 < per ? nt - j0 : per;
    if (w.nt < 0) w.nt = 0;
    w.ns = 2 * w.nt - (w.nt > 0 && (w.t0 + w.nt) * TILE - STEP >= w.hi ? 1 : 0);   // a last half tile without keys is left out
    w.all_hi = clamp_pos(w.s.start + first + 1);
    if (w.all_hi > w.hi) w.all_hi = w.hi;
    w.all_lo = A.window ? clamp_pos(w.s.start + last + 1 - A.window) : 0;
    return w;
}
__device__ __forceinline__ bool whole_tile(const Item &w, int key0) { return key0 >= w.all_lo && key0 + TILE <= w.all_hi; }

// Upper words of the operand descriptors (the lower word is address / 16 | leading offset / 16 << 16): 128-byte
// swizzle, eight rows 1024 bytes apart.  V's elements run along its rows ([key][64] tiles of 128-byte rows):
// eight keys 1024 bytes apart, the next 64 elements of D the leading offset on.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kDescK = 1u << 16, kDescV = (uint32_t)((TILE * 128) >> 4) << 16;
template <uint32_t LOW>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a | LOW), "r"(b | LOW), "r"(idesc), "r"((uint32_t)accumulate), "n"(kDescHigh)
        : "memory");
}
template <uint32_t LOW>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "r"(b | LOW), "r"(idesc), "r"((uint32_t)accumulate), "n"(kDescHigh)
        : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// 64 columns of a warp's 32 lanes, on their way (tmem_arrive makes them usable) -- the registers are not to be
// touched before it.
__device__ __forceinline__ void tmem_issue_64(uint32_t taddr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, "
        "%22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, "
        "%42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, "
        "%62, %63}, [%64];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]),
          "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]),
          "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]),
          "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]),
          "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_arrive(uint32_t (&r)[64]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31]), "+r"(r[32]), "+r"(r[33]), "+r"(r[34]), "+r"(r[35]),
                   "+r"(r[36]), "+r"(r[37]), "+r"(r[38]), "+r"(r[39]), "+r"(r[40]), "+r"(r[41]), "+r"(r[42]),
                   "+r"(r[43]), "+r"(r[44]), "+r"(r[45]), "+r"(r[46]), "+r"(r[47]), "+r"(r[48]), "+r"(r[49]),
                   "+r"(r[50]), "+r"(r[51]), "+r"(r[52]), "+r"(r[53]), "+r"(r[54]), "+r"(r[55]), "+r"(r[56]),
                   "+r"(r[57]), "+r"(r[58]), "+r"(r[59]), "+r"(r[60]), "+r"(r[61]), "+r"(r[62]), "+r"(r[63])
                 :
                 : "memory");
}

__device__ __forceinline__ float4 lds_f4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
    return v;
}
// One step's scores of one row, 64: P' packed, block sums into `add` (scaled by 2^-e), the largest
// z = x + e - base.  MASKED: keys outside [lo, hi) of the step are hidden.  The scales are fetched while
// the scores come: when the tensor core reads its operands from shared memory a load from there takes
// several times as long.
template <bool MASKED>
__device__ __forceinline__ void soft_step(uint32_t s_tmem, uint32_t sc, float rowf, float base, int lo, int hi,
                                          uint32_t (&p)[STEP / 2], float &add, float &top) {
    uint32_t v[64];
    float4 q[4];
    tmem_issue_64(s_tmem, v);
#pragma unroll
    for (int b = 0; b < 4; ++b) q[b] = lds_f4(sc + 16 * b);
    tmem_arrive(v);
    add = 0.0f;
    top = -INFINITY;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const float2 f = make_float2(rowf * q[b].x, rowf * q[b].x), c = make_float2(q[b].y - base, q[b].y - base);
        float2 sum = make_float2(0.0f, 0.0f);
        float big = -INFINITY;
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
            const int i = 16 * b + k;
            float2 z = fma2_rn(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), f, c);
            if (MASKED) {
                if (i < lo || i >= hi) z.x = -INFINITY;
                if (i + 1 < lo || i + 1 >= hi) z.y = -INFINITY;
            }
            big = fmax3(big, z.x, z.y);
            z.x = ex2(z.x);
            z.y = ex2(z.y);
            sum = __fadd2_rn(sum, z);
            p[i / 2] = pack_f16(z.x, z.y);
        }
        add = __fmaf_rn(sum.x + sum.y, q[b].z, add);
        top = fmaxf(top, big);
    }
}

template <int N> __device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

template <typename TQ, int D>
__global__ void __launch_bounds__(THREADS, 1)
kv_prefill_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v, const Args A) {
    using S = Shape<D>;
    extern __shared__ uint8_t raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + S::OFF_BAR);
    uint64_t *qfull = bars, *sfull = bars + 2, *pfull = bars + 6, *pvdone = bars + 10, *drain = bars + 14,     // sfull, pfull, pvdone: [tile][buffer]
             *full = bars + 16, *empty = bars + 19, *rawfull = bars + 22, *rawempty = bars + 25;               // [RING]
    __shared__ uint32_t tmem_base_sm;
    __shared__ int abort_sm;
    volatile int *abort_flag = &abort_sm;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    if (threadIdx.x == 0) {
        abort_sm = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(qfull + i, 128);
            mbar_init(drain + i, 1);
        }
        for (int i = 0; i < RING; ++i) {
            mbar_init(full + i, 128);
            mbar_init(empty + i, 2);
            mbar_init(rawfull + i, 1);
            mbar_init(rawempty + i, 4);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(sfull + i, 1);
            mbar_init(pfull + i, 128);
            mbar_init(pvdone + i, 1);
        }
        fence_mbar_init();
    }
    if (warp == MMA_WARP) {
        tmem_alloc_1(&tmem_base_sm, 512);
        tmem_relinquish_1();
    }
    griddep_launch_dependents();
    griddep_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sm;    // S of tile t, buffer b: at 128 t + 64 b; O: at 256 + 128 t
    const Item w = item_of(A, blockIdx.x);

    if (w.any) {
        const int tiles = w.rows - w.row0 > 128 ? 2 : 1;           // tiles of rows that have any
        if (warp < SOFT_WARPS) {
            regs_up<SOFT_REGS>();
            const int t = warp >> 2, tid = threadIdx.x & 127;
            const int r = 128 * t + tid, row = w.row0 + r;
            const bool mine = row < w.rows;
            const int tok = mine ? row / A.group : w.s.n - 1, hq = w.head * A.group + row % A.group;
            if (t < tiles) {
                const uint32_t lane_base = (uint32_t)(warp & 3) << 21;     // 32 lanes a warp, lane in bits 16 on
                const uint32_t s_tmem = tmem + lane_base + 128 * t, o_tmem = tmem + lane_base + 256 + 128 * t;
                float rowf = A.scale_log2;
                // the row of Q: fp16 into the swizzled tile; bf16 lifted to fp16's upper range by a power of two
                {
                    uint4 v[D / 8];
                    const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const TQ *>(A.q.data) +
                                                                       (int64_t)(w.s.row0 + tok) * A.q.ld_tok +
                                                                       (int64_t)hq * A.q.ld_head);
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) v[i] = mine ? src[i] : make_uint4(0, 0, 0, 0);
                    if (!std::is_same<TQ, __half>::value) {
                        uint32_t top = 0;
#pragma unroll
                        for (int i = 0; i < D / 8; ++i) {
                            const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) top = max(top, max(x[k] & 0x7fffu, (x[k] >> 16) & 0x7fffu));
                        }
                        const int e = min(max((int)(top >> 7) - 127, -100), 126);
                        const float f = pow2(14 - e);
                        rowf *= top < 0x7f80u ? pow2(e - 14) : NAN;
#pragma unroll
                        for (int i = 0; i < D / 8; ++i) {
                            uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                x[k] = pack_f16(__uint_as_float(x[k] << 16) * f, __uint_as_float(x[k] & 0xffff0000u) * f);
                            v[i] = make_uint4(x[0], x[1], x[2], x[3]);
                        }
                    } else {
                        __half2 z = __float2half2_rn(0.0f);
#pragma unroll
                        for (int i = 0; i < D / 8; ++i)
                            z = add_unless_finite(v[i].x, add_unless_finite(v[i].y, add_unless_finite(v[i].z, add_unless_finite(v[i].w, z))));
                        rowf += __low2float(z) + __high2float(z);
                    }
                    const uint32_t dst = smem_u32(sm + S::OFF_Q + t * S::OPERAND);
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) st_shared_v4(dst + (i / 8) * (TILE * 128) + sw128_offset(tid, i % 8), v[i]);
                    fence_proxy_async_smem();
                    mbar_arrive(qfull + t);
                }
                const int64_t at = w.s.start + tok;
                const int row_hi = min(clamp_pos(at + 1), w.hi), row_lo = A.window ? clamp_pos(at + 1 - A.window) : 0;
                float base = 0.0f, l = 0.0f;
                bool has = false, settled = false, ok = true;
                for (int j = 0; j < w.ns && ok; ++j) {
                    const int buf = j & 1;
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(sfull + 2 * t + buf, (j >> 1) & 1, abort_flag, A.timeout_ns));
                    if (!ok) break;
                    tc_fence_after();
                    const int key0 = w.t0 * TILE + j * STEP, slot = (j >> 1) % SLOTS;
                    const bool whole = whole_tile(w, key0 - buf * STEP);
                    const uint32_t sc = smem_u32(sm + S::OFF_SC) + slot * 128 + 64 * buf;
                    uint32_t p[STEP / 2];
                    float add, top;
                    for (int pass = 0;; ++pass) {
                        if (whole) soft_step<false>(s_tmem + 64 * buf, sc, rowf, base, 0, 0, p, add, top);
                        else soft_step<true>(s_tmem + 64 * buf, sc, rowf, base, row_lo - key0, row_hi - key0, p, add, top);
                        if (pass || (settled && !__any_sync(0xffffffffu, top > kLift + kSlack))) break;
                        // seldom: raise the references, and take the step again
                        float up = 0.0f, f = 1.0f;
                        if (has) {
                            up = fmaxf(top - kLift, 0.0f);
                            f = ex2(-up);
                        } else if (top > -INFINITY) {
                            up = top - kLift;              // the row's first keys: its sums are still 0
                            has = true;
                        }
                        base += up;
                        l *= f;
                        if (j > 0 && __any_sync(0xffffffffu, f != 1.0f)) {
                            // the step before is the last whose product may still run: this one's P' is not out yet
                            ok = __all_sync(0xffffffffu, mbar_wait_bounded(pvdone + 2 * t + (buf ^ 1), ((j - 1) >> 1) & 1, abort_flag, A.timeout_ns));
                            tc_fence_after();
#pragma unroll
                            for (int ch = 0; ch < D / 32; ++ch) {
                                float o[32];
                                uint32_t b[32];
                                tmem_ld_32x32b_x32_sync(o_tmem + 32 * ch, o);
#pragma unroll
                                for (int k = 0; k < 32; ++k) b[k] = __float_as_uint(o[k] * f);
                                tmem_st_32x32b_x32(o_tmem + 32 * ch, b);
                            }
                        }
                        settled = __all_sync(0xffffffffu, has);
                    }
                    tmem_st_32x32b_x32(s_tmem + 64 * buf, p);
                    l += add;
                    if (!whole) {                          // NaN values were taken out of the product: into the sums of who sees them
                        const int n = 2 * (j >> 1) + 1;    // the values' place in the ring
                        ok = __all_sync(0xffffffffu, mbar_wait_bounded(full + n % RING, (n / RING) & 1, abort_flag, A.timeout_ns));
                        const uint32_t *bad = reinterpret_cast<const uint32_t *>(sm + S::OFF_NAN + slot * TILE + buf * STEP);
                        for (int k = 0; k < STEP / 4; ++k) {
                            const uint32_t x = bad[k];
                            if (!x) continue;
                            for (int i = 0; i < 4; ++i) {
                                const int key = key0 + 4 * k + i;
                                if (((x >> (8 * i)) & 1) && key >= row_lo && key < row_hi) l = NAN;
                            }
                        }
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(pfull + 2 * t + buf);
                }
                // All products: a barrier that fires once.  (Not the last phases of pvdone one after the other: a warp that
                // comes late finds both complete, and a parity does not tell "two phases on" from "not yet".)
                if (w.ns > 0 && ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(drain + t, 0, abort_flag, A.timeout_ns));
                tc_fence_after();
                if (ok) {
                    const float m = has ? base : -INFINITY;
                    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                    TQ *dst = static_cast<TQ *>(const_cast<void *>(A.out.data)) + (int64_t)(w.s.row0 + tok) * A.out.ld_tok +
                              (int64_t)hq * A.out.ld_head;
                    const int64_t slot = (int64_t)blockIdx.x * ROWS + r;
#pragma unroll
                    for (int ch = 0; ch < D / 32; ++ch) {
                        float o[32];
                        if (w.ns > 0) {
                            tmem_ld_32x32b_x32_sync(o_tmem + 32 * ch, o);
                        } else {
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] = 0.0f;
                        }
                        if (mine) {
#pragma unroll
                            for (int k = 0; k < 32; k += 8) {
                                float x[8];
#pragma unroll
                                for (int n = 0; n < 8; ++n) x[n] = A.splits == 1 ? o[k + n] * inv : o[k + n];
                                if (A.splits == 1) store_n(dst + 32 * ch + k, x);
                                else store_n(A.part_o + slot * D + 32 * ch + k, x);
                            }
                        }
                        __syncwarp();
                    }
                    if (mine) {
                        if (A.splits > 1) {
                            A.part_ml[2 * slot] = m;
                            A.part_ml[2 * slot + 1] = l;
                        } else if (A.lse) {
                            A.lse[(int64_t)(w.s.row0 + tok) * A.q.heads + hq] =
                                l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
                        }
                    }
                }
            }
        } else if (warp < MMA_WARP) {
            regs_down<CONV_REGS>();
            // ---- codes to operands: keys, then values of each tile (keys first: the scores run ahead)
            constexpr int PER = D / 16;                            // 16-byte chunks of codes a row, and of a thread
            constexpr int SKIP = 128 / PER;                        // rows between a thread's chunks
            const int t = threadIdx.x - 32 * CONV_WARP, chunk = t % PER, r0 = t / PER;
            bool ok = true;
            for (int n = 0; n < 2 * w.nt && ok; ++n) {
                const int st = n % RING, key0 = (w.t0 + n / 2) * TILE;
                const uint32_t ph = (n / RING) & 1;
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(rawfull + st, ph, abort_flag, A.timeout_ns));
                if (!ok) break;
                const uint32_t src = smem_u32(sm + S::OFF_RAW + st * S::CODES) + 16 * t;
                const int here = *reinterpret_cast<const volatile int *>(sm + S::OFF_HERE + 4 * st);
                uint4 v[PER];
#pragma unroll
                for (int i = 0; i < PER; ++i) v[i] = dec::lds128(src + 2048 * i);      // rows r0 + SKIP i lie 2048 bytes apart
                __syncwarp();
                if (lane == 0) mbar_arrive(rawempty + st);
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(empty + st, ph ^ 1, abort_flag, A.timeout_ns));
                if (!ok) break;
                const bool whole = whole_tile(w, key0);
                if (!whole || here != 255) {
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        const int row = r0 + SKIP * i;
                        const bool gone = !((here >> (row / 16)) & 1) || key0 + row >= w.hi;
                        uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w}, any = 0;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if (gone) x[k] = 0;
                            if (!whole && (n & 1)) {               // NaN values: out of the product (see soft_step's caller)
                                const uint32_t nan = nan_bytes(x[k]);
                                any |= nan;
                                x[k] &= ~((nan >> 7) * 0xffu);
                            }
                        }
                        v[i] = make_uint4(x[0], x[1], x[2], x[3]);
                        const uint32_t votes = __ballot_sync(0xffffffffu, any != 0);
                        if (chunk == 0 && (n & 1))
                            sm[S::OFF_NAN + (n / 2 % SLOTS) * TILE + row] = (votes >> (lane & ~(PER - 1))) & ((1u << PER) - 1) ? 1 : 0;
                    }
                }
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int row = r0 + SKIP * i;
                    // 16 codes: chunks 2 c and 2 c + 1 of the row's half; lanes of the other half store theirs in
                    // the other order, so that eight lanes always touch eight different bank groups
                    const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                    const uint4 lo = make_uint4(cvt_lo(x[0]), cvt_hi(x[0]), cvt_lo(x[1]), cvt_hi(x[1]));
                    const uint4 hi = make_uint4(cvt_lo(x[2]), cvt_hi(x[2]), cvt_lo(x[3]), cvt_hi(x[3]));
                    const uint32_t half = smem_u32(sm + S::OFF_OP + st * S::OPERAND) + (chunk / 4) * (TILE * 128), c = 2 * (chunk % 4);
                    const bool swap = (chunk / 4) & 1;
                    st_shared_v4(half + sw128_offset(row, c + swap), swap ? hi : lo);
                    st_shared_v4(half + sw128_offset(row, c + 1 - swap), swap ? lo : hi);
                }
                fence_proxy_async_smem();
                mbar_arrive(full + st);
            }
        } else if (regs_down<MMA_REGS>(); w.nt == 0) {
        } else if (warp < MMA_WARP + tiles) {
            // ---- the products of one tile: its O += P' V, then its next scores.  The whole warp runs along and one
            // lane issues, so that addresses stay warp-uniform; with one warp for both tiles, issuing from a
            // single-lane branch, an instruction took 190 clocks to leave (64 is what it computes).
            constexpr uint32_t QK = mma_idesc_f16_f32(128, STEP), PV = mma_idesc_f16_f32(128, D) | (1u << 16);   // V: rows along D
            const int t = warp - MMA_WARP;
            const bool leader = elect_one();
            const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(sm), 0) >> 4, tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t q_lo = base + ((S::OFF_Q + t * S::OPERAND) >> 4), op_lo = base + (S::OFF_OP >> 4);
            const uint32_t s_tmem = tm + 128 * t, o_tmem = tm + 256 + 128 * t;
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t ph) {
                ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar, ph, abort_flag, A.timeout_ns));
            };
            // what both tiles read is free when both have committed; the tile that is not there is committed for
            auto release = [&](uint64_t *bar) {
                mma_commit_1(bar);
                if (tiles == 1) mma_commit_1(bar);
            };
            auto scores = [&](int j) {                             // of step j, into the buffer that P'(j - 2) leaves
                const int n = 2 * (j >> 1), st = n % RING, buf = j & 1;
                if (buf == 0) wait(full + st, (n / RING) & 1);
                if (!ok) return;
                tc_fence_after();
                if (leader) {
                    const uint32_t b = op_lo + st * (S::OPERAND >> 4) + buf * ((STEP * 128) >> 4);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = ((k / 4) * TILE * 128 + (k % 4) * 32) >> 4;
                        mma_ss<kDescK>(s_tmem + 64 * buf, q_lo + off, b + off, QK, k > 0);
                    }
                    mma_commit_1(sfull + 2 * t + buf);
                    if (buf || j + 1 == w.ns) release(empty + st);
                }
                __syncwarp();
            };
            wait(qfull + t, 0);
            scores(0);
            if (w.ns > 1) scores(1);
            for (int j = 0; j < w.ns && ok; ++j) {
                const int n = 2 * (j >> 1) + 1, st = n % RING, buf = j & 1;
                if (buf == 0) wait(full + st, (n / RING) & 1);
                wait(pfull + 2 * t + buf, (j >> 1) & 1);
                if (!ok) break;
                tc_fence_after();
                if (leader) {
                    const uint32_t b = op_lo + st * (S::OPERAND >> 4) + buf * ((STEP * 128) >> 4);
                    mma_ts<kDescV>(o_tmem, s_tmem + 64 * buf, b, PV, j > 0);
#pragma unroll
                    for (int k = 1; k < STEP / 16; ++k)
                        mma_ts<kDescV>(o_tmem, s_tmem + 64 * buf + 8 * k, b + ((k * 2048) >> 4), PV, true);
                    mma_commit_1(pvdone + 2 * t + buf);
                    if (buf || j + 1 == w.ns) release(empty + st);
                }
                __syncwarp();
                if (j + 2 < w.ns) scores(j + 2);
            }
            if (leader) mma_commit_1(drain + t);                   // every product this thread issued has finished when this fires
            __syncwarp();
            mbar_wait_bounded(drain + t, 0, abort_flag, A.timeout_ns);
        } else if (warp == LOAD_WARP) {
            // ---- codes and scales, up to RING tiles ahead; a lane looks after a block of 16 keys (of eight)
            const int page_bits = 31 - __clz(A.C.page), per_box = A.box_rows / kBlock;
            if (lane == 0 && w.s.len > (A.B.max_pages * A.C.page < kMaxLen ? A.B.max_pages * A.C.page : kMaxLen))
                atomicOr(&g_dev_error, kDevErrBadIndex);
            // first row of block `lane & 7` of a tile in the pool; -1: no such keys, or a bad page
            auto page_at = [&](int it) -> int64_t {
                const int pos = (w.t0 + it) * TILE + 16 * (lane & 7);
                return it < w.nt && pos < w.hi ? A.B.pages[(int64_t)w.b * A.B.ld_pages + (pos >> page_bits)] : 0;
            };
            auto row_at = [&](int it, int64_t page) -> int {
                const int pos = (w.t0 + it) * TILE + 16 * (lane & 7);
                if (it >= w.nt || pos >= w.hi) return -1;
                if (page < 0 || page >= A.C.n_pages) {
                    atomicOr(&g_dev_error, kDevErrBadIndex);
                    return -1;
                }
                return (int)((page * A.C.heads + w.head) * A.C.page) + (pos & (A.C.page - 1));
            };
            auto scale_at = [&](int row) { return lane < 16 && row >= 0 ? A.C.scales[lane >> 3][row / 16] : -1.0f; };   // 0-7 keys, 8-15 values
            bool ok = true;
            int row = row_at(0, page_at(0));
            float scale = scale_at(row);
            int64_t page = page_at(1);
            int n = 0;
            for (; n < 2 * w.nt && ok; ++n) {
                const int st = n % RING, it = n / 2;
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(rawempty + st, ((n / RING) & 1) ^ 1, abort_flag, A.timeout_ns));
                if (!ok) break;
                const uint32_t here = __ballot_sync(0xffffffffu, row >= 0) & 255;
                const bool box = lane < 8 && row >= 0 && lane % per_box == 0;
                const int boxes = __popc(__ballot_sync(0xffffffffu, box));
                if ((n & 1) == 0) {
                    const float vs = __shfl_sync(0xffffffffu, scale, (lane & 7) + 8);
                    if (lane < 8) {
                        const uint32_t bits = __float_as_uint(vs);
                        float4 q = make_float4(0.0f, -INFINITY, 1.0f, 0.0f);       // a block that is not there: hidden
                        if (row >= 0) q = make_float4(scale, (float)((int)(bits >> 23) - 127), __uint_as_float(0x7f000000u - bits), 0.0f);
                        reinterpret_cast<float4 *>(sm + S::OFF_SC)[(it % SLOTS) * 8 + lane] = q;
                    }
                }
                if (lane == 0) *reinterpret_cast<volatile int *>(sm + S::OFF_HERE + 4 * st) = (int)here;
                __syncwarp();
                if (lane == 0) mbar_arrive_expect_tx(rawfull + st, boxes * A.box_rows * D);
                __syncwarp();
                if (box)
                    tma_load_2d(sm + S::OFF_RAW + st * S::CODES + lane * kBlock * D, n & 1 ? &tmap_v : &tmap_k, 0, row, rawfull + st);
                if (n & 1) {                                       // on to the next tile; the page numbers after it are on their way
                    row = row_at(it + 1, page);
                    scale = scale_at(row);
                    page = page_at(it + 2);
                }
            }
            if (!ok) {                                             // given up: let the copies in flight land
                for (int k = n > RING ? n - RING : 0; k < n; ++k) {
                    const uint64_t t0 = global_timer_ns();
                    while (!mbar_try_wait_hint(rawfull + k % RING, (k / RING) & 1, 20000u))
                        if (global_timer_ns() - t0 > A.timeout_ns) break;
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == MMA_WARP) {
        tc_fence_after();
        tmem_dealloc_1(tmem, 512);
    }
}

// One warp per (row, query head): the parts of its splits, summed in order.
template <typename TQ, int D>
__global__ void __launch_bounds__(256) kv_prefill_join_kernel(const Args A) {
    constexpr int N = D / 32;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int64_t t = i / A.q.heads;
    const int hq = (int)(i % A.q.heads);
    if (t >= A.T) return;
    const int b = seq_of_row(A.B, t);
    if (b < 0) return;
    const Seq s = seq_info(A.B, b, A.T, A.max_tokens);
    if (t - s.row0 >= s.n) return;
    const int row = (int)(t - s.row0) * A.group + hq % A.group;
    const int tiles = (s.n * A.group + ROWS - 1) / ROWS;
    const int64_t from_end = tiles - 1 - row / ROWS;
    const int64_t block0 = ((from_end * A.B.n_seqs + b) * A.C.heads + hq / A.group) * A.splits;
    const int r = row % ROWS;
    float mx = -INFINITY;
    for (int k = 0; k < A.splits; ++k) mx = fmaxf(mx, A.part_ml[((block0 + k) * ROWS + r) * 2]);
    float L = 0.0f, v[N] = {};
#pragma unroll 4
    for (int k = 0; k < A.splits; ++k) {
        const int64_t at = (block0 + k) * ROWS + r;
        const float2 p = *reinterpret_cast<const float2 *>(A.part_ml + at * 2);
        float x[N];
        load_n(A.part_o + at * D + lane * N, x);
        const float f = dec::part_weight(p.x, mx);
        L = __fmaf_rn(f, p.y, L);
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] = __fmaf_rn(f, x[n], v[n]);
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] *= inv;
    store_n(static_cast<TQ *>(const_cast<void *>(A.out.data)) + t * A.out.ld_tok + (int64_t)hq * A.out.ld_head + lane * N, v);
    if (A.lse && lane == 0) A.lse[t * A.q.heads + hq] = L == 0.0f ? -INFINITY : (mx + log2f(L)) * 0.6931471805599453f;
}

}  // namespace pre
}  // namespace kv
}  // namespace awq
