// Host side of the cache operators of include/awq.h: argument checks, workspace
// layout and launches.  A translation unit of its own, so that both compile at
// once; it has its own device error word, which awq_get_status() reads too.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "awq.h"
#include "awq_host.h"

#define g_dev_error g_kv_dev_error             // this unit's word, defined with the helpers of awq_device.cuh
#include "awq_kv.cuh"
#include "awq_kv_decode.cuh"
#include "awq_kv_prefill.cuh"

namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
awq_status cuda_status(cudaError_t e) { return e == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA; }

// The current device's SM count, queried once; it must be an sm_100 part.
struct DevInfo {
    int sms = 0, cc_major = 0;
};
awq_status device_info(DevInfo &out) {
    static std::mutex mu;
    static DevInfo known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return AWQ_ERR_CUDA;
    std::lock_guard<std::mutex> lk(mu);
    DevInfo &d = known[dev];
    if (d.sms == 0 && (cudaDeviceGetAttribute(&d.cc_major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
                       cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)) {
        d.sms = 0;
        return AWQ_ERR_CUDA;
    }
    if (d.cc_major != 10) return AWQ_ERR_UNSUPPORTED;
    out = d;
    return AWQ_OK;
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (no -lcuda).
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

bool kv_dtype_ok(int t) { return t >= AWQ_F32 && t <= AWQ_BF16; }

// Rows whose accesses may be 16 bytes wide: aligned base, strides of whole
// 8-element groups.
bool kv_rows_aligned(const awq_rows &r) {
    return aligned16(r.data) && r.token_stride % 8 == 0 && r.head_stride % 8 == 0;
}
// Element-aligned base of a known type.
bool kv_rows_base(const awq_rows &r) {
    return r.data && kv_dtype_ok(r.dtype) && reinterpret_cast<uintptr_t>(r.data) % (r.dtype == AWQ_F32 ? 4 : 2) == 0;
}
bool kv_rows_in(const awq_rows &r) {
    return kv_rows_base(r) && r.heads >= 1 && r.token_stride >= 0 && r.head_stride >= 0;
}
// Written rows must not overlap: heads inside a token, or tokens inside a head.
bool kv_rows_out(const awq_rows &r, int64_t T, int64_t D) {
    if (!kv_rows_base(r) || r.heads < 1 || r.head_stride < D || r.token_stride < D) return false;
    if (r.heads == 1 || T == 1) return true;
    return r.token_stride >= (r.heads - 1) * r.head_stride + D || r.head_stride >= (T - 1) * r.token_stride + D;
}
awq::kv::Rows kv_rows(const awq_rows &r) { return {r.data, r.token_stride, r.head_stride, r.heads, r.dtype}; }

bool kv_cache_ok(const awq_kv_cache &c) {
    if (!c.k_codes || !c.v_codes || !c.k_scales || !c.v_scales || !aligned16(c.k_codes) || !aligned16(c.v_codes) ||
        !aligned16(c.k_scales) || !aligned16(c.v_scales))
        return false;
    if (c.page_size != 16 && c.page_size != 32 && c.page_size != 64 && c.page_size != 128 && c.page_size != 256)
        return false;
    if (c.head_dim != 64 && c.head_dim != 128) return false;
    // rows of all pages are addressed by a 32-bit tensor coordinate
    return c.heads >= 1 && c.heads <= 1024 && c.n_pages >= 1 &&
           c.n_pages <= kMaxDim / ((int64_t)c.heads * c.page_size);
}
awq::kv::Cache kv_cache(const awq_kv_cache &c) {
    awq::kv::Cache k;
    k.codes[0] = static_cast<uint8_t *>(c.k_codes);
    k.codes[1] = static_cast<uint8_t *>(c.v_codes);
    k.scales[0] = c.k_scales;
    k.scales[1] = c.v_scales;
    k.n_pages = c.n_pages;
    k.page = c.page_size;
    k.heads = c.heads;
    k.dim = c.head_dim;
    return k;
}
bool kv_batch_ok(const awq_kv_batch &b, int64_t T) {
    if (!b.seq_lens || !b.pages || b.n_seqs < 1 || b.n_seqs > (1 << 20) || b.max_pages < 1 || b.max_pages > kMaxDim ||
        b.page_stride < b.max_pages)
        return false;
    return T >= 1 && T <= kMaxDim && (b.cu_tokens || T == b.n_seqs);
}
awq::kv::Batch kv_batch(const awq_kv_batch &b) {
    return {b.seq_lens, b.cu_tokens, b.pages, b.page_stride, b.max_pages, (int)b.n_seqs};
}
// A table for rotations of the first rot_dim of D elements.
bool kv_rope_ok(const awq_rope_cfg &r, int64_t D) {
    return r.table && aligned16(r.table) && r.n_pos >= 1 && r.n_pos <= kMaxDim && r.rot_dim >= 2 && r.rot_dim <= D &&
           r.rot_dim % 2 == 0 && (r.layout == AWQ_ROPE_HALF || r.layout == AWQ_ROPE_INTERLEAVED);
}
awq::kv::Rope kv_rope(const awq_rope_cfg &r) {
    return {reinterpret_cast<const float2 *>(r.table), r.n_pos, r.rot_dim, r.layout == AWQ_ROPE_INTERLEAVED};
}

// A launch whose start may overlap the end of the kernel before it on the stream
// (programmatic dependent launch): the kernel waits for that one (griddep_wait)
// before it reads or writes anything in global memory, in every block of threads.
// Calls in a row, with and without: rope of 16384 tokens 52.6 and 55.1 us, append of
// seven prompts 87.0 and 89.9, of 256 single tokens (replayed) 6.5 and 7.2.
template <typename... P>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, P... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Threads of a block that rotates: enough for one round of loads a token; blocks of them make 1024 an SM.
int rope_threads(int64_t items, bool interleaved) {
    const int64_t want = (items / (interleaved ? 4 : 2) + 31) / 32 * 32;
    return want < 32 ? 32 : (want > 128 ? 128 : (int)want);
}

// Blocks that stay, 1024 threads an SM.
template <typename TI, typename TO>
cudaError_t launch_rope(const awq::kv::RopeArgs &A, bool vec, int sms, cudaStream_t st) {
    const int64_t items = (int64_t)A.x.heads * (vec ? awq::kv::rope_items(A.dim, A.r.rot, A.r.interleaved) : A.dim / 2);
    const int threads = rope_threads(items, A.r.interleaved);
    const int64_t grid = std::min<int64_t>(A.T, (int64_t)sms * (1024 / threads));
    auto kernel = !vec              ? awq::kv::rope_any_kernel
                  : A.r.interleaved ? awq::kv::rope_kernel<TI, TO, true>
                                    : awq::kv::rope_kernel<TI, TO, false>;
    return launch_overlapped(kernel, dim3((unsigned)grid), threads, 0, st, A);
}
template <typename TI>
cudaError_t launch_rope_to(const awq::kv::RopeArgs &A, bool vec, int sms, cudaStream_t st) {
    if (A.y.dtype == awq::kv::kF32) return launch_rope<TI, float>(A, vec, sms, st);
    if (A.y.dtype == awq::kv::kF16) return launch_rope<TI, __half>(A, vec, sms, st);
    return launch_rope<TI, __nv_bfloat16>(A, vec, sms, st);
}

template <typename TI, typename TO, bool INTER>
auto launch_append_of(int dim, bool ragged) {
    return ragged ? (dim == 64 ? awq::kv::kv_append_kernel<TI, TO, 64, 4, INTER> : awq::kv::kv_append_kernel<TI, TO, 128, 4, INTER>)
                  : (dim == 64 ? awq::kv::kv_append_kernel<TI, TO, 64, 1, INTER> : awq::kv::kv_append_kernel<TI, TO, 128, 1, INTER>);
}
template <typename TI, typename TO>
cudaError_t launch_append_dim(const awq::kv::AppendArgs &A, dim3 grid, cudaStream_t st) {
    const bool ragged = A.B.cu != nullptr;
    auto kernel = A.r.interleaved ? launch_append_of<TI, TO, true>(A.C.dim, ragged) : launch_append_of<TI, TO, false>(A.C.dim, ragged);
    return launch_overlapped(kernel, grid, awq::kv::kAppendThreads, 0, st, A);
}
template <typename TI>
cudaError_t launch_append(const awq::kv::AppendArgs &A, dim3 grid, cudaStream_t st) {
    if (A.q_out.dtype == awq::kv::kF16) return launch_append_dim<TI, __half>(A, grid, st);
    return launch_append_dim<TI, __nv_bfloat16>(A, grid, st);
}

// Codes as a 2-D tensor of bytes [n_pages * heads * page][D], boxes of `box_rows`
// rows, swizzled over their width or as they are.
bool encode_kv_map(CUtensorMap *m, const void *codes, const awq::kv::Cache &c, int box_rows, bool swizzle = true) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)c.dim, (cuuint64_t)(c.n_pages * c.heads * c.page)};
    cuuint64_t strides[1] = {(cuuint64_t)c.dim};
    cuuint32_t box[2] = {(cuuint32_t)c.dim, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(codes), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE,
              !swizzle ? CU_TENSOR_MAP_SWIZZLE_NONE
                       : (c.dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B),
              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Runs `set` the first time it is reached on the current device (one flag per use of a lambda type).
template <typename F>
cudaError_t once_per_device(F set) {
    static std::atomic<bool> done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
    if (!done[dev].load(std::memory_order_acquire)) {
        if ((e = set()) != cudaSuccess) return e;
        done[dev].store(true, std::memory_order_release);
    }
    return cudaSuccess;
}

// Most blocks of the decode attention's first kernel, and rows of a tile.
constexpr int64_t kDecMaxGrid = 512, kDecMaxRows = 32;
struct DecWs {
    size_t ml_off, o_off, total;
};
DecWs dec_ws(int D) {
    DecWs w;
    w.ml_off = round_up(kDecMaxGrid * sizeof(awq::kv::dec::Meta), 256);
    w.o_off = w.ml_off + round_up(kDecMaxGrid * 2 * kDecMaxRows * 2 * 4, 256);
    w.total = w.o_off + round_up((size_t)kDecMaxGrid * 2 * kDecMaxRows * D * 4, 256);
    return w;
}

template <typename TQ, int D, int NT, int GR>
cudaError_t launch_decode_rows(awq::kv::dec::Args &A, int sms,
                               int64_t most_rows, cudaStream_t st) {
    using S = awq::kv::dec::Shape<D, NT, GR>;
    auto kernel = awq::kv::dec::kv_decode_kernel<TQ, D, NT, GR>;
    A.rows = S::ROWS;
    A.tile = S::TILE;
    A.box_rows = std::min(A.C.page, S::TILE);
    CUtensorMap mk, mv;
    if (!encode_kv_map(&mk, A.C.codes[0], A.C, A.box_rows) || !encode_kv_map(&mv, A.C.codes[1], A.C, A.box_rows))
        return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)std::min<int64_t>((int64_t)S::BLOCKS * sms, kDecMaxGrid);
    const unsigned rows = (unsigned)std::min<int64_t>(most_rows, S::ROWS);
    cudaError_t e = once_per_device([&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::BYTES);
    });
    if (e != cudaSuccess) return e;
    A.rt_most = (int)((most_rows + S::ROWS - 1) / S::ROWS);
    const int64_t segments = (int64_t)A.B.n_seqs * A.C.heads * A.rt_most;
    A.by_segment = segments <= grid;
    e = launch_overlapped(kernel, dim3(grid), awq::kv::dec::THREADS, S::BYTES, st, mk, mv, (const awq::kv::dec::Args)A);
    if (e != cudaSuccess) return e;
    constexpr int W = awq::kv::dec::JOIN_WARPS;
    // Dim 64: the join is launched plainly, dim 128: early.  Calls in a row, early and plainly (us): dim 64, 24 / 12 / 6
    // sequences of 32 heads of their own, window 2048: 58, 34, 24 and 43, 29, 20.5; 64 x 64 heads over 8, to 8192 keys: 69 and
    // 57; 24 and 6 x 32 over 8: 29.5, 18.6 and 30.8, 19.4.  Dim 128: the same three of own heads: 65, 38, 24.3 and 65, 39.5,
    // 26; 64 x 64 over 8: 96.8 and 98.4; 32 over 8: 44.6, 18.5 and 46.4, 20.4; 131072 keys: 52.9 and 53.8; but 24 x 32 own heads
    // of 2048 keys: 79 and 74.6.  The dimension stands for what it mostly goes with, and no more; why an early start can cost
    // that much, the counters of a kernel by itself do not show.
    const dim3 joins = A.by_segment ? dim3((unsigned)segments, rows) : dim3(grid, (rows + W - 1) / W);
    auto join = A.by_segment ? awq::kv::dec::kv_decode_join_kernel<TQ, D, W> : awq::kv::dec::kv_decode_join_kernel<TQ, D, 1>;
    if (D == 128) return launch_overlapped(join, joins, 32 * W, 0, st, (const awq::kv::dec::Args)A);
    join<<<joins, 32 * W, 0, st>>>(A);
    return cudaGetLastError();
}
// Tiles of 8 query rows while a sequence has no more: half the products of 16 (131072 keys of 8 heads: 52 and 56 us).
// Tiles of 32 take the keys once for two groups of warps, which convert them each (88 us).
template <typename TQ, int D>
cudaError_t launch_decode(awq::kv::dec::Args &A, int sms,
                          int64_t most_rows, cudaStream_t st) {
    if (most_rows <= 8) return launch_decode_rows<TQ, D, 1, 1>(A, sms, most_rows, st);
    if (most_rows <= 16) return launch_decode_rows<TQ, D, 2, 1>(A, sms, most_rows, st);
    return launch_decode_rows<TQ, D, 2, 2>(A, sms, most_rows, st);
}

// The kernel for many rows: blocks of threads, and splits of the keys while they do not fill the machine.
constexpr int64_t kPreSplitBlocks = 148;
int64_t pre_items(const awq::kv::Batch &B, const awq::kv::Cache &C, int64_t most_rows) {
    return (int64_t)B.n_seqs * C.heads * ((most_rows + awq::kv::pre::ROWS - 1) / awq::kv::pre::ROWS);
}
size_t pre_ml_bytes() { return kPreSplitBlocks * awq::kv::pre::ROWS * 2 * 4; }
size_t pre_ws(int D) { return pre_ml_bytes() + (size_t)kPreSplitBlocks * awq::kv::pre::ROWS * D * 4; }

template <typename TQ, int D>
cudaError_t launch_prefill(const awq::kv::dec::Args &P, int64_t most_rows, void *ws, cudaStream_t st) {
    using S = awq::kv::pre::Shape<D>;
    auto kernel = awq::kv::pre::kv_prefill_kernel<TQ, D>;
    cudaError_t e = once_per_device([&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::BYTES);
    });
    if (e != cudaSuccess) return e;
    const int64_t items = pre_items(P.B, P.C, most_rows);
    const int64_t key_tiles = (P.B.max_pages * P.C.page + awq::kv::pre::TILE - 1) / awq::kv::pre::TILE;
    const int64_t splits = std::max<int64_t>(1, std::min(kPreSplitBlocks / items, key_tiles / 2));
    if (items * splits > kMaxDim) return cudaErrorInvalidConfiguration;
    awq::kv::pre::Args A;
    A.C = P.C;
    A.B = P.B;
    A.T = P.T;
    A.q = P.q;
    A.out = P.out;
    A.scale_log2 = P.scale_log2;
    A.window = P.window;
    A.lse = P.lse;
    A.group = P.group;
    A.splits = (int)splits;
    A.max_tokens = P.max_tokens;
    A.part_ml = static_cast<float *>(ws);
    A.part_o = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + pre_ml_bytes());
    A.timeout_ns = P.timeout_ns;
    A.box_rows = std::min(P.C.page, awq::kv::pre::TILE);
    CUtensorMap mk, mv;
    if (!encode_kv_map(&mk, P.C.codes[0], P.C, A.box_rows, false) || !encode_kv_map(&mv, P.C.codes[1], P.C, A.box_rows, false))
        return cudaErrorInvalidValue;
    e = launch_overlapped(kernel, dim3((unsigned)(items * splits)), awq::kv::pre::THREADS, S::BYTES, st, mk, mv,
                          (const awq::kv::pre::Args)A);
    if (e != cudaSuccess || splits == 1) return e;
    const int64_t warps = P.T * P.q.heads;
    return launch_overlapped(awq::kv::pre::kv_prefill_join_kernel<TQ, D>, dim3((unsigned)((warps + 7) / 8)), 256, 0, st,
                             (const awq::kv::pre::Args)A);
}
// Up to kDecRows rows of a sequence and key head the kernel for few rows, from there on the other: over 131072 keys of 8
// heads the first takes 88 us with 32 rows, the other 122 with 40; over 8 sequences of 8000 keys 61 and 74.  More rows
// would be a second tile, and every key read twice.
constexpr int64_t kDecRows = 32;
template <typename TQ, int D>
cudaError_t launch_attention(awq::kv::dec::Args &A, int sms, int64_t most_rows, void *ws, cudaStream_t st) {
    if (most_rows <= kDecRows) return launch_decode<TQ, D>(A, sms, most_rows, st);
    return launch_prefill<TQ, D>(A, most_rows, ws, st);
}

}  // namespace

extern "C" {

awq_status awq_rope_table(int64_t n_pos, int32_t rot_dim, double base, awq_rope_scaling sc, float *table,
                          void *stream) {
    if (!table || !aligned16(table) || n_pos < 1 || n_pos > kMaxDim || rot_dim < 2 || rot_dim % 2 || rot_dim > 65536 ||
        !(base > 1.0 && base <= 1e12))
        return AWQ_ERR_INVALID_ARG;
    if (sc.kind < AWQ_ROPE_PLAIN || sc.kind > AWQ_ROPE_YARN) return AWQ_ERR_INVALID_ARG;
    if (sc.kind != AWQ_ROPE_PLAIN && !(sc.factor >= 1.0 && sc.factor <= 1e6)) return AWQ_ERR_INVALID_ARG;
    if (sc.kind == AWQ_ROPE_NTK && rot_dim < 4) return AWQ_ERR_INVALID_ARG;
    awq::kv::TableArgs A;
    A.table = reinterpret_cast<float2 *>(table);
    A.n_pos = n_pos;
    A.half = rot_dim / 2;
    A.log_base = std::log(base);
    A.inv_factor = 1.0;
    A.ramp_lo = 0.0;
    A.ramp_hi = 1.0;
    A.magnitude = 1.0;
    if (sc.kind == AWQ_ROPE_LINEAR) {
        A.inv_factor = 1.0 / sc.factor;
        A.ramp_lo = -1.0;                      // every pair past the ramp
        A.ramp_hi = 0.0;
    } else if (sc.kind == AWQ_ROPE_NTK) {
        A.log_base += std::log(sc.factor) * rot_dim / (rot_dim - 2);
    } else if (sc.kind == AWQ_ROPE_YARN) {
        if (!(sc.original >= 1.0 && sc.original <= 1e12) || !(sc.beta_fast > 0.0 && sc.beta_fast <= 1e6) ||
            !(sc.beta_slow > 0.0 && sc.beta_slow <= sc.beta_fast) || !(sc.magnitude >= 0.0 && sc.magnitude <= 1e6))
            return AWQ_ERR_INVALID_ARG;
        const double two_pi = 6.283185307179586;
        const double lo = std::floor(rot_dim * std::log(sc.original / (sc.beta_fast * two_pi)) / (2.0 * A.log_base));
        const double hi = std::ceil(rot_dim * std::log(sc.original / (sc.beta_slow * two_pi)) / (2.0 * A.log_base));
        A.inv_factor = 1.0 / sc.factor;
        A.ramp_lo = lo > 0.0 ? lo : 0.0;
        A.ramp_hi = hi < rot_dim - 1 ? hi : rot_dim - 1;
        if (A.ramp_hi - A.ramp_lo < 0.001) A.ramp_hi = A.ramp_lo + 0.001;
        A.magnitude = sc.magnitude > 0.0 ? sc.magnitude : 0.1 * std::log(sc.factor) + 1.0;
    }
    DevInfo d;
    if (awq_status e = device_info(d)) return e;
    const int grid = (int)std::min<int64_t>((n_pos * A.half + 255) / 256, 16 * d.sms);
    awq::kv::rope_table_kernel<<<grid, 256, 0, (cudaStream_t)stream>>>(A);
    return cuda_status(cudaGetLastError());
}

awq_status awq_rope(awq_rows x, awq_rows y, int64_t T, int32_t head_dim, const int32_t *positions, awq_rope_cfg r,
                    int32_t inverse, void *stream) {
    if (T < 1 || T > kMaxDim || head_dim < 2 || head_dim % 2 || head_dim > 65536 || !positions ||
        (inverse != 0 && inverse != 1) || !kv_rope_ok(r, head_dim) || !kv_rows_in(x) || !kv_rows_out(y, T, head_dim) ||
        x.heads != y.heads)
        return AWQ_ERR_INVALID_ARG;
    if ((int64_t)x.heads * head_dim > kMaxDim) return AWQ_ERR_INVALID_ARG;     // the kernels count a token's elements in 32 bits
    // in place: element for element the same memory, or another array altogether
    if (x.data == y.data &&
        (x.dtype != y.dtype || x.token_stride != y.token_stride || x.head_stride != y.head_stride))
        return AWQ_ERR_INVALID_ARG;
    DevInfo d;
    if (awq_status e = device_info(d)) return e;
    awq::kv::RopeArgs A;
    A.T = T;
    A.x = kv_rows(x);
    A.y = kv_rows(y);
    A.dim = head_dim;
    A.inverse = inverse;
    A.positions = positions;
    A.r = kv_rope(r);
    const bool vec = kv_rows_aligned(x) && kv_rows_aligned(y) && head_dim % 8 == 0 &&
                     r.rot_dim % (A.r.interleaved ? 8 : 16) == 0;
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = x.dtype == AWQ_F32   ? launch_rope_to<float>(A, vec, d.sms, st)
                    : x.dtype == AWQ_F16 ? launch_rope_to<__half>(A, vec, d.sms, st)
                                         : launch_rope_to<__nv_bfloat16>(A, vec, d.sms, st);
    return cuda_status(e);
}

awq_status awq_kv_append(awq_kv_cache c, awq_kv_batch b, int64_t T, awq_rows k, awq_rows v, awq_rows q, awq_rows q_out,
                         awq_rope_cfg r, void *stream) {
    if (!kv_cache_ok(c) || !kv_batch_ok(b, T)) return AWQ_ERR_INVALID_ARG;
    if (!kv_rows_in(k) || !kv_rows_in(v) || !kv_rows_aligned(k) || !kv_rows_aligned(v) || k.dtype != v.dtype ||
        k.heads != c.heads || v.heads != c.heads)
        return AWQ_ERR_INVALID_ARG;
    if (r.table && !kv_rope_ok(r, c.head_dim)) return AWQ_ERR_INVALID_ARG;
    if (q.data) {
        if (!r.table || !kv_rows_in(q) || !kv_rows_out(q_out, T, c.head_dim) || !kv_rows_aligned(q) ||
            !kv_rows_aligned(q_out) || q.dtype != k.dtype || q_out.dtype == AWQ_F32 || q.heads != q_out.heads || q.heads > 65536)
            return AWQ_ERR_INVALID_ARG;
        if (q.data == q_out.data && (q.dtype != q_out.dtype || q.token_stride != q_out.token_stride ||
                                     q.head_stride != q_out.head_stride))
            return AWQ_ERR_INVALID_ARG;
    }
    DevInfo d;
    if (awq_status e = device_info(d)) return e;
    awq::kv::AppendArgs A;
    A.C = kv_cache(c);
    A.B = kv_batch(b);
    A.T = T;
    A.kv[0] = kv_rows(k);
    A.kv[1] = kv_rows(v);
    A.q = kv_rows(q);
    A.q_out = kv_rows(q_out);
    if (!q.data) A.q_out.dtype = awq::kv::kF16;
    A.r = r.table ? kv_rope(r) : awq::kv::Rope{nullptr, 0, 0, 0};
    const int chunk = b.cu_tokens ? 16 : 1, teams = awq::kv::kAppendThreads / 32 / (b.cu_tokens ? 4 : 1);
    const int64_t chunks = (T + chunk - 1) / chunk;
    // a team takes about one (block, head) while that does not make far too many blocks of threads
    A.parts = (c.heads + teams - 1) / teams;
    while (A.parts > 1 && chunks * A.parts > 16 * d.sms) A.parts = (A.parts + 1) / 2;
    A.appends = chunks * A.parts;
    A.q_rows = (int)std::min<int64_t>(8, std::max<int64_t>(1, T / (8 * d.sms)));
    const int64_t blocks = A.appends + (q.data ? (T + A.q_rows - 1) / A.q_rows : 0);
    if (blocks > kMaxDim) return AWQ_ERR_INVALID_ARG;
    const dim3 grid((unsigned)blocks);
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = k.dtype == AWQ_F32   ? launch_append<float>(A, grid, st)
                    : k.dtype == AWQ_F16 ? launch_append<__half>(A, grid, st)
                                         : launch_append<__nv_bfloat16>(A, grid, st);
    return cuda_status(e);
}

size_t awq_kv_attention_workspace_bytes(awq_kv_cache c, int64_t T, int32_t q_heads, int32_t max_tokens) {
    if (T < 1 || q_heads < 1 || max_tokens < 1 || c.head_dim < 1) return 0;
    const int64_t rows = c.heads < 1 ? 1 : (int64_t)max_tokens * (q_heads / c.heads);
    return rows <= kDecRows ? dec_ws(c.head_dim).total : pre_ws(c.head_dim);
}

awq_status awq_kv_attention(awq_kv_cache c, awq_kv_batch b, int64_t T, awq_rows q, awq_rows out, float scale,
                            int32_t max_tokens, int64_t window, float *lse, void *ws, size_t ws_bytes, void *stream) {
    if (!kv_cache_ok(c) || !kv_batch_ok(b, T)) return AWQ_ERR_INVALID_ARG;
    if (!kv_rows_in(q) || !kv_rows_out(out, T, c.head_dim) || !kv_rows_aligned(q) || !kv_rows_aligned(out) ||
        (q.dtype != AWQ_F16 && q.dtype != AWQ_BF16) || out.dtype != q.dtype || q.heads != out.heads ||
        q.heads % c.heads || q.heads > 65535 || out.data == q.data)
        return AWQ_ERR_INVALID_ARG;
    if (!(scale > 0.0f && scale <= 1e6f) || window < 0 || max_tokens < 1 || (!b.cu_tokens && max_tokens != 1) ||
        reinterpret_cast<uintptr_t>(lse) % 4 || T > kMaxDim / (2 * q.heads) || max_tokens > kMaxDim / (2 * q.heads))
        return AWQ_ERR_INVALID_ARG;
    if (!ws || ws_bytes < awq_kv_attention_workspace_bytes(c, T, q.heads, max_tokens) ||
        (reinterpret_cast<uintptr_t>(ws) & 255u))
        return AWQ_ERR_WORKSPACE;
    DevInfo d;
    if (awq_status e = device_info(d)) return e;
    awq::kv::dec::Args A;
    A.C = kv_cache(c);
    A.B = kv_batch(b);
    A.T = T;
    A.q = kv_rows(q);
    A.out = kv_rows(out);
    A.scale_log2 = scale * 1.4426950408889634f;
    A.window = window;
    A.lse = lse;
    A.group = q.heads / c.heads;
    A.max_tokens = max_tokens;
    const DecWs w = dec_ws(c.head_dim);
    A.meta = static_cast<awq::kv::dec::Meta *>(ws);
    A.part_ml = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + w.ml_off);
    A.part_o = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + w.o_off);
    A.timeout_ns = (uint64_t)awq_host::wait_timeout_ms() * 1000000ull;
    const int64_t most = (int64_t)max_tokens * A.group;
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (c.head_dim == 64)
        e = q.dtype == AWQ_F16 ? launch_attention<__half, 64>(A, d.sms, most, ws, st)
                               : launch_attention<__nv_bfloat16, 64>(A, d.sms, most, ws, st);
    else
        e = q.dtype == AWQ_F16 ? launch_attention<__half, 128>(A, d.sms, most, ws, st)
                               : launch_attention<__nv_bfloat16, 128>(A, d.sms, most, ws, st);
    if (e != cudaSuccess) return AWQ_ERR_CUDA;
    return cuda_status(cudaGetLastError());
}

}  // extern "C"

bool awq_host::take_kv_errors(unsigned *flags) {
    if (cudaMemcpyFromSymbol(flags, awq::g_dev_error, sizeof(*flags)) != cudaSuccess) return false;
    const unsigned zero = 0;
    return !*flags || cudaMemcpyToSymbol(awq::g_dev_error, &zero, sizeof(zero)) == cudaSuccess;
}
