"""The operators between a decode step's quantized projections: rotary
positions, a paged 8-bit cache of keys and values, and the attention over it.

Like the rest of the binding these functions only check and marshal arguments
into the C ABI of ``include/awq.h``.  A cache is a plain dict of tensors
(:func:`kv_cache`); rows are tensors [T, heads, head_dim] whose last dimension
is contiguous, so slices of one fused projection can be passed as they are.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math

import torch

from .persist import _check_config

__all__ = ["rope_table", "rope", "kv_cache", "kv_append", "kv_attention", "kv_attention_workspace_bytes",
           "attention_step"]

_P, _i64, _i32, _f64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_double
_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_LAYOUTS = {"half": 0, "interleaved": 1}
_SCALINGS = {None: 0, "none": 0, "linear": 1, "ntk": 2, "yarn": 3}
_MAX = (1 << 31) - 1                                       # of the ABI's 32-bit fields: ctypes would wrap what is larger
_CODES = (torch.float8_e4m3fn, torch.uint8)


class Rows(ctypes.Structure):
    _fields_ = [("data", _P), ("token_stride", _i64), ("head_stride", _i64), ("heads", _i32), ("dtype", _i32)]


class RopeScaling(ctypes.Structure):
    _fields_ = [("kind", _i32), ("factor", _f64), ("original", _f64), ("beta_fast", _f64), ("beta_slow", _f64),
                ("magnitude", _f64)]


class RopeCfg(ctypes.Structure):
    _fields_ = [("table", _P), ("n_pos", _i64), ("rot_dim", _i32), ("layout", _i32)]


class KVCache(ctypes.Structure):
    _fields_ = [("k_codes", _P), ("v_codes", _P), ("k_scales", _P), ("v_scales", _P), ("n_pages", _i64),
                ("page_size", _i32), ("heads", _i32), ("head_dim", _i32)]


class KVBatch(ctypes.Structure):
    _fields_ = [("seq_lens", _P), ("cu_tokens", _P), ("pages", _P), ("n_seqs", _i64), ("page_stride", _i64),
                ("max_pages", _i64)]


def declare(L):
    """The entry points' signatures (called once, when the library is loaded)."""
    L.awq_rope_table.argtypes = [_i64, _i32, _f64, RopeScaling, _P, _P]
    L.awq_rope.argtypes = [Rows, Rows, _i64, _i32, _P, RopeCfg, _i32, _P]
    L.awq_kv_append.argtypes = [KVCache, KVBatch, _i64, Rows, Rows, Rows, Rows, RopeCfg, _P]
    L.awq_kv_attention_workspace_bytes.argtypes = [KVCache, _i64, _i32, _i32]
    L.awq_kv_attention_workspace_bytes.restype = ctypes.c_size_t
    L.awq_kv_attention.argtypes = [KVCache, KVBatch, _i64, Rows, Rows, ctypes.c_float, _i32, _i64, _P, _P,
                                   ctypes.c_size_t, _P]
    for fn in ("awq_rope_table", "awq_rope", "awq_kv_append", "awq_kv_attention"):
        getattr(L, fn).restype = ctypes.c_int


_loaded = None


def _lib():
    global _loaded
    if _loaded is None:
        from . import lib
        _loaded = lib()
    return _loaded


def _check(code, where):
    if code != 0:
        from . import AWQError
        raise AWQError(code, where)


@contextlib.contextmanager
def _enter(device, stream):
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


_HERE = contextlib.nullcontext()


def _on(device: int, stream):
    """Context for a call on `device`: the tensors' device current, and memory
    that the call allocates taken on the stream that uses it.  A stream of another
    device is refused: its kernels would run there, on this device's memory."""
    if stream is None:
        return _HERE if device == torch.cuda.current_device() else _enter(device, None)
    if stream.device.index != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on cuda:{device}")
    return _enter(device, stream)


def _raw_stream(stream, device: int) -> int:
    # the bare handle: current_stream() builds an object, which costs more than a small kernel
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


def _where(t, device: int, name: str):
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")


def _rows(t: torch.Tensor, name: str, device: int) -> Rows:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.get_device() != device:
        _where(t, device, name)
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    T, H, D = t.shape
    tok, head, one = t.stride()
    if one != 1:
        raise ValueError(f"{name} must have contiguous elements")
    if H * D > _MAX:
        raise ValueError(f"{name}: {H} heads of {D} elements are counted in 32 bits")
    return Rows(t.data_ptr(), tok if T > 1 else H * D, head if H > 1 else D, H, code)


def _new_rows(like: torch.Tensor, dtype: torch.dtype):
    """Contiguous rows of like's shape, and their description (nothing of them needs a check but the type)."""
    t = torch.empty_like(like, dtype=dtype, memory_format=torch.contiguous_format)
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"the result must be float32, float16 or bfloat16, got {dtype}")
    _, H, D = t.shape
    return t, Rows(t.data_ptr(), H * D, D, H, code)


def _cuda(t, name: str) -> int:
    """The device of a CUDA tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _ints(t: torch.Tensor, name: str, device: int, n: int) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32:
        raise TypeError(f"{name} must be an int32 CUDA tensor")
    if t.get_device() != device:
        _where(t, device, name)
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous of shape {(n,)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _buffer(t, name: str, device: int):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8:
        raise TypeError(f"{name} must be a uint8 CUDA tensor")
    if t.get_device() != device:
        _where(t, device, name)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _cache(c: dict, device: int, D: int) -> KVCache:
    k, v, ks, vs = c["k_codes"], c["v_codes"], c["k_scales"], c["v_scales"]
    if k.dim() != 4 or v.shape != k.shape:
        raise ValueError("k_codes and v_codes must be [pages, heads, page, head_dim] alike")
    n, H, P, dim = k.shape
    if dim != D:
        raise ValueError(f"head_dim {D}, the cache's is {dim}")
    if k.dtype not in _CODES or v.dtype not in _CODES:
        raise TypeError(f"k_codes and v_codes must be float8_e4m3fn, got {k.dtype} and {v.dtype}")
    if ks.dtype != torch.float32 or vs.dtype != torch.float32:
        raise TypeError(f"k_scales and v_scales must be float32, got {ks.dtype} and {vs.dtype}")
    if ks.shape != (n, H, P // 16) or vs.shape != ks.shape:
        raise ValueError(f"k_scales and v_scales must be {(n, H, P // 16)}, got {tuple(ks.shape)} and {tuple(vs.shape)}")
    if not k.get_device() == v.get_device() == ks.get_device() == vs.get_device() == device:
        for t in (k, v, ks, vs):
            if t.get_device() != device:
                _where(t, device, "the cache")
    if not (k.is_contiguous() and v.is_contiguous() and ks.is_contiguous() and vs.is_contiguous()):
        raise ValueError("the cache's tensors must be contiguous")
    return KVCache(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), n, P, H, D)


def _batch(seq_lens, pages, cu_tokens, T, device: int) -> KVBatch:
    if not isinstance(pages, torch.Tensor) or pages.dim() != 2 or pages.dtype != torch.int32:
        raise TypeError("pages must be an int32 CUDA tensor [sequences, pages]")
    if pages.get_device() != device:
        _where(pages, device, "pages")
    n, width = pages.shape
    row, one = pages.stride()
    if n == 1:
        row = width
    if width < 1 or (width > 1 and one != 1) or row < width:
        raise ValueError("pages must have at least one column and contiguous rows that do not overlap")
    lens = _ints(seq_lens, "seq_lens", device, n)
    cu = None
    if cu_tokens is not None:
        cu = _ints(cu_tokens, "cu_tokens", device, n + 1)
    elif T != n:
        raise ValueError(f"without cu_tokens every sequence has one new token: {T} rows, {n} sequences")
    return KVBatch(lens, cu, pages.data_ptr(), n, row, width)


def _rope_cfg(table, layout, device: int) -> RopeCfg:
    code = _LAYOUTS.get(layout)
    if code is None:
        raise ValueError(f"layout must be 'half' or 'interleaved', got {layout!r}")
    if not isinstance(table, torch.Tensor) or table.dtype != torch.float32 or not table.is_cuda:
        raise TypeError("table must be a float32 CUDA tensor")
    if table.dim() != 3 or table.shape[2] != 2 or not table.is_contiguous():
        raise ValueError("table must be contiguous [positions, rot_dim / 2, 2], as rope_table returns it")
    if table.get_device() != device:
        _where(table, device, "table")
    n, half, _ = table.shape
    if half > 32768:
        raise ValueError(f"table: rot_dim must be at most 65536, got {2 * half}")
    return RopeCfg(table.data_ptr(), n, 2 * half, code)


def rope_table(n_pos: int, rot_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
               original: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0, magnitude: float = 0.0,
               device="cuda", stream=None) -> torch.Tensor:
    """float32 [n_pos, rot_dim / 2, 2]: cosine and sine of pos * base^(-2 i / rot_dim), formed in binary64.

    scaling stretches it for contexts longer than trained: "linear" (f / factor), "ntk" (a larger base) or "yarn"
    (fast pairs kept, slow ones interpolated; `original` is the trained context, magnitude 0 means
    0.1 ln(factor) + 1)."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be None, 'linear', 'ntk' or 'yarn', got {scaling!r}")
    if rot_dim > 65536:
        raise ValueError(f"rot_dim must be at most 65536, got {rot_dim}")
    device = torch.device(device)
    if device.type != "cuda":
        raise TypeError("the table lives on a CUDA device")
    index = torch.cuda.current_device() if device.index is None else device.index
    sc = RopeScaling(_SCALINGS[scaling], factor, original, beta_fast, beta_slow, magnitude)
    with _on(index, stream):
        t = torch.empty((n_pos, rot_dim // 2, 2), dtype=torch.float32, device=torch.device("cuda", index))
        _check(_lib().awq_rope_table(n_pos, rot_dim, base, sc, t.data_ptr(), _raw_stream(stream, index)),
               "awq_rope_table")
    return t


def rope(x: torch.Tensor, positions: torch.Tensor, table: torch.Tensor, layout: str = "half", inverse: bool = False,
         dtype: torch.dtype | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rotary positions of x [T, heads, head_dim]: pair i of the first rot_dim elements turns by its row's angle
    (positions int32 [T]); the rest is copied.  The result has x's type, or `dtype`, or goes to `out` (x itself:
    in place).  inverse=True applies the transpose, which is the gradient: dx = rope(dy, ..., inverse=True)."""
    device = _cuda(x, "x")
    xr = _rows(x, "x", device)
    T, H, D = x.shape
    pos = _ints(positions, "positions", device, T)
    cfg = _rope_cfg(table, layout, device)
    with _on(device, stream):
        if out is None:
            out, yr = _new_rows(x, dtype or x.dtype)
        elif out.shape != x.shape or (dtype is not None and out.dtype != dtype):
            raise ValueError("out must have x's shape and the asked type")
        else:
            yr = _rows(out, "out", device)
        if T == 0:
            return out
        _check(_lib().awq_rope(xr, yr, T, D, pos, cfg, 1 if inverse else 0,
                               _raw_stream(stream, device)), "awq_rope")
    return out


def kv_cache(n_pages: int, heads: int, page_size: int = 64, head_dim: int = 128, device="cuda") -> dict:
    """An empty paged cache: e4m3 codes [n_pages, heads, page_size, head_dim] and one float32 scale per block of
    16 tokens and head, for keys and values.  Nothing in it is read before it was appended."""
    codes, scales = (n_pages, heads, page_size, head_dim), (n_pages, heads, page_size // 16)
    return dict(k_codes=torch.empty(codes, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn),
                v_codes=torch.empty(codes, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn),
                k_scales=torch.empty(scales, dtype=torch.float32, device=device),
                v_scales=torch.empty(scales, dtype=torch.float32, device=device))


def kv_append(cache: dict, k: torch.Tensor, v: torch.Tensor, seq_lens: torch.Tensor, pages: torch.Tensor,
              cu_tokens: torch.Tensor | None = None, table: torch.Tensor | None = None, layout: str = "half",
              q: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
              q_dtype: torch.dtype = torch.float16, stream=None):
    """Append k and v [T, heads, head_dim] to the cache, k rotated to its positions by `table` on the way.

    seq_lens int32 [n]: tokens of each sequence, the new ones included; pages int32 [n, max_pages]; cu_tokens
    int32 [n + 1]: the new tokens' rows of each sequence (None: row b is sequence b's one new token).  With q
    (k's type) its rotated rows are returned, in q_dtype or in q_out; otherwise None."""
    device = _cuda(k, "k")
    kr, vr = _rows(k, "k", device), _rows(v, "v", device)
    T, H, D = k.shape
    if v.shape != k.shape:
        raise ValueError("k and v must have one shape")
    C = _cache(cache, device, D)
    B = _batch(seq_lens, pages, cu_tokens, T, device)
    cfg = RopeCfg() if table is None else _rope_cfg(table, layout, device)
    if q is not None and table is None:
        raise ValueError("q is rotated by `table`: without one there is nothing to do for it")
    with _on(device, stream):
        qr, qo = Rows(), Rows()
        if q is not None:
            qr = _rows(q, "q", device)
            if q.shape[0] != T or q.shape[2] != D:
                raise ValueError("q must have k's tokens and head_dim")
            if q_out is None:
                q_out, qo = _new_rows(q, q_dtype)
            elif q_out.shape != q.shape:
                raise ValueError("q_out must have q's shape")
            else:
                qo = _rows(q_out, "q_out", device)
        if T:
            _check(_lib().awq_kv_append(C, B, T, kr, vr, qr, qo, cfg, _raw_stream(stream, device)), "awq_kv_append")
    return q_out if q is not None else None


@functools.lru_cache(maxsize=256)
def _workspace_bytes(heads: int, head_dim: int, q_heads: int, max_tokens: int) -> int:
    return int(_lib().awq_kv_attention_workspace_bytes(KVCache(None, None, None, None, 1, 16, heads, head_dim), 1, q_heads,
                                                       max_tokens))


def kv_attention_workspace_bytes(cache: dict, T: int, q_heads: int, max_tokens: int = 1) -> int:
    """Bytes of `workspace` that kv_attention needs for these sizes."""
    _, H, _, D = cache["k_codes"].shape
    if max_tokens > _MAX:
        raise ValueError(f"max_tokens {max_tokens} does not fit 32 bits")
    return _workspace_bytes(H, D, q_heads, max_tokens)


def kv_attention(cache: dict, q: torch.Tensor, seq_lens: torch.Tensor, pages: torch.Tensor,
                 cu_tokens: torch.Tensor | None = None, max_tokens: int = 1, scale: float | None = None,
                 window: int = 0, return_lse: bool = False, out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None):
    """Causal attention of the new tokens' queries q [T, q_heads, head_dim] (fp16 or bf16) over the cache, their
    own keys appended before.  seq_lens, pages and cu_tokens as in kv_append; max_tokens bounds the new tokens of
    any sequence (one with more is reported by get_status and not computed) and chooses the kernel for the whole batch:
    single tokens beside long prompts are faster in a call of their own.  scale defaults to head_dim^-0.5; window > 0
    hides keys that far back.  Rows that see no key give 0.  workspace: uint8, kv_attention_workspace_bytes, for
    callers that keep one; calls that share it must be ordered.  Returns out [T, q_heads, head_dim], with return_lse
    also the float32 log-sum-exp [T, q_heads]."""
    device = _cuda(q, "q")
    qr = _rows(q, "q", device)
    T, H, D = q.shape
    C = _cache(cache, device, D)
    B = _batch(seq_lens, pages, cu_tokens, T, device)
    if max_tokens > _MAX:
        raise ValueError(f"max_tokens {max_tokens} does not fit 32 bits")
    L = _lib()
    with _on(device, stream):
        if out is None:
            out, outr = _new_rows(q, q.dtype)
        elif out.shape != q.shape:
            raise ValueError("out must have q's shape")
        else:
            outr = _rows(out, "out", device)
        lse = q.new_empty((T, H), dtype=torch.float32) if return_lse else None
        if T:
            ws = workspace
            if ws is None:
                ws = q.new_empty(_workspace_bytes(C.heads, D, H, max_tokens), dtype=torch.uint8)
            else:
                _buffer(ws, "workspace", device)
            _check(L.awq_kv_attention(C, B, T, qr, outr,
                                      1.0 / math.sqrt(D) if scale is None else scale, max_tokens, window,
                                      lse.data_ptr() if return_lse else None, ws.data_ptr(), ws.numel(),
                                      _raw_stream(stream, device)), "awq_kv_attention")
    return (out, lse) if return_lse else out


def _packed(layer: dict, name: str, K: int, bits: int | None, group: int | None):
    """Bits and group size of a packed layer of K inputs: its own, where it says them, else those given.  Its tensors
    must have the shapes that these ask for: the kernel reads so many words a row."""
    cfg = []
    for key, given, usual in (("bits", bits, 4), ("group_size", group, 128)):
        own = layer.get(key)
        if own is not None and given is not None and own != given:
            raise ValueError(f"{name} was packed with {key} {own}, asked for {given}")
        cfg.append(own if own is not None else usual if given is None else given)
    _check_config(*cfg, True)
    b, g = cfg
    N, per = layer["codes"].shape[0], 16 if b == 2 else 8
    if K % g:
        raise ValueError(f"{name}: {K} inputs are not groups of {g}")
    for key, shape in (("codes", (N, K // per)), ("scales", (N, K // g)), ("zeros", (N, K // g)), ("s_best", (K,))):
        if layer[key].shape != shape:
            raise ValueError(f"{name}: {key} of {b} bits in groups of {g} over {K} inputs must be {shape}, "
                             f"got {tuple(layer[key].shape)}")
    return b, g


def attention_step(x: torch.Tensor, qkv: dict, o: dict, cache: dict, seq_lens: torch.Tensor, pages: torch.Tensor,
                   table: torch.Tensor | None, q_heads: int, cu_tokens: torch.Tensor | None = None,
                   max_tokens: int = 1, layout: str = "half", window: int = 0, bits: int | None = None,
                   group: int | None = None, stream=None) -> torch.Tensor:
    """One attention block of a quantized model on its new tokens x [T, hidden] (fp16): the packed query/key/value
    projection, the append with the rotation, the attention over the cache, and the packed output projection.

    qkv and o are packed layers (quantize_layer's or load_quantized's dicts); qkv stacks the rows of the q_heads
    query heads, then of the cache's key heads, then of its value heads.  A layer's own "bits" and "group_size"
    (load_quantized's dicts have them) are what it is read with; `bits` and `group` stand for those of a layer
    that does not say (4 and 128 if not given), and must agree with one that does.  Returns float32 [T, rows of o]; rows past the
    last sequence (padding behind cu_tokens[n]) are not defined and touch no others."""
    from . import qlinear
    heads, D = cache["k_codes"].shape[1], cache["k_codes"].shape[3]
    if qkv["codes"].shape[0] != (q_heads + 2 * heads) * D:
        raise ValueError(f"qkv has {qkv['codes'].shape[0]} rows, {q_heads} + 2 x {heads} heads of {D} need "
                         f"{(q_heads + 2 * heads) * D}")
    # what the attention would refuse, before the tokens are appended
    if q_heads < 1 or q_heads % heads:
        raise ValueError(f"{q_heads} query heads are not a multiple of the cache's {heads}")
    if window < 0 or not 1 <= max_tokens <= _MAX or (cu_tokens is None and max_tokens != 1):
        raise ValueError(f"window must be at least 0 and max_tokens 1 or more (1 without cu_tokens), got {window} and {max_tokens}")
    if x.dim() != 2:
        raise ValueError("x must be [tokens, hidden]")
    T, hidden = x.shape
    of_qkv = _packed(qkv, "qkv", hidden, bits, group)
    of_o = _packed(o, "o", q_heads * D, bits, group)
    device = _cuda(x, "x")
    for layer, name in ((qkv, "qkv"), (o, "o")):
        for key in ("codes", "scales", "zeros", "s_best"):
            if layer[key].get_device() != device:
                _where(layer[key], device, f"{name}'s {key}")
    with _on(device, stream):
        y = qlinear(qkv["codes"], qkv["scales"], qkv["zeros"], qkv["s_best"], x, *of_qkv, stream=stream)
        y = y.view(T, q_heads + 2 * heads, D)
        q, k, v = y[:, :q_heads], y[:, q_heads:q_heads + heads], y[:, q_heads + heads:]
        if table is None:
            kv_append(cache, k, v, seq_lens, pages, cu_tokens, stream=stream)
            qr = q.to(torch.float16)
        else:
            qr = kv_append(cache, k, v, seq_lens, pages, cu_tokens, table, layout, q=q, stream=stream)
        a = kv_attention(cache, qr, seq_lens, pages, cu_tokens, max_tokens, window=window, stream=stream)
        return qlinear(o["codes"], o["scales"], o["zeros"], o["s_best"], a.view(T, q_heads * D), *of_o,
                       stream=stream)
