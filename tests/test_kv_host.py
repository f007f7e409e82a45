"""The cache operators without a GPU: pins of their oracle, argument checks of
the C entry points and of the binding, workspace sizes."""
import ctypes
import math

import numpy as np
import pytest
import torch

import awq_activation_aware_b200 as awq
from awq_activation_aware_b200.kv import KVBatch, KVCache, RopeCfg, RopeScaling, Rows
from oracle import kv as okv

P = 0x10000              # aligned, never dereferenced: validation fails first


# ----- pins of the oracle ----------------------------------------------------
def test_e4m3_values_are_torchs():
    codes = np.arange(256, dtype=np.uint8)
    theirs = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(okv.e4m3_decode(codes), theirs)


def test_e4m3_rounding_is_torchs():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal(20000) * 10.0 ** rng.uniform(-4, 3, 20000)).astype(np.float32)
    mids = ((okv.E4M3[:126] + okv.E4M3[1:127]) / 2).astype(np.float32)      # every tie
    x = np.clip(np.concatenate([x, mids, -mids, [0.0, -0.0, 448.0, -448.0]]), -448, 448).astype(np.float32)
    theirs = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(okv.e4m3_encode(x), theirs)
    assert okv.e4m3_encode([1e9, -1e9, np.nan]).tolist() == [126, 254, 127]


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.0001, 1), (447.9, 0), (224.0, -1), (1.75, -8), (0.0, -40),
                                    (1e38, 40), (1.0, -8), (2.0 ** -60, -40)])
def test_exponent(amax, e):
    assert okv.exponent(float(np.float32(amax))) == e


def test_rotation_is_a_product_of_complex_numbers():
    rng = np.random.default_rng(1)
    x, pos = rng.standard_normal((5, 2, 12)), np.array([0, 1, 7, 100, 3])
    f, _ = okv.frequencies(8)
    w = np.exp(1j * pos[:, None] * f[None])[:, None]
    cs = okv.rope_table(101, 8)[pos]
    y = okv.rotate(x, cs, "interleaved")
    z = (x[..., 0:8:2] + 1j * x[..., 1:8:2]) * w
    np.testing.assert_allclose(y[..., 0:8:2] + 1j * y[..., 1:8:2], z, atol=1e-13)
    np.testing.assert_array_equal(y[..., 8:], x[..., 8:])
    h = okv.rotate(x, cs, "half")
    np.testing.assert_allclose(h[..., :4] + 1j * h[..., 4:8], (x[..., :4] + 1j * x[..., 4:8]) * w, atol=1e-13)
    np.testing.assert_allclose(okv.rotate(y, cs, "interleaved", inverse=True), x, atol=1e-13)


def test_scalings_in_closed_form():
    f, _ = okv.frequencies(64)
    np.testing.assert_allclose(okv.frequencies(64, scaling="linear", factor=4.0)[0], f / 4)
    # ntk: the fastest pair stays, the slowest is interpolated by the factor
    n, _ = okv.frequencies(64, scaling="ntk", factor=4.0)
    assert n[0] == 1.0 and math.isclose(n[-1], f[-1] / 4, rel_tol=1e-12)
    y, m = okv.frequencies(64, scaling="yarn", factor=8.0, original=4096)
    assert y[0] == f[0] and math.isclose(y[-1], f[-1] / 8) and math.isclose(m, 0.1 * math.log(8) + 1)
    assert np.all(y <= f) and np.all(y >= f / 8)


def test_growing_a_block_token_by_token_equals_one_append():
    """Powers of two keep earlier codes: the codes differ only where the grown scale makes them subnormal."""
    rng = np.random.default_rng(2)
    k = (rng.standard_normal((16, 1, 64)) * 4.0 ** rng.integers(-1, 2, (16, 1, 1))).astype(np.float32)
    new = lambda: {w + n: np.zeros(s, t) for w in "kv" for n, s, t in (                      # noqa: E731
        ("_codes", (1, 1, 16, 64), np.uint8), ("_scales", (1, 1, 1), np.float32))}
    one, many, pages = new(), new(), np.zeros((1, 1), np.int32)
    okv.append(one, k, k, [16], pages, [0, 16])
    for i in range(16):
        okv.append(many, k[i:i + 1], k[i:i + 1], [i + 1], pages)
    assert one["k_scales"] == many["k_scales"]
    a, b = okv.e4m3_decode(one["k_codes"]), okv.e4m3_decode(many["k_codes"])
    normal = np.abs(a) >= 2.0 ** -6
    np.testing.assert_array_equal(a[normal], b[normal])
    assert np.abs(a - b).max() <= 2.0 ** -9


def test_attention_oracle_against_torch():
    rng = np.random.default_rng(3)
    H, HQ, D, S = 2, 4, 64, 50
    cache = {w + "_codes": okv.e4m3_encode(rng.standard_normal((4, H, 16, D))) for w in "kv"}
    cache |= {w + "_scales": (2.0 ** rng.integers(-2, 3, (4, H, 1))).astype(np.float32) for w in "kv"}
    pages = np.array([[2, 0, 3, 1]], np.int32)
    q = rng.standard_normal((5, HQ, D))
    out, lse, _ = okv.attention(cache, q, [S], pages, [0, 5])
    dense = [torch.from_numpy((okv.e4m3_decode(cache[w + "_codes"][pages[0]]) * cache[w + "_scales"][pages[0]][..., None])
                              .transpose(1, 0, 2, 3).reshape(H, 64, D)[:, :S].repeat(HQ // H, axis=0)) for w in "kv"]
    x = torch.einsum("thd,hsd->hts", torch.from_numpy(q), dense[0]) / 8.0
    x.masked_fill_(torch.arange(S)[None] > torch.arange(S - 5, S)[:, None], float("-inf"))
    np.testing.assert_allclose(out, torch.einsum("hts,hsd->thd", x.softmax(-1), dense[1]).numpy(), rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(lse, x.logsumexp(-1).T.numpy(), rtol=1e-12)
    out, lse, _ = okv.attention(cache, q[:1], [0], pages)
    assert not out.any() and np.all(np.isneginf(lse))


# ----- the C entry points ------------------------------------------------------
ROWS = dict(data=P, token_stride=4096, head_stride=128, heads=8, dtype=1)
CACHE = dict(k_codes=P, v_codes=P, k_scales=P, v_scales=P, n_pages=100, page_size=64, heads=8, head_dim=128)
BATCH = dict(seq_lens=P, cu_tokens=P, pages=P, n_seqs=4, page_stride=10, max_pages=10)
CFG = dict(table=P, n_pos=1000, rot_dim=128, layout=0)


def _st(cls, base, kw):
    return cls(**{**base, **kw})


BAD_CACHE = [dict(k_codes=None), dict(v_codes=None), dict(k_scales=None), dict(v_scales=None), dict(k_codes=P + 8),
             dict(v_scales=P + 4), dict(n_pages=0), dict(page_size=48), dict(page_size=8), dict(page_size=512),
             dict(heads=0), dict(head_dim=80), dict(head_dim=256), dict(n_pages=1 << 23)]
BAD_BATCH = [dict(seq_lens=None), dict(pages=None), dict(n_seqs=0), dict(max_pages=0), dict(page_stride=9),
             dict(cu_tokens=None, n_seqs=5)]


def test_rope_rejects_bad_arguments():
    L = awq.lib()

    def call(x={}, y={}, r={}, **kw):
        a = dict(T=16, head_dim=128, positions=P, inverse=0)
        a.update(kw)
        return L.awq_rope(_st(Rows, ROWS, x), _st(Rows, ROWS, dict(data=2 * P) | y), a["T"], a["head_dim"], a["positions"],
                          _st(RopeCfg, CFG, r), a["inverse"], None)

    for kw in (dict(T=0), dict(T=1 << 31), dict(head_dim=127), dict(head_dim=0), dict(positions=None), dict(inverse=2),
               dict(x=dict(data=None)), dict(x=dict(data=P + 1)), dict(x=dict(dtype=3)), dict(x=dict(heads=0)),
               dict(x=dict(head_stride=-1)), dict(y=dict(data=None)), dict(y=dict(data=P + 3)), dict(y=dict(heads=4)),
               dict(y=dict(head_stride=64)), dict(y=dict(token_stride=128)), dict(y=dict(token_stride=0)),
               dict(y=dict(data=P, dtype=0)), dict(y=dict(data=P, head_stride=256)),
               dict(r=dict(table=None)), dict(r=dict(table=P + 8)), dict(r=dict(rot_dim=130)), dict(r=dict(rot_dim=3)),
               dict(r=dict(rot_dim=0)), dict(r=dict(n_pos=0)), dict(r=dict(layout=2))):
        assert call(**kw) == 1, kw


def test_rope_table_rejects_bad_arguments():
    L = awq.lib()

    def call(n=10, rot=64, base=1e4, table=P, **kw):
        s = dict(kind=0, factor=1.0, original=0.0, beta_fast=32.0, beta_slow=1.0, magnitude=0.0)
        return L.awq_rope_table(n, rot, base, RopeScaling(**{**s, **kw}), table, None)

    yarn = dict(kind=3, factor=2.0, original=100.0)
    for kw in (dict(n=0), dict(rot=0), dict(rot=7), dict(base=1.0), dict(base=math.nan), dict(base=math.inf),
               dict(table=None), dict(table=P + 4), dict(kind=4), dict(kind=-1), dict(kind=1, factor=0.5),
               dict(kind=1, factor=math.nan), dict(kind=2, rot=2, factor=2.0), {**yarn, "original": 0.0},
               {**yarn, "beta_slow": 0.0}, {**yarn, "beta_slow": 64.0}, {**yarn, "magnitude": -1.0},
               {**yarn, "beta_fast": math.nan}):
        assert call(**kw) == 1, kw


def test_append_rejects_bad_arguments():
    L = awq.lib()

    def call(c={}, b={}, k={}, v={}, q=dict(data=None), qo={}, r={}, T=4):
        return L.awq_kv_append(_st(KVCache, CACHE, c), _st(KVBatch, BATCH, b), T, _st(Rows, ROWS, k), _st(Rows, ROWS, v),
                               _st(Rows, ROWS, q), _st(Rows, ROWS, dict(data=2 * P) | qo), _st(RopeCfg, CFG, r), None)

    bad = [dict(c=x) for x in BAD_CACHE] + [dict(b=x) for x in BAD_BATCH]
    bad += [dict(T=0), dict(k=dict(data=None)), dict(k=dict(data=P + 8)), dict(k=dict(heads=4)), dict(v=dict(heads=16)),
            dict(v=dict(dtype=2)), dict(k=dict(token_stride=4100)), dict(v=dict(head_stride=4)), dict(r=dict(rot_dim=130)),
            dict(r=dict(rot_dim=5)), dict(r=dict(layout=-1)), dict(r=dict(table=P + 8)), dict(q={}, r=dict(table=None)),
            dict(q=dict(dtype=0)), dict(q={}, qo=dict(data=None)), dict(q={}, qo=dict(head_stride=64)),
            dict(q={}, qo=dict(heads=4)), dict(q={}, qo=dict(data=P, dtype=2)), dict(q=dict(data=P + 2))]
    for kw in bad:
        assert call(**kw) == 1, kw


def test_attention_rejects_bad_arguments():
    L = awq.lib()

    def call(c={}, b={}, q={}, o={}, T=4, scale=0.1, max_tokens=4, window=0, lse=None, ws=P, n=1 << 40):
        return L.awq_kv_attention(_st(KVCache, CACHE, c), _st(KVBatch, BATCH, b), T, _st(Rows, ROWS, dict(heads=32) | q),
                                  _st(Rows, ROWS, dict(heads=32, data=2 * P) | o), scale, max_tokens, window, lse, ws, n,
                                  None)

    bad = [dict(c=x) for x in BAD_CACHE] + [dict(b=x) for x in BAD_BATCH]
    bad += [dict(T=0), dict(q=dict(dtype=0), o=dict(dtype=0)), dict(o=dict(dtype=2)), dict(q=dict(heads=33), o=dict(heads=33)),
            dict(q=dict(heads=16)), dict(q=dict(data=P + 8)), dict(o=dict(data=P)), dict(o=dict(token_stride=128)),
            dict(q=dict(token_stride=4098)), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf),
            dict(max_tokens=0), dict(max_tokens=2, b=dict(cu_tokens=None)), dict(window=-1)]
    for kw in bad:
        assert call(**kw) == 1, kw
    for kw in (dict(ws=None), dict(ws=P + 16), dict(n=0)):
        assert call(**kw) == 5, kw


def test_binding_refuses_host_tensors_and_unknown_names():
    x = torch.zeros((2, 2, 64))
    with pytest.raises(TypeError):
        awq.rope(x, torch.zeros(2, dtype=torch.int32), torch.zeros((4, 32, 2)))
    with pytest.raises(ValueError):
        awq.rope_table(4, 64, scaling="cubic")
    with pytest.raises(TypeError):
        awq.rope_table(4, 64, device="cpu")
    with pytest.raises(TypeError):
        awq.kv_append(awq.kv_cache(1, 2, 16, 64, device="cpu"), x, x, None, None)
    with pytest.raises(TypeError):
        awq.kv_attention(awq.kv_cache(1, 2, 16, 64, device="cpu"), x, None, None)


def test_workspace_size_query_runs_without_a_gpu():
    n = awq.lib().awq_kv_attention_workspace_bytes(KVCache(**CACHE), 4, 32, 1)
    assert n > 0 and n % 256 == 0


# ----- the configuration of the packed layers of a step ------------------------
def _packed_layer(N, K, bits, group):
    return dict(codes=torch.zeros((N, K // (16 if bits == 2 else 8)), dtype=torch.int32),
                scales=torch.zeros((N, K // group), dtype=torch.float16),
                zeros=torch.zeros((N, K // group), dtype=torch.float16), s_best=torch.ones(K))


class _Reached(Exception):
    pass


def _step_reads(monkeypatch, qkv, o, K=256, **kw):
    """(bits, group) that a step of 4 + 2 + 2 heads of 64 hands to each of its projections."""
    calls = []

    def qlinear(codes, scales, zeros, s_best, X, bits=4, group=128, **_):
        calls.append((bits, group))
        if len(calls) == 2:
            raise _Reached
        return torch.zeros((X.shape[0], codes.shape[0]))

    monkeypatch.setattr(awq, "qlinear", qlinear)
    monkeypatch.setattr(awq.kv, "_cuda", lambda t, name: -1)                # host tensors: device -1
    monkeypatch.setattr(awq.kv, "_on", lambda *a: awq.kv._HERE)
    monkeypatch.setattr(awq.kv, "kv_append", lambda *a, q=None, **k: q)
    monkeypatch.setattr(awq.kv, "kv_attention", lambda cache, q, *a, **k: q.contiguous())
    with pytest.raises(_Reached):
        awq.attention_step(torch.zeros((3, K), dtype=torch.float16), qkv, o, awq.kv_cache(2, 2, 16, 64, device="cpu"),
                           None, None, torch.zeros(1), 4, **kw)
    return calls


@pytest.mark.parametrize("a", [(2, 64), (3, 128), (4, 64), (4, 128)])
@pytest.mark.parametrize("b", [(2, 128), (4, 128), (4, 64)])
def test_a_step_reads_each_layer_as_it_was_packed(monkeypatch, a, b):
    said = [dict(zip(("bits", "group_size"), x)) for x in (a, b)]
    qkv, o = _packed_layer(512, 256, *a) | said[0], _packed_layer(320, 256, *b) | said[1]
    assert _step_reads(monkeypatch, qkv, o) == [a, b]
    # layers that do not say: what the call gives, 4 and 128 without
    assert _step_reads(monkeypatch, _packed_layer(512, 256, *a), _packed_layer(320, 256, *a), bits=a[0], group=a[1]) == [a] * 2
    plain = _packed_layer(512, 256, 4, 128), _packed_layer(320, 256, 4, 128)
    assert _step_reads(monkeypatch, *plain) == [(4, 128)] * 2
    assert _step_reads(monkeypatch, plain[0], o) == [(4, 128), b]


def test_a_step_refuses_layers_that_it_would_misread():
    """Refused by shapes and configuration alone, before anything is launched (these are host tensors)."""
    x, cache = torch.zeros((3, 256), dtype=torch.float16), awq.kv_cache(2, 2, 16, 64, device="cpu")

    def call(qkv={}, o={}, **kw):
        qkv = _packed_layer(512, 256, 4, 128) | qkv
        awq.attention_step(x, qkv, _packed_layer(320, 256, 4, 128) | o, cache, None, None, None, 4, **kw)

    two = _packed_layer(512, 256, 2, 64)
    bad = [dict(qkv=two), dict(o={k: v[:320] if v.dim() == 2 else v for k, v in two.items()}),      # 2 bits read as 4
           dict(qkv=dict(bits=2)), dict(o=dict(bits=2)), dict(qkv=dict(group_size=64)), dict(o=dict(group_size=64)),
           dict(qkv=dict(bits=4), bits=2), dict(o=dict(bits=4), bits=3), dict(o=dict(group_size=128), group=64),
           dict(bits=2), dict(group=64), dict(bits=5), dict(group=32), dict(group=0), dict(qkv=dict(bits=8)),
           dict(qkv=dict(s_best=torch.ones(128))), dict(o=dict(zeros=torch.zeros((320, 1), dtype=torch.float16))),
           dict(o=dict(codes=torch.zeros((320, 16), dtype=torch.int32))),
           dict(qkv=dict(scales=torch.zeros((511, 2), dtype=torch.float16)))]
    for kw in bad:
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(ValueError):
        awq.attention_step(x[0], _packed_layer(512, 256, 4, 128), _packed_layer(320, 256, 4, 128), cache, None, None, None, 4)
    with pytest.raises(TypeError):                                         # the right shapes, on the host
        call()


# ----- sizes past 32 bits -------------------------------------------------------
def test_rope_refuses_tokens_past_32_bits():
    """Elements of a token are counted in 32 bits."""
    L = awq.lib()

    def call(heads, dim, rot=64):
        x = dict(heads=heads, head_stride=dim, token_stride=heads * dim)
        return L.awq_rope(Rows(**{**ROWS, **x}), Rows(**{**ROWS, **x, "data": 2 * P}), 16, dim, P,
                          RopeCfg(**{**CFG, "rot_dim": rot}), 0, None)

    for heads, dim in ((65536, 65536), (32768, 65536), (1 << 30, 2), ((1 << 31) - 1, 128)):
        assert call(heads, dim, 2) == 1, (heads, dim)


def test_binding_refuses_sizes_that_a_32_bit_field_would_wrap():
    """On host tensors (device -1) of any size in no memory."""
    one = torch.zeros((1, 1, 2), dtype=torch.float16)
    assert awq.kv._rows(one, "x", -1).heads == 1
    for shape in ((1, (1 << 32) + 1, 2), (1, 1 << 31, 2), (1, 1 << 30, 2), (5, 1 << 16, 1 << 15)):
        x = torch.zeros(shape[2], dtype=torch.float16).expand(shape)
        with pytest.raises(ValueError, match="32 bits"):
            awq.kv._rows(x, "x", -1)
    with pytest.raises(ValueError, match="rot_dim"):
        awq.rope_table(1, (1 << 32) + 64)
    with pytest.raises(ValueError, match="32 bits"):
        awq.kv_attention_workspace_bytes(awq.kv_cache(1, 2, 16, 64, device="cpu"), 4, 2, (1 << 32) + 1)


# ----- streams and devices -------------------------------------------------------
class _Stream:
    """What the binding asks of a stream, without a device."""
    def __init__(self, index):
        self.device, self.cuda_stream = torch.device("cuda", index), 0


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """A launch there would read and write this device's memory from the other one."""
    monkeypatch.setattr(awq.kv, "_enter", lambda device, stream: ("entered", device))
    assert awq.kv._on(0, _Stream(0)) == ("entered", 0) and awq.kv._on(3, _Stream(3)) == ("entered", 3)
    for device, other in ((0, 1), (1, 0)):
        with pytest.raises(ValueError, match="stream"):
            awq.kv._on(device, _Stream(other))


def test_status_is_read_on_the_streams_device(monkeypatch):
    """Every device has its own error words: the ones of the stream's device are asked for."""
    import contextlib
    current, asked = [0], []

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], torch.device(d).index
        yield
        current[0] = before

    class Lib:
        @staticmethod
        def awq_get_status(stream):
            asked.append(current[0])
            return 1 if current[0] == 1 else 0

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(awq, "lib", lambda: Lib)
    awq.get_status(_Stream(0))
    with pytest.raises(awq.AWQError):
        awq.get_status(_Stream(1))
    assert asked == [0, 1]


def test_a_step_is_refused_before_it_appends(monkeypatch):
    """What the attention would refuse, the step refuses first: the cache keeps its state."""
    done = []
    monkeypatch.setattr(awq, "qlinear", lambda codes, *a, **k: done.append("qlinear") or torch.zeros((3, codes.shape[0])))
    monkeypatch.setattr(awq.kv, "_cuda", lambda t, name: -1)
    monkeypatch.setattr(awq.kv, "_on", lambda *a: awq.kv._HERE)
    monkeypatch.setattr(awq.kv, "kv_append", lambda *a, q=None, **k: done.append("append") or q)
    cache = awq.kv_cache(2, 2, 16, 64, device="cpu")
    x, table, cu = torch.zeros((3, 256), dtype=torch.float16), torch.zeros(1), torch.zeros(1)

    def call(q_heads, **kw):
        awq.attention_step(x, _packed_layer((q_heads + 4) * 64, 256, 4, 128), _packed_layer(320, q_heads * 64, 4, 64) |
                           dict(bits=4, group_size=64), cache, None, None, table, q_heads, **kw)

    for bad in (dict(q_heads=3), dict(q_heads=0), dict(q_heads=4, window=-1), dict(q_heads=4, max_tokens=0, cu_tokens=cu),
                dict(q_heads=4, max_tokens=2), dict(q_heads=4, max_tokens=1 << 31, cu_tokens=cu)):
        with pytest.raises(ValueError):
            call(**bad)
    assert not done
