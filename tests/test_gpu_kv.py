"""The cache operators on the GPU against their oracle.

Acceptance:
  * rotation: bit-exact (every binary32 operation is pinned, one rounding to the
    result's type); the table: half a unit of binary32 beside the binary64 value;
  * append: codes and scales bit-exact, every other byte of the cache untouched;
  * attention: the tolerance of `bound` below, derived from the roundings.
"""
import numpy as np
import pytest
import torch

from oracle import kv as okv

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def awq():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import awq_activation_aware_b200 as m
    m.set_wait_timeout_ms(2000)
    return m


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().double().cpu().numpy()


# ----- rotary positions ---------------------------------------------------------
@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=3.0), dict(scaling="ntk", factor=4.0),
                                dict(scaling="yarn", factor=8.0, original=4096.0),
                                dict(base=5e5, scaling="yarn", factor=16.0, original=8192.0, beta_fast=16.0,
                                     beta_slow=2.0, magnitude=1.25)])
@pytest.mark.parametrize("n,rot", [(1, 2), (131072, 64), (1000, 128), (777, 20)])
def test_rope_table(awq, n, rot, kw):
    if kw.get("scaling") == "ntk" and rot == 2:
        pytest.skip("ntk has no exponent for one pair")
    t = f64(awq.rope_table(n, rot, **kw))
    awq.get_status()
    ref = okv.rope_table(n, rot, **kw)
    # one rounding to binary32 (2^-24 of the value), and binary64 angles up to n off by a few 2^-53 of themselves
    assert np.all(np.abs(t - ref) <= 2.0 ** -24 * np.abs(ref) + 16 * (n + 1) * 2.0 ** -53)


def _rounded(y32, dtype):
    return torch.from_numpy(y32).to(dtype)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 2, 2), (5, 3, 128, 128), (33, 8, 128, 64), (7, 2, 80, 20), (64, 5, 64, 64),
                                       (3, 2, 6, 4), (9, 40, 256, 32), (200, 1, 128, 128)])
def test_rope(awq, T, H, D, rot, layout):
    rng = np.random.default_rng(T * 1000 + D)
    table = awq.rope_table(300, rot, scaling="yarn", factor=4.0, original=64.0)
    cs = table.cpu().numpy()
    pos = rng.integers(0, 300, T)
    x = rng.standard_normal((T, H, D)).astype(np.float32)
    for src in (F32, F16, BF16):
        xd = dev(x, src)
        for dst in (F32, F16, BF16):
            for inverse in (False, True):
                y = awq.rope(xd, ints(pos), table, layout, inverse, dtype=dst)
                ref = okv.rotate(xd.float().cpu().numpy(), cs[pos], layout, inverse)
                assert torch.equal(y.cpu(), _rounded(ref, dst)), (src, dst, inverse)
        z = awq.rope(xd.clone(), ints(pos), table, layout)
        w = xd.clone()
        assert awq.rope(w, ints(pos), table, layout, out=w) is w           # in place
        assert torch.equal(z, w)
    awq.get_status()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_strided_and_unaligned_rows(awq, layout):
    table = awq.rope_table(50, 64)
    pos = ints(np.arange(11))
    base = torch.randn((11, 300, 64), device="cuda", dtype=F16)
    big = torch.randn(11 * 3 * 64 + 1, device="cuda", dtype=F16)
    views = {"slice of a projection": base[:, 10:14], "every other head": base[:, ::100],
             "heads first": torch.randn((3, 11, 64), device="cuda", dtype=F16).transpose(0, 1),
             "one element off": big[1:].view(11, 3, 64), "one row for all": base[:1, :4].expand(11, 4, 64)}
    for name, x in views.items():
        ref = okv.rotate(x.float().cpu().numpy(), table.cpu().numpy()[:11], layout)
        assert torch.equal(awq.rope(x, pos, table, layout).cpu(), _rounded(ref, F16)), name
        out = torch.full((11, x.shape[1] + 2, 65), 7.0, device="cuda", dtype=F16)
        awq.rope(x, pos, table, layout, out=out[:, 1:-1, :64])
        assert torch.equal(out[:, 1:-1, :64].cpu(), _rounded(ref, F16)), name
        assert bool((out[:, 0] == 7).all() and (out[:, -1] == 7).all() and (out[..., 64] == 7).all()), name
    with pytest.raises(awq.AWQError):                                      # written rows would overlap
        awq.rope(base[:, :4], pos, table, out=base[:1, :4].expand(11, 4, 64))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_inverse_is_the_gradient(awq, layout):
    rng = np.random.default_rng(5)
    table = awq.rope_table(40, 32, scaling="yarn", factor=4.0, original=10.0)      # magnitude above 1
    x, w = rng.standard_normal((4, 2, 48)).astype(np.float32), rng.standard_normal((4, 2, 48)).astype(np.float32)
    pos = ints([3, 39, 0, 17])
    g = f64(awq.rope(dev(w), pos, table, layout, inverse=True))
    # against the formula: the transpose of the rotation, with the table's own entries in binary64
    ref = okv.rotate(w.astype(np.float64), table.cpu().numpy().astype(np.float64)[[3, 39, 0, 17]], layout, True)
    np.testing.assert_allclose(g, ref, atol=3 * 2.0 ** -24 * np.abs(w).max() * 1.2, rtol=0)
    # against differences: the map is linear, so a step of 1 is exact but for the roundings of the two results,
    # each of three operations (3 * 2^-24) on values up to 1.14 (|x1| + |x2|) <= 12
    for i in range(0, x.size, 7):
        e = np.zeros(x.size, np.float32)
        e[i] = 1.0
        hi = f64(awq.rope(dev(x + e.reshape(x.shape)), pos, table, layout))
        lo = f64(awq.rope(dev(x - e.reshape(x.shape)), pos, table, layout))
        d = ((hi - lo) / 2 * w).sum()
        assert abs(d - g.reshape(-1)[i]) <= 2 * 2 * 4 * 2.0 ** -24 * 12 * np.abs(w).max()


def test_rope_position_outside_the_table_is_reported(awq):
    table = awq.rope_table(8, 64)
    x = torch.randn((3, 2, 64), device="cuda", dtype=F16)
    out = torch.full_like(x, 5.0)
    awq.rope(x, ints([7, 8, -1]), table, out=out)
    with pytest.raises(awq.AWQError):
        awq.get_status()
    assert bool((out[1:] == 5).all()) and not bool((out[0] == 5).all())
    awq.rope(x, ints([0, 1, 2]), table)
    awq.get_status()


# ----- append -------------------------------------------------------------------
def _random_cache(rng, n_pages, H, P, D):
    """Codes of every value that is not NaN, scales powers of two."""
    c = {}
    for w in "kv":
        codes = rng.integers(0, 256, (n_pages, H, P, D)).astype(np.uint8)
        codes[(codes & 127) == 127] = 3
        c[w + "_codes"] = codes
        c[w + "_scales"] = (2.0 ** rng.integers(-12, -6, (n_pages, H, P // 16))).astype(np.float32)
    return c


def _upload(c):
    return {k: dev(x).view(torch.float8_e4m3fn) if k.endswith("codes") else dev(x) for k, x in c.items()}


def _same(cache, ref):
    for k, x in ref.items():
        got = cache[k].view(torch.uint8).cpu().numpy() if k.endswith("codes") else cache[k].cpu().numpy()
        np.testing.assert_array_equal(got, x, err_msg=k)


def _pages(rng, lens, P, extra=0):
    """A page table of distinct pages in random order (unused entries point far outside), and the pool's size."""
    need = [-(-int(n) // P) for n in lens]
    order = rng.permutation(sum(need) + extra).astype(np.int32)
    t = np.full((len(lens), max(max(need), 1) + 1), 1 << 30, np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return t, max(len(order), 1)


APPENDS = [  # lengths after the append, new tokens of each (None: one each)
    ([1], None), ([16], None), ([17], None), ([33, 1, 0, 64, 65, 7], None), ([5, 40, 16, 100], [5, 24, 16, 1]),
    ([300, 0, 3, 129], [77, 0, 3, 129]), ([31, 48], [15, 17]), ([2], [3]),
]


@pytest.mark.parametrize("lens,new", APPENDS)
@pytest.mark.parametrize("P,H,D,layout,rot", [(16, 2, 64, "half", 64), (64, 3, 128, "interleaved", 128),
                                              (32, 1, 128, "half", 20), (256, 2, 64, "interleaved", 6),
                                              (128, 2, 128, None, 0)])
def test_append(awq, lens, new, P, H, D, layout, rot):
    rng = np.random.default_rng(len(lens) * 100 + P)
    cu = None if new is None else np.concatenate([[0], np.cumsum(new)])
    T = len(lens) if new is None else int(cu[-1]) + 3                      # three rows that belong to nobody
    pages, n_pages = _pages(rng, lens, P, 2)
    base = _random_cache(rng, n_pages, H, P, D)
    table = awq.rope_table(max(max(lens), 1), rot) if rot else None
    HQ = 5
    x = (rng.standard_normal((T, HQ + 2 * H, D)) * 4.0 ** rng.integers(-3, 3, (T, 1, 1))).astype(np.float32)
    for src in (F32, F16, BF16):
        xd = dev(x, src)
        xf = xd.float().cpu().numpy()
        cache, ref = _upload(base), {k: v.copy() for k, v in base.items()}
        q, k, v = xd[:, :HQ], xd[:, HQ:HQ + H], xd[:, HQ + H:]
        q_out = torch.full((T, HQ, D), 9.0, device="cuda", dtype=BF16)
        got = awq.kv_append(cache, k, v, ints(lens), ints(pages), None if cu is None else ints(cu), table,
                            layout or "half", q=q if rot else None, q_out=q_out if rot else None)
        awq.get_status()
        cs = table.cpu().numpy() if rot else None
        okv.append(ref, xf[:, HQ:HQ + H], xf[:, HQ + H:], lens, pages, cu, cs, layout or "half")
        _same(cache, ref)
        if not rot:
            assert got is None
            continue
        assert got is q_out
        places = okv.rows_of(lens, cu, T)
        for t, p in enumerate(places):
            if p is None or p[1] < 0:
                assert bool((q_out[t] == 9).all())
            else:
                y = okv.rotate(xf[t:t + 1, :HQ], cs[[p[1]]], layout)
                assert torch.equal(q_out[t:t + 1].cpu(), _rounded(y, BF16))


def test_append_token_by_token(awq):
    """Every growth of every block on the way, each step bit-exact."""
    rng = np.random.default_rng(8)
    H, D, P = 2, 128, 32
    pages = np.array([[2, 0, 1], [3, 5, 4]], np.int32)
    ref = _random_cache(rng, 6, H, P, D)
    cache = _upload(ref)
    table = awq.rope_table(96, D)
    for n in range(1, 70):
        k, v = ((rng.standard_normal((2, H, D)) * 2.0 ** rng.integers(-8, 9, (2, H, 1))).astype(np.float32) for _ in "kv")
        awq.kv_append(cache, dev(k), dev(v), ints([n, n + 9]), ints(pages), table=table)
        okv.append(ref, k, v, [n, n + 9], pages, None, table.cpu().numpy())
    awq.get_status()
    _same(cache, ref)


def test_append_values_at_the_edges(awq):
    """Zeros, infinities and NaN (stored as NaN, out of the scale), values past both ends of the scales, ties."""
    D, P = 64, 16
    x = np.zeros((6, 1, D), np.float32)
    x[1, 0, :8] = [np.inf, -np.inf, np.nan, 1.0, -448.0, 448.0, 0.5, -0.0]
    x[2, 0, :4] = [3e38, -1e30, 1.0, 0.0]
    x[3, 0, :4] = [1e-38, 2e-45, -1e-20, 0.0]
    x[4, 0] = np.arange(D) / 64 + 1                                       # ties of the three fraction bits
    x[5, 0] = np.nan
    ref = _random_cache(np.random.default_rng(0), 6, 1, P, D)
    cache, pages = _upload(ref), np.arange(6, dtype=np.int32)[:, None]
    awq.kv_append(cache, dev(x), dev(x), ints([1] * 6), ints(pages))
    okv.append(ref, x, x, [1] * 6, pages)
    _same(cache, ref)
    # the same in the middle of a block
    awq.kv_append(cache, dev(x[::-1].copy()), dev(x), ints([2] * 6), ints(pages))
    okv.append(ref, x[::-1], x, [2] * 6, pages)
    awq.get_status()
    _same(cache, ref)


def test_append_reports_pages_and_positions_outside(awq):
    rng = np.random.default_rng(1)
    ref = _random_cache(rng, 4, 1, 16, 64)
    cache = _upload(ref)
    x = rng.standard_normal((4, 1, 64)).astype(np.float32)
    pages = np.array([[0, 1], [4, 1], [-1, 2], [3, 2]], np.int32)
    lens = [17, 5, 3, 40]                                                  # fine, two bad pages, past the table's 32
    awq.kv_append(cache, dev(x), dev(x), ints(lens), ints(pages))
    with pytest.raises(awq.AWQError):
        awq.get_status()
    okv.append(ref, x[:1], x[:1], lens[:1], pages[:1])
    _same(cache, ref)
    awq.kv_append(cache, dev(x[:1]), dev(x[:1]), ints([18]), ints(pages[:1]), table=awq.rope_table(17, 64))
    with pytest.raises(awq.AWQError):                                      # past the rotary table
        awq.get_status()
    _same(cache, ref)


# ----- attention ----------------------------------------------------------------
def bound(out, info, dtype, D):
    """What the roundings can add up to.  Probabilities are rounded to fp16 (2^-11 of each, or 2^-22 of the largest
    where fp16 is subnormal), scores are binary32 sums of D exact products (each addition at most 2^-23 of the sum of
    the magnitudes, twice a rounding to nearest since the tensor cores may truncate) and the exponential is off by
    2^-22: all relative to the mass sum p |v|; sums over n keys add n / 8 such additions; the result is rounded once."""
    mass, reach, peak, keys = info
    delta = (D + 8) * 2.0 ** -23 * reach
    rel = 2.0 ** -11 + 2 * delta + 2.0 ** -21 + (keys / 8 + 64) * 2.0 ** -23
    eps = torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -25 if dtype == F16 else 0.0                             # half a step of subnormal fp16
    return (1 + eps) * (mass * rel[..., None] * 2 + (keys * 2.0 ** -22 * peak)[..., None]) + eps * np.abs(out) + tiny


def lse_bound(lse, info, D):
    _, reach, _, keys = info
    return (D + 8) * 2.0 ** -23 * reach + (keys / 8 + 64) * 2.0 ** -23 + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0))


def _attend_case(seed, lens, new, H, G, D, P, spoil=True):
    rng = np.random.default_rng(seed)
    cu = None if new is None else np.concatenate([[0], np.cumsum(new)])
    T = len(lens) if new is None else int(cu[-1])
    pages, n_pages = _pages(rng, lens, P, 1)
    c = {}
    for w in "kv":
        x = rng.standard_normal((n_pages, H, P // 16, 16, D))
        if w == "k":
            x *= np.exp(0.7 * rng.standard_normal(D))
        e = np.ceil(np.log2(np.abs(x).max((3, 4)) / 448))
        codes = okv.e4m3_encode(x * 2.0 ** -e[..., None, None]).reshape(n_pages, H, P, D)
        e += rng.integers(-3, 4, e.shape)                                  # blocks of very different sizes
        c[w + "_codes"], c[w + "_scales"] = codes, (2.0 ** e).astype(np.float32)
    if spoil:                                                              # NaN wherever no token is
        seen = np.zeros((n_pages, P), bool)
        for b, n in enumerate(lens):
            for j in range(n):
                seen[pages[b, j // P], j % P] = True
        for w in "kv":
            c[w + "_codes"].transpose(0, 2, 1, 3)[~seen] = 127
            blocks = ~seen.reshape(n_pages, P // 16, 16).any(-1)
            c[w + "_scales"].transpose(0, 2, 1)[blocks] = np.nan
    q = rng.standard_normal((T, H * G, D))
    return c, q, np.asarray(lens, np.int32), cu, pages


def _attend(awq, c, q, lens, cu, pages, dtype, D, window=0, scale=None, **kw):
    new = 1 if cu is None else max(int(np.diff(cu).max()), 1)
    qd = dev(q, dtype)
    out, lse = awq.kv_attention(_upload(c), qd, ints(lens), ints(pages), None if cu is None else ints(cu), new, scale,
                                window, return_lse=True, **kw)
    awq.get_status()
    ref, rl, info = okv.attention(c, f64(qd), lens, pages, cu, scale, window)
    return out, lse, ref, rl, info


def _close(out, lse, ref, rl, info, dtype, D):
    d = np.abs(f64(out) - ref)
    lim = bound(ref, info, dtype, D)
    assert np.all(d <= lim), (float((d / lim).max()), np.unravel_index((d / lim).argmax(), d.shape))
    empty = np.isneginf(rl)
    got = f64(lse)
    assert np.array_equal(np.isneginf(got), empty) and not f64(out)[empty].any()
    assert np.all(np.abs(got[~empty] - rl[~empty]) <= lse_bound(rl, info, D)[~empty])


SINGLES = [[1], [16], [17], [0, 15, 64, 65], [63, 0, 128, 129, 1], [1000], [517, 2049, 33]]
HEADS = [(1, 1), (2, 4), (1, 8), (3, 5), (2, 16), (1, 32), (8, 1)]


@pytest.mark.parametrize("lens", SINGLES)
@pytest.mark.parametrize("H,G", HEADS)
def test_attention_single_tokens(awq, lens, H, G):
    i = SINGLES.index(lens) + HEADS.index((H, G))
    P, D, dtype = [16, 64, 32, 128, 256][i % 5], [64, 128][i % 2], [F16, BF16][(i // 2) % 2]
    c, q, lens, cu, pages = _attend_case(i, lens, None, H, G, D, P)
    _close(*_attend(awq, c, q, lens, cu, pages, dtype, D), dtype, D)


@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_every_page_size(awq, P, D, dtype):
    c, q, lens, cu, pages = _attend_case(P + D, [300, 1, 77], None, 2, 4, D, P)
    _close(*_attend(awq, c, q, lens, cu, pages, dtype, D), dtype, D)


RAGGED = [  # lengths, new tokens
    ([5], [5]), ([64], [3]), ([300, 40, 0, 129], [7, 40, 0, 1]), ([1000], [130]), ([257, 600], [257, 2]),
    ([33, 500, 1, 90], [33, 129, 1, 64]), ([2, 10], [5, 4]), ([1537], [513]),
]


@pytest.mark.parametrize("lens,new", RAGGED)
@pytest.mark.parametrize("H,G", [(1, 1), (2, 4), (1, 8), (2, 5), (1, 7)])
def test_attention_several_tokens(awq, lens, new, H, G):
    i = RAGGED.index((lens, new)) * 3 + H + G
    P, D, dtype = [16, 64, 32, 128, 256][i % 5], [128, 64][i % 2], [BF16, F16][(i // 2) % 2]
    c, q, lens, cu, pages = _attend_case(i, lens, new, H, G, D, P)
    _close(*_attend(awq, c, q, lens, cu, pages, dtype, D), dtype, D)


@pytest.mark.parametrize("window", [1, 5, 16, 64, 100, 5000])
@pytest.mark.parametrize("new", [None, [1, 40, 3, 200]])
def test_attention_window(awq, window, new):
    c, q, lens, cu, pages = _attend_case(window, [1, 300, 64, 701], new, 2, 4, 64 if new else 128, 32)
    D = q.shape[2]
    _close(*_attend(awq, c, q, lens, cu, pages, F16, D, window=window), F16, D)


@pytest.mark.parametrize("scale", [1e-3, 1.0, 4.0])
@pytest.mark.parametrize("new", [None, [90]])
def test_attention_flat_and_sharp_rows(awq, scale, new):
    """Scores from nearly equal to one key taking everything."""
    c, q, lens, cu, pages = _attend_case(int(scale * 100), [700], new, 2, 4, 128, 64)
    _close(*_attend(awq, c, q, lens, cu, pages, F16, 128, scale=scale), F16, 128)


@pytest.mark.parametrize("new", [None, [70]])
def test_attention_dominant_key_with_small_value(awq, new):
    """One key takes nearly all the weight and its value block is tiny: the others' values decide the result."""
    c, q, lens, cu, pages = _attend_case(3, [400], new, 1, 4, 128, 64)
    page = pages[0, 0]
    c["k_codes"][page, :, 0] = okv.e4m3_encode(np.full(128, 200.0))
    q = np.abs(q)
    c["v_scales"][page, :, 0] = 2.0 ** -30
    _close(*_attend(awq, c, q, lens, cu, pages, F16, 128), F16, 128)


def test_attention_of_zero_values(awq):
    """Blocks of zeros have the least scale; they still take their weight."""
    c, q, lens, cu, pages = _attend_case(4, [100], None, 1, 8, 64, 32)
    c["v_codes"][pages[0, 0]] = 0
    c["v_scales"][pages[0, 0]] = 2.0 ** -40
    _close(*_attend(awq, c, q, lens, cu, pages, BF16, 64), BF16, 64)


@pytest.mark.parametrize("new", [None, [1, 40]])
def test_attention_extreme_scales(awq, new):
    """Value blocks from the least to the largest scale; keys whose scores stay finite."""
    c, q, lens, cu, pages = _attend_case(5, [90, 200], new, 2, 2, 64, 16)
    ids = pages[pages < (1 << 30)]
    c["v_scales"][ids[::2]] = 2.0 ** -40
    c["v_scales"][ids[1::2]] = 2.0 ** 6
    _close(*_attend(awq, c, q, lens, cu, pages, BF16, 64), BF16, 64)


@pytest.mark.parametrize("new", [None, [3, 2], [50, 40]])
def test_attention_strided_rows_and_rows_of_nobody(awq, new):
    c, q, lens, cu, pages = _attend_case(6, [70, 81], new, 2, 4, 128, 64)
    T = q.shape[0]
    ref, rl, info = okv.attention(c, f64(dev(q, F16)), lens, pages, cu)
    pad = 0 if new is None else 2
    big = torch.full((T + pad, 20, 128), float("nan"), device="cuda", dtype=F16)
    big[:T, 3:11] = dev(q, F16)
    out = torch.full((T + pad, 10, 136), 7.0, device="cuda", dtype=F16)
    qd, od = big[:, 3:11], out[:, 1:9, :128]
    kw = dict(cu_tokens=None if cu is None else ints(cu), max_tokens=1 if new is None else max(new))
    wide = torch.full((2, pages.shape[1] + 3), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, :pages.shape[1]] = ints(pages)
    got, lse = awq.kv_attention(_upload(c), qd, ints(lens), wide[:, :pages.shape[1]], out=od, return_lse=True, **kw)
    awq.get_status()
    assert got is od
    _close(od[:T], lse[:T], ref, rl, info, F16, 128)
    rest = out.clone()
    rest[:T, 1:9, :128] = 7.0
    assert bool((rest == 7).all())


@pytest.mark.parametrize("new", [None, [40, 9]])
def test_attention_reports_pages_outside(awq, new):
    """A bad page is reported and read as if its keys were not there; the other sequence is as ever."""
    c, q, lens, cu, pages = _attend_case(7, [100, 90], new, 2, 4, 64, 32)
    good = _attend(awq, c, q, lens, cu, pages, F16, 64)
    bad = pages.copy()
    bad[0, 1], bad[0, 2] = c["k_codes"].shape[0], -5
    n = 1 if new is None else max(new)
    out = awq.kv_attention(_upload(c), dev(q, F16), ints(lens), ints(bad), None if cu is None else ints(cu), n)
    with pytest.raises(awq.AWQError):
        awq.get_status()
    first = 1 if new is None else new[0]
    assert torch.equal(out[first:], good[0][first:])
    assert bool(torch.isfinite(out).all())
    long = awq.kv_attention(_upload(c), dev(q, F16), ints([100, 10 ** 6]), ints(pages),
                            None if cu is None else ints(cu), n)
    with pytest.raises(awq.AWQError):                                      # longer than the table
        awq.get_status()
    assert torch.equal(long[:first], good[0][:first])


def test_attention_far_pages(awq):
    """Pages whose codes lie past 4 GiB."""
    H, P, D, n_pages = 8, 64, 128, 70000
    cache = awq.kv_cache(n_pages, H, P, D)
    assert cache["k_codes"].numel() > 1 << 32
    c, q, lens, cu, pages = _attend_case(9, [200], None, H, 2, D, P, spoil=False)
    far = np.array([[n_pages - 1, 3, n_pages - 2, 68000, 0]], np.int32)[:, :pages.shape[1]]
    for k in c:
        for i, j in zip(far[0], pages[0]):
            if j < len(c[k]):
                cache[k].view(torch.uint8 if "codes" in k else F32)[int(i)] = dev(c[k][j])
    qd = dev(q, F16)
    ref, rl, info = okv.attention(c, f64(qd), lens, pages)
    out, lse = awq.kv_attention(cache, qd, ints(lens), ints(far), return_lse=True)
    awq.get_status()
    _close(out, lse, ref, rl, info, F16, D)
    out, lse = awq.kv_attention(cache, qd, ints(lens), ints(far), cu_tokens=ints([0, 1]), max_tokens=100, return_lse=True)
    _close(out, lse, ref, rl, info, F16, D)
    # and appended there
    x = torch.randn((1, H, D), device="cuda", dtype=F16)
    before = {k: cache[k].view(torch.uint8 if "codes" in k else F32)[n_pages - 2].clone() for k in cache}
    ref = {k: v.cpu().numpy()[None] for k, v in before.items()}
    awq.kv_append(cache, x, x, ints([150]), ints(far))
    awq.get_status()
    okv.append(ref, x.float().cpu().numpy(), x.float().cpu().numpy(), [150 - 128], np.array([[0]]))
    _same({k: cache[k][n_pages - 2:n_pages - 1] for k in cache}, ref)


@pytest.mark.parametrize("new", [None, [4, 2, 3], [90, 120, 10]])
def test_attention_repeats_to_the_bit(awq, new):
    c, q, lens, cu, pages = _attend_case(10, [3000, 500, 1111], new, 2, 8, 128, 64)
    a = _attend(awq, c, q, lens, cu, pages, BF16, 128)
    b = _attend(awq, c, q, lens, cu, pages, BF16, 128)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    _close(*a, BF16, 128)


@pytest.mark.parametrize("new", [None, [5, 3], [60, 130]])
def test_captured_steps_share_a_workspace(awq, new):
    """Two captured graphs with one workspace, replayed in turn with other lengths, on a stream of their own."""
    cases = [_attend_case(20 + i, [900, 333], new, 2, 4, 128, 64) for i in range(2)]
    n = 1 if new is None else max(new)
    ws = torch.empty(awq.kv_attention_workspace_bytes(_upload(cases[0][0]), cases[0][1].shape[0], 8, n),
                     dtype=torch.uint8, device="cuda")
    ws.fill_(0xff)
    side, graphs = torch.cuda.Stream(), []
    for c, q, lens, cu, pages in cases:
        s = dict(cache=_upload(c), q=dev(q, F16), lens=ints(lens), pages=ints(pages), cu=None if cu is None else ints(cu))
        s["out"] = torch.zeros(q.shape, device="cuda", dtype=F16)
        call = lambda s=s: awq.kv_attention(s["cache"], s["q"], s["lens"], s["pages"], s["cu"], n, out=s["out"],  # noqa: E731
                                            workspace=ws)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                call()
        s["out"].zero_()
        graphs.append((g, s))
    torch.cuda.synchronize()
    for lens in ([900, 333], [700, 332]):
        for (g, s), (c, q, _, cu, pages) in zip(graphs, cases):
            s["lens"].copy_(ints(lens))
            g.replay()
        torch.cuda.synchronize()
        for (g, s), (c, q, _, cu, pages) in zip(graphs, cases):
            ref, _, info = okv.attention(c, f64(s["q"]), lens, pages, cu)
            assert np.all(np.abs(f64(s["out"]) - ref) <= bound(ref, info, F16, 128))
    awq.get_status()


def test_another_stream_than_the_current_one(awq):
    c, q, lens, cu, pages = _attend_case(30, [640], None, 2, 4, 128, 64)
    side = torch.cuda.Stream()
    s = [_upload(c), dev(q, F16), ints(lens), ints(pages)]
    x = torch.randn((1, 2, 128), device="cuda")
    table = awq.rope_table(700, 128)
    torch.cuda.synchronize()
    y = awq.rope(x, ints([5]), table, stream=side)
    out, lse = awq.kv_attention(*s, return_lse=True, stream=side)
    awq.kv_append(s[0], x, x, s[2], s[3], table=table, stream=side)
    side.synchronize()
    awq.get_status(side)
    assert torch.equal(y, awq.rope(x, ints([5]), table))
    ref, rl, info = okv.attention(c, f64(s[1]), lens, pages)
    _close(out, lse, ref, rl, info, F16, 128)


def test_binding_refuses(awq):
    cache = awq.kv_cache(4, 2, 16, 64)
    x = torch.zeros((2, 2, 64), device="cuda", dtype=F16)
    lens, pages = ints([1, 1]), ints([[0], [1]])
    with pytest.raises(ValueError):
        awq.kv_append(cache, x, x, lens, pages, q=x)                       # q without a table
    with pytest.raises(ValueError):
        awq.kv_append(cache, x[:1], x[:1], lens, pages)                    # one row, two sequences
    with pytest.raises(ValueError):
        awq.kv_attention(cache, torch.zeros((2, 2, 128), device="cuda", dtype=F16), lens, pages)
    with pytest.raises(TypeError):
        awq.kv_attention(cache, x, lens.long(), pages)
    with pytest.raises(TypeError):
        awq.kv_attention({**cache, "k_codes": cache["k_codes"].half()}, x, lens, pages)
    with pytest.raises(ValueError):
        awq.kv_attention({**cache, "v_scales": cache["v_scales"][:2]}, x, lens, pages)
    with pytest.raises(ValueError):
        awq.kv_attention(cache, x.transpose(1, 2), lens, pages)
    with pytest.raises(awq.AWQError):
        awq.kv_attention(cache, x.float(), lens, pages)
    with pytest.raises(awq.AWQError):
        awq.kv_attention(cache, x, lens, pages, workspace=torch.empty(1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(awq.AWQError):
        awq.kv_attention(cache, torch.zeros((2, 3, 64), device="cuda", dtype=F16), lens, pages)
    empty = awq.kv_attention(cache, x[:0], lens[:0], pages[:0])
    assert empty.shape == (0, 2, 64) and awq.rope(x[:0], lens[:0], awq.rope_table(4, 64)).shape == (0, 2, 64)
    assert awq.kv_append(cache, x[:0], x[:0], lens[:0], pages[:0]) is None
    awq.get_status()


def test_a_workspace_of_the_wrong_kind_is_refused(awq):
    """Host memory, another type, every second byte: refused before anything is launched."""
    cache, x = awq.kv_cache(4, 2, 16, 64), torch.zeros((2, 2, 64), device="cuda", dtype=F16)
    lens, pages = ints([0, 0]), ints([[0], [1]])
    n = awq.kv_attention_workspace_bytes(cache, 2, 2)
    for ws, error in ((torch.empty(n, dtype=torch.uint8), TypeError),
                      (torch.empty(n, dtype=torch.float32, device="cuda"), TypeError),
                      (torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2], ValueError), (n, TypeError)):
        with pytest.raises(error):
            awq.kv_attention(cache, x, lens, pages, workspace=ws)
    own = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert not bool(awq.kv_attention(cache, x, lens, pages, workspace=own).any())      # no keys: zeros
    awq.get_status()


@pytest.mark.parametrize("D,G,new,past", [(128, 8, 40, 300), (64, 2, 150, 0), (128, 4, 9, 1500), (128, 8, 1, 900),
                                          (64, 1, 1, 700), (128, 4, 4, 200), (64, 8, 3, 1100)])
def test_many_calls_in_a_row_never_wait_in_vain(awq, D, G, new, past):
    """Some millions of blocks of threads, launched as densely as a graph can: a wait that a late warp may miss runs
    into its limit here (reported, and seen in the time), and all results are those of the first call."""
    n, H = 48, 2
    c, q, lens, cu, pages = _attend_case(71, [past + new + i % 5 for i in range(n)], [new] * n, H, G, D, 64)
    cache, qd, l, u, p = _upload(c), dev(q, F16), ints(lens), ints(cu), ints(pages)
    ws = torch.empty(awq.kv_attention_workspace_bytes(cache, q.shape[0], H * G, new), dtype=torch.uint8, device="cuda")
    first = awq.kv_attention(cache, qd, l, p, u, new, workspace=ws)
    out = torch.empty_like(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(100):
            awq.kv_attention(cache, qd, l, p, u, new, workspace=ws, out=out)
    for _ in range(100):
        g.replay()
    torch.cuda.synchronize()
    awq.get_status()
    assert torch.equal(out, first)


# ----- a run of them together ----------------------------------------------------
@pytest.mark.parametrize("new", [None, [40, 3]])
def test_attention_step_of_a_quantized_block(awq, new):
    """qkv projection, append, attention, output projection as a model's step runs them: the step equals its parts,
    and the parts equal the oracle, over a prompt and the token after it."""
    import oracle
    from awq_activation_aware_b200 import synth
    HQ, H, D, hidden, P = 8, 2, 64, 512, 32
    W, X, _ = synth.generate(synth.make_config((HQ + 2 * H) * D, hidden, 256, bits=4, group=128, seed=3))
    qkv = awq.quantize_layer(dev(W), dev(X))
    Wo, Xo, _ = synth.generate(synth.make_config(hidden, HQ * D, 256, bits=4, group=128, seed=4))
    o = awq.quantize_layer(dev(Wo), dev(Xo))
    lens = [40, 3]
    pages = np.array([[1, 4, 0], [2, 3, 5]], np.int32)
    table = awq.rope_table(96, D)
    cache = awq.kv_cache(6, H, P, D)
    ref = {k: np.zeros(t.shape, np.uint8 if k.endswith("codes") else np.float32) for k, t in cache.items()}
    steps = [(lens, [0, 40, 43], 40), ([41, 4], None, 1)]
    if new is None:
        steps = [([1, 1], None, 1), ([2, 2], None, 1)]
    at = 0
    for ln, cu, n in steps:
        T = 2 if cu is None else cu[-1]
        x = dev(X[at:at + T])
        at += T
        y = awq.attention_step(x, qkv, o, cache, ints(ln), ints(pages), table, HQ, None if cu is None else ints(cu), n)
        awq.get_status()
        # the parts, on the host
        Y = awq.qlinear(qkv["codes"], qkv["scales"], qkv["zeros"], qkv["s_best"], x).view(T, HQ + 2 * H, D).cpu().numpy()
        okv.append(ref, Y[:, HQ:HQ + H], Y[:, HQ + H:], ln, pages, cu, table.cpu().numpy())
        written = {k: cache[k].view(torch.uint8 if k.endswith("codes") else F32).cpu().numpy() for k in cache}
        pos = np.array([p[1] for p in okv.rows_of(ln, cu, T)])
        for b, L in enumerate(ln):
            for j in range(L):
                for w in "kv":
                    np.testing.assert_array_equal(written[w + "_codes"][pages[b, j // P], :, j % P],
                                                  ref[w + "_codes"][pages[b, j // P], :, j % P])
        q = _rounded(okv.rotate(Y[:, :HQ], table.cpu().numpy()[pos], "half"), F16)
        a, _, info = okv.attention(ref, q.double().numpy(), ln, pages, cu)
        a_got = awq.kv_attention(cache, q.cuda(), ints(ln), ints(pages), None if cu is None else ints(cu), n)
        assert np.all(np.abs(f64(a_got) - a) <= bound(a, info, F16, D))
        out = awq.qlinear(o["codes"], o["scales"], o["zeros"], o["s_best"], a_got.view(T, HQ * D))
        assert torch.equal(y, out)
        Yr = oracle.qlinear(o["codes"].cpu().numpy().view(np.uint32), o["scales"].cpu().numpy(), o["zeros"].cpu().numpy(),
                            o["s_best"].cpu().numpy(), a_got.view(T, -1).cpu().numpy(), 4, 128)
        assert np.abs(f64(y) - Yr).max() <= 1e-4 * np.abs(Yr).max()
    awq.get_status()


# ----- where the kernels change over, and what a hostile call could reach ---------
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,G", [(1, 8), (3, 3), (2, 8), (17, 1), (3, 8), (8, 4), (11, 3), (5, 8), (64, 2), (43, 3), (129, 2)])
def test_attention_at_every_number_of_rows(awq, D, n, G):
    """Rows a key head from 8 to 258: tiles of 8, 16 and 32 rows, then 128 and 256."""
    c, q, lens, cu, pages = _attend_case(n * G + D, [n + 100, n + 700, n], [n, max(n - 1, 1), n], 2, G, D, 64)
    _close(*_attend(awq, c, q, lens, cu, pages, BF16 if G % 2 else F16, D), BF16 if G % 2 else F16, D)


@pytest.mark.parametrize("n", [1, 6, 40])
def test_attention_of_many_short_sequences(awq, n):
    """More sequences than blocks of threads, empty ones among them."""
    rng = np.random.default_rng(n)
    lens = rng.integers(0, 40, 700)
    lens[::7] = 0
    new = None if n == 1 else np.minimum(lens, rng.integers(0, n + 1, 700))
    if new is not None:
        new[0], lens[0] = n, max(lens[0], n)
    c, q, lens, cu, pages = _attend_case(n, lens, new, 1, 4, 64, 16)
    _close(*_attend(awq, c, q, lens, cu, pages, F16, 64), F16, 64)


@pytest.mark.parametrize("n,G", [(4, 2), (8, 4), (40, 4)])
def test_attention_nan_only_where_it_is_seen(awq, n, G):
    """A value or key that is NaN reaches the rows that see it and no other."""
    c, q, lens, cu, pages = _attend_case(50 + n, [150, 90], [n, n], 2, G, 128, 32)
    clean = _attend(awq, c, q, lens, cu, pages, F16, 128)
    hidden = 150 - n + n // 2                                              # seen by the later half of the first sequence's rows
    for w, at in (("v", (pages[0, hidden // 32], 1, hidden % 32, 5)), ("k", (pages[0, hidden // 32], 0, hidden % 32, 9))):
        d = {k: v.copy() for k, v in c.items()}
        d[w + "_codes"][at] = 127
        out, lse = _attend(awq, d, q, lens, cu, pages, F16, 128)[:2]
        head = slice(G, 2 * G) if w == "v" else slice(0, G)
        sees = torch.zeros(out.shape[:2], dtype=torch.bool, device="cuda")
        sees[n // 2:n, head] = True
        assert torch.equal(out[~sees], clean[0][~sees]) and torch.equal(lse[~sees], clean[1][~sees])
        bad = torch.isnan(out[sees])
        assert bool(bad[:, 5].all()) if w == "v" else bool(bad.all())


@pytest.mark.parametrize("new", [[5, 3], [70, 3]])
def test_attention_reports_more_tokens_than_promised(awq, new):
    c, q, lens, cu, pages = _attend_case(60, [200, 90], new, 2, 4, 64, 32)
    good = _attend(awq, c, q, lens, cu, pages, F16, 64)[0]
    out = torch.full(q.shape, 7.0, device="cuda", dtype=F16)
    awq.kv_attention(_upload(c), dev(q, F16), ints(lens), ints(pages), ints(cu), new[0] - 1, out=out)
    with pytest.raises(awq.AWQError):
        awq.get_status()
    assert bool((out[:new[0]] == 7).all())                                 # not computed, not touched
    d = f64(out[new[0]:]) - f64(good[new[0]:])
    assert np.abs(d).max() <= 2.0 ** -9 * np.abs(f64(good)).max()          # the other sequence is (by another kernel, maybe)


@pytest.mark.parametrize("new", [None, [6, 5], [90, 70]])
def test_two_calls_at_once(awq, new):
    """Two streams, each with its own workspace."""
    cases = [_attend_case(70 + i, [1500, 700], new, 2, 4, 128, 64) for i in range(2)]
    n = 1 if new is None else max(new)
    alone = [_attend(awq, *c, F16, 128)[0] for c in cases]
    args = [(_upload(c), dev(q, F16), ints(lens), ints(pages), None if cu is None else ints(cu), n)
            for c, q, lens, cu, pages in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(8):
        for i in range(2):
            outs[i].append(awq.kv_attention(*args[i], stream=streams[i]))
    torch.cuda.synchronize()
    awq.get_status()
    for i in range(2):
        assert all(torch.equal(o, alone[i]) for o in outs[i])


@pytest.mark.parametrize("new", [None, [3, 0, 40]])
def test_a_captured_step_follows_its_inputs(awq, new):
    """Append and attention captured together, replayed as the sequences grow, equal to the calls made one by one."""
    rng = np.random.default_rng(80)
    H, HQ, D, P = 2, 8, 64, 32
    T = 3 if new is None else sum(new)
    pages = rng.permutation(18).astype(np.int32).reshape(3, 6)
    table = awq.rope_table(192, D)
    cu = None if new is None else ints(np.concatenate([[0], np.cumsum(new)]))
    n = 1 if new is None else max(new)
    base = _random_cache(rng, 18, H, P, D)
    live, ref = _upload(base), _upload(base)
    x = torch.randn((T, HQ + 2 * H, D), device="cuda")
    lens = ints([50, 1, 40])
    out = torch.empty((T, HQ, D), device="cuda", dtype=F16)
    ws = torch.empty(awq.kv_attention_workspace_bytes(live, T, HQ, n), dtype=torch.uint8, device="cuda")

    def step(cache, out):
        q = awq.kv_append(cache, x[:, HQ:HQ + H], x[:, HQ + H:], lens, ints_pages, cu, table, q=x[:, :HQ])
        return awq.kv_attention(cache, q, lens, ints_pages, cu, n, out=out, workspace=ws)

    ints_pages = ints(pages)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(_upload(base), out)                                           # kernels are loaded before the capture
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step(live, out)
    torch.cuda.synchronize()
    for i in range(5):
        x.copy_(torch.randn_like(x) * 2.0 ** i)
        lens += 7 if new else 1
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        want = step(ref, torch.empty_like(out))
        awq.get_status()
        assert torch.equal(got, want)
        for k in live:
            a, b = (t[k].view(torch.uint8) if k.endswith("codes") else t[k] for t in (live, ref))
            assert torch.equal(a, b)


@pytest.mark.parametrize("cu", [[0, 5, 3, 9], [2, 4, 4, 40], [-3, 2, 5, 6]])
def test_token_offsets_that_make_no_sense_stay_inside_the_arrays(awq, cu):
    """Offsets that decrease, start late or pass the rows: whatever is computed, rows and pages outside are not touched."""
    rng = np.random.default_rng(90)
    c, _, _, _, pages = _attend_case(90, [40, 33, 60], None, 1, 2, 64, 16)
    T = 8
    x = torch.randn((T + 2, 4, 64), device="cuda", dtype=F16)
    guard = torch.full((T + 2, 2, 64), 7.0, device="cuda", dtype=F16)
    cache = _upload(c)
    awq.kv_append(cache, x[:T, 2:3], x[:T, 3:], ints([40, 33, 60]), ints(pages), ints(cu), awq.rope_table(64, 64),
                  q=x[:T, :2], q_out=guard[:T])
    for most in (16, 40):
        awq.kv_attention(cache, x[:T, :2], ints([40, 33, 60]), ints(pages), ints(cu), most, out=guard[:T])
    torch.cuda.synchronize()
    try:
        awq.get_status()
    except awq.AWQError:
        pass
    assert bool((guard[T:] == 7).all())


# ----- NaN queries and keys, wherever the work is cut -----------------------------
def _close_but_nan(out, lse, ref, rl, info, dtype, D):
    """As _close, but rows whose log-sum-exp is NaN have to be NaN in every element and in the log-sum-exp."""
    bad = np.isnan(rl)
    assert bad.any()
    got, got_lse = f64(out), f64(lse)
    assert np.isnan(got[bad]).all() and np.isnan(got_lse[bad]).all()
    assert not np.isnan(got[~bad]).any() and not np.isnan(got_lse[~bad]).any()
    fine = np.nonzero(~bad)
    _close(out[fine], lse[fine], ref[fine], rl[fine], tuple(x[fine] for x in info), dtype, D)


NAN_CASES = [  # lengths, new tokens, key heads, group, page columns beyond the sequences': what is cut how
    ([40], None, 1, 4, 0), ([33], None, 2, 8, 0),                  # one unit of keys, two warps' parts of it
    ([1000, 0, 300], None, 2, 4, 0), ([513], None, 8, 8, 0),       # segments cut, joined by segment
    ([200] * 300, None, 2, 1, 0),                                  # more segments than blocks of threads
    ([1000, 2, 300], [4, 5, 2], 2, 4, 0), ([900, 129], [8, 3], 2, 4, 0),     # drafts: tiles of 16 and 32 rows
    ([90, 2], [90, 5], 2, 4, 0), ([700, 0, 300], [90, 0, 20], 2, 4, 0), ([513], [40], 1, 8, 40),   # the kernel for many rows
]


@pytest.mark.parametrize("D,dtype", [(128, F16), (64, BF16)])
@pytest.mark.parametrize("lens,new,H,G,extra", NAN_CASES)
def test_attention_of_nan_queries(awq, lens, new, H, G, extra, D, dtype):
    """A NaN in a query, in one element or in all, is NaN in its row's result whatever the row is joined from; a row
    without keys stays empty, and no other row is touched."""
    c, q, lens, cu, pages = _attend_case(100 + len(lens) + G, lens, new, H, G, D, 32)
    pages = np.concatenate([pages, np.full((len(lens), extra), 1 << 30, np.int32)], 1)
    q[::2, 0], q[1::3, -1, 5], q[-1, (H * G) // 2, D - 1] = np.nan, np.nan, np.nan
    _close_but_nan(*_attend(awq, c, q, lens, cu, pages, dtype, D), dtype, D)


@pytest.mark.parametrize("D,dtype", [(128, F16), (64, BF16)])
@pytest.mark.parametrize("lens,new,H,G,extra", NAN_CASES)
@pytest.mark.parametrize("from_end", [1, 33])
def test_attention_of_nan_keys(awq, lens, new, H, G, extra, D, dtype, from_end):
    """A NaN in a sequence's last key (which opens a tile of its own where the length is 64 n + 1), or in one further
    back: NaN in the rows that see it, and in their log-sum-exp."""
    c, q, lens, cu, pages = _attend_case(200 + len(lens) + G, lens, new, H, G, D, 32)
    pages = np.concatenate([pages, np.full((len(lens), extra), 1 << 30, np.int32)], 1)
    for b, n in enumerate(lens):
        if n >= from_end:
            c["k_codes"][pages[b, (n - from_end) // 32], b % H, (n - from_end) % 32, 7] = 127
    _close_but_nan(*_attend(awq, c, q, lens, cu, pages, dtype, D), dtype, D)


# ----- steps of layers packed in other ways, and with the other options ------------
@pytest.mark.parametrize("a,b,layout,window", [((2, 64), (4, 128), "interleaved", 0), ((4, 64), (2, 128), None, 5),
                                               ((3, 128), (3, 64), "half", 20)])
def test_attention_step_of_reloaded_layers(awq, tmp_path, a, b, layout, window):
    """Layers packed with different bits and groups, saved and loaded: the step reads each as it was packed, and equals
    its parts (layout None: no rotation)."""
    from awq_activation_aware_b200 import persist, synth
    HQ, H, D, hidden = 4, 2, 64, 384
    layers = []
    for i, (N, K, (bits, group)) in enumerate((((HQ + 2 * H) * D, hidden, a), (hidden, HQ * D, b))):
        W, X, _ = synth.generate(synth.make_config(N, K, 256, bits=bits, group=group, seed=5 + i))
        persist.save_quantized(tmp_path / "layer", awq.quantize_layer(dev(W), dev(X), bits=bits, group=group), bits, group)
        layers.append(persist.load_quantized(tmp_path / "layer", "cuda"))
    qkv, o = layers
    lin = lambda q, x: awq.qlinear(q["codes"], q["scales"], q["zeros"], q["s_best"], x, q["bits"], q["group_size"])  # noqa: E731
    table = awq.rope_table(64, D) if layout else None
    pages = ints([[1, 0], [3, 2]])
    cache, mine = (awq.kv_cache(4, H, 32, D) for _ in range(2))
    gen = torch.Generator(device="cuda").manual_seed(6)
    for lens, cu, most in (([30, 7], [0, 30, 37], 30), ([31, 8], None, 1)):
        T = 2 if cu is None else cu[-1]
        x = torch.randn((T, hidden), device="cuda", generator=gen).half()
        cu = None if cu is None else ints(cu)
        y = awq.attention_step(x, qkv, o, cache, ints(lens), pages, table, HQ, cu, most, layout or "half", window)
        z = lin(qkv, x).view(T, HQ + 2 * H, D)
        q = awq.kv_append(mine, z[:, HQ:HQ + H], z[:, HQ + H:], ints(lens), pages, cu, table, layout or "half",
                          q=z[:, :HQ] if layout else None)
        at = awq.kv_attention(mine, q if layout else z[:, :HQ].half(), ints(lens), pages, cu, most, window=window)
        assert torch.equal(y, lin(o, at.view(T, HQ * D)))
        assert bool(torch.isfinite(y).all()) and bool(y.abs().max() > 0)
    for bad in (dict(bits=a[0] - 1), dict(group=64 if a[1] == 128 else 128)):
        with pytest.raises(ValueError):
            awq.attention_step(x, qkv, o, cache, ints(lens), pages, table, HQ, **bad)
    with pytest.raises(TypeError):                                         # a layer that is not on the device
        awq.attention_step(x, qkv, o | dict(zeros=o["zeros"].cpu()), cache, ints(lens), pages, table, HQ)
    awq.get_status()


def _guarded(t, fill):
    """t's values in the middle of a larger buffer, and that buffer's view as bytes."""
    pad = 4096                                                             # bytes: keeps every alignment
    raw = torch.full((t.numel() * t.element_size() + 2 * pad,), fill, dtype=torch.uint8, device="cuda")
    mid = raw[pad:-pad].view(t.dtype).view(t.shape)
    mid.copy_(t)
    return mid, raw


@pytest.mark.parametrize("cu", [[0, 5, 3, 9], [2, 4, 4, 40], [-3, 2, 5, 6], [9, 9, 9, 9], [8, 6, 2, 0], [0, -5, 8, 8],
                                [-(1 << 31), 3, 3, (1 << 31) - 1], [0, 3, 6, 8]])
@pytest.mark.parametrize("lens", [[40, 33, 60], [-7, 0, 2], [(1 << 31) - 1, 47, -(1 << 31)]])
def test_senseless_offsets_and_lengths_touch_nothing_else(awq, cu, lens):
    """Append and attention (both kernels) with offsets that decrease, start late or pass the rows, and lengths past the
    page table or below zero.  The memory around every array that is written, pages that no table names, and rows past
    the given ones keep their bytes."""
    rng = np.random.default_rng(91)
    H, HQ, D, P, T = 1, 2, 64, 16, 8
    base = _random_cache(rng, 16, H, P, D)
    pages = np.array([[3, 14, 7, 9], [1, 12, 5, 11], [2, 6, 13, 8]], np.int32)      # 0, 4, 10 and 15 are nobody's
    held = {k: _guarded(t.view(torch.uint8) if k.endswith("codes") else t, 0x5a) for k, t in _upload(base).items()}
    cache = {k: v[0] for k, v in held.items()}
    x = torch.randn((T + 2, HQ + 2 * H, D), device="cuda", dtype=F16)
    table = awq.rope_table(64, D)
    q_out, q_raw = _guarded(torch.zeros((T, HQ, D), dtype=F16), 0x5a)
    out, out_raw = _guarded(torch.zeros((T, HQ, D), dtype=F16), 0x5a)
    lse, lse_raw = _guarded(torch.zeros((T, HQ)), 0x5a)
    awq.kv_append(cache, x[:T, HQ:HQ + H], x[:T, HQ + H:], ints(lens), ints(pages), ints(cu), table, q=x[:T, :HQ], q_out=q_out)
    wide = torch.full((3, 9), 15, dtype=torch.int32, device="cuda")       # columns past max_pages name a page of nobody
    wide[:, :4] = ints(pages)
    raws = [raw for _, raw in held.values()] + [q_raw, out_raw, lse_raw]
    for most in (1, 8, 16, 40):
        n = awq.kv_attention_workspace_bytes(cache, T, HQ, most)
        ws = torch.full((n + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
        seq, off = ints(lens), ints(cu)
        code = awq.lib().awq_kv_attention(
            awq.kv._cache(cache, 0, D), awq.kv._batch(seq, wide[:, :4], off, T, 0), T, awq.kv._rows(x[:T, :HQ], "q", 0),
            awq.kv._rows(out, "out", 0), 0.125, most, 0, lse.data_ptr(), ws.data_ptr(), n,
            torch.cuda.current_stream().cuda_stream)
        assert code == 0
        torch.cuda.synchronize()
        assert bool((ws[n:] == 0x5a).all())
    for raw in raws:
        assert bool((raw[:4096] == 0x5a).all() and (raw[-4096:] == 0x5a).all())
    for k, b in base.items():
        got = cache[k].cpu().numpy()
        np.testing.assert_array_equal(got[[0, 4, 10, 15]], b[[0, 4, 10, 15]], err_msg=k)
        # no position of a page table is reached by a sequence without tokens in it
        if lens == [-7, 0, 2]:
            np.testing.assert_array_equal(got[[14, 7, 9, 12, 5, 11, 6, 13, 8]], b[[14, 7, 9, 12, 5, 11, 6, 13, 8]], err_msg=k)
    try:
        awq.get_status()
    except awq.AWQError as e:
        assert e.code == 1


@pytest.mark.parametrize("D,dtype", [(128, F16), (64, BF16), (64, F16)])
@pytest.mark.parametrize("lens,new,H,G,extra", NAN_CASES)
def test_attention_of_infinite_queries(awq, lens, new, H, G, extra, D, dtype):
    """An infinite element makes every score of its row infinite or NaN, so the row is NaN -- also where all scores are
    -inf: channels whose keys have one sign are common."""
    c, q, lens, cu, pages = _attend_case(300 + len(lens) + G, lens, new, H, G, D, 32)
    pages = np.concatenate([pages, np.full((len(lens), extra), 1 << 30, np.int32)], 1)
    codes = c["k_codes"][..., 7]
    codes[codes != 127] &= 127                                             # this channel's keys: none below zero, none zero
    codes[codes == 0] = 1
    q[::2, 0, 7], q[1::3, -1, 7], q[-1, (H * G) // 2, 7] = -np.inf, np.inf, -np.inf
    with np.errstate(invalid="ignore"):                                    # the oracle's inf - inf
        _close_but_nan(*_attend(awq, c, q, lens, cu, pages, dtype, D), dtype, D)


def _step_of(awq, HQ, H, D, hidden, seed):
    """Random packed layers of an attention block: Q, K and V stacked, and the output projection."""
    from awq_activation_aware_b200 import synth
    out = []
    for i, (N, K) in enumerate((((HQ + 2 * H) * D, hidden), (hidden, HQ * D))):
        W, X, _ = synth.generate(synth.make_config(N, K, 256, bits=4, group=128, seed=seed + i))
        out.append(awq.quantize_layer(dev(W), dev(X)))
    return out


@pytest.mark.parametrize("new", [[1, 1], [3, 2], [40, 9]])
def test_attention_step_of_a_padded_batch(awq, new):
    """Rows behind the last sequence may hold anything: no other row, and no byte of the cache, depends on them."""
    HQ, H, D, hidden = 4, 2, 64, 256
    qkv, o = _step_of(awq, HQ, H, D, hidden, 11)
    T, pad, lens = sum(new), 5, [new[0] + 20, new[1]]
    pages, table, cu = ints([[1, 0, 4], [3, 2, 5]]), awq.rope_table(96, D), ints([0, new[0], T])
    x = torch.randn((T + pad, hidden), device="cuda").half()
    base, got = _upload(_random_cache(np.random.default_rng(12), 6, H, 32, D)), []
    for fill in (0.0, float("nan"), 6e4):
        x[T:] = fill
        cache = {k: t.clone() for k, t in base.items()}
        y = awq.attention_step(x, qkv, o, cache, ints(lens), pages, table, HQ, cu, max(new))
        got.append([y[:T]] + [t.view(torch.uint8) if t.dtype != F32 else t for t in cache.values()])
    awq.get_status()
    assert bool(torch.isfinite(got[0][0]).all())
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


@pytest.mark.parametrize("new", [None, [6, 0, 2]])
def test_a_captured_attention_step_follows_its_inputs(awq, new):
    """The whole step captured once, replayed as the sequences grow, equal to the step called each time."""
    HQ, H, D, hidden = 4, 2, 64, 256
    qkv, o = _step_of(awq, HQ, H, D, hidden, 13)
    T, most = (3, 1) if new is None else (sum(new), max(new))
    cu = None if new is None else ints(np.concatenate([[0], np.cumsum(new)]))
    pages, table = ints(np.random.default_rng(14).permutation(12).reshape(3, 4)), awq.rope_table(128, D)
    base = _random_cache(np.random.default_rng(15), 12, H, 32, D)
    live, ref = _upload(base), _upload(base)
    x, lens = torch.randn((T, hidden), device="cuda").half(), ints([30, 9, 64])
    step = lambda cache: awq.attention_step(x, qkv, o, cache, lens, pages, table, HQ, cu, most)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(_upload(base))                                                # kernels are loaded before the capture
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = step(live)
    torch.cuda.synchronize()
    for i in range(4):
        x.copy_(torch.randn_like(x) * (i + 1))
        lens += most
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, step(ref))
        for k in live:
            a, b = (t[k].view(torch.uint8) if k.endswith("codes") else t[k] for t in (live, ref))
            assert torch.equal(a, b)
    awq.get_status()
