"""Oracle of the cache operators (test infrastructure only): rotary positions,
append to the paged 8-bit cache, attention over it.

Attention and the angles are binary64.  Rotation and append are stated in
binary32 operations, each rounded once (numpy rounds every operation), because
their codes are compared bit for bit.  Nothing here comes from the library.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK, E_MIN, E_MAX = 16, -40, 40

# The 256 values of e4m3: sign, 4 exponent bits (bias 7), 3 fraction bits;
# exponent 0 is subnormal, 0x7f and 0xff are NaN, there is no infinity.
_mag = np.array([(f / 8) * 2.0 ** -6 if x == 0 else (1 + f / 8) * 2.0 ** (x - 7) for x in range(16) for f in range(8)])
_mag[127] = np.nan
E4M3 = np.concatenate([_mag, -_mag])


def e4m3_encode(x) -> np.ndarray:
    """Codes of float32 values: nearest, ties to the even code, saturated at 448, NaN to NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_mag[:127], a), 0, 126)          # _mag[hi - 1] < a <= _mag[hi]
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = a - _mag[lo], _mag[hi] - a
    code = np.where((dlo < dhi) | ((dlo == dhi) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(x), 127, code)
    return (code | (np.signbit(x) & ~np.isnan(x)) * 128).astype(np.uint8)


def e4m3_decode(c) -> np.ndarray:
    return E4M3[np.asarray(c)]


def frequencies(rot, base=10000.0, scaling=None, factor=1.0, original=0.0, beta_fast=32.0, beta_slow=1.0,
                magnitude=0.0):
    """(f [rot / 2], magnitude) in binary64."""
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling != "yarn":
        return f, 1.0
    edge = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    lo, hi = max(math.floor(edge(beta_fast)), 0), min(math.ceil(edge(beta_slow)), rot - 1)
    w = np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
    return f * (1 - w) + f / factor * w, magnitude or 0.1 * math.log(factor) + 1.0


def rope_table(n_pos, rot, **kw):
    """float64 [n_pos, rot / 2, 2]."""
    f, m = frequencies(rot, **kw)
    t = np.arange(n_pos, dtype=np.float64)[:, None] * f[None, :]
    return np.stack([np.cos(t), np.sin(t)], axis=-1) * m


def rotate(x, cs, layout, inverse=False):
    """Rows x [T, H, D] turned by cs [T, rot / 2, 2]; in cs's type (binary32: one rounding an operation)."""
    half = cs.shape[1]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1] * cs.dtype.type(-1 if inverse else 1)
    y = np.array(x, dtype=cs.dtype)
    a, b = (slice(0, half), slice(half, 2 * half)) if layout == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    x1, x2 = y[..., a].copy(), y[..., b].copy()
    y[..., a] = x1 * c - x2 * s
    y[..., b] = x2 * c + x1 * s
    return y


def rows_of(seq_lens, cu, T):
    """(sequence, position) of every row; None for rows that belong to nobody."""
    out = [None] * T
    for b in range(len(seq_lens)):
        r0, r1 = (b, b + 1) if cu is None else (int(cu[b]), int(cu[b + 1]))
        for t in range(r0, min(r1, T)):
            out[t] = (b, int(seq_lens[b]) - (r1 - r0) + t - r0)
    return out


def exponent(amax) -> int:
    """The least e in [-40, 40] with amax <= 448 * 2^e."""
    for e in range(E_MIN, E_MAX):
        if amax <= 448.0 * 2.0 ** e:
            return e
    return E_MAX


def append(cache, k, v, seq_lens, pages, cu=None, table=None, layout="half"):
    """Append in place to a dict of numpy arrays (codes uint8, scales float32); k, v float32, table float32."""
    T, H, D = k.shape
    P = cache["k_codes"].shape[2]
    limit = pages.shape[1] * P if table is None else min(pages.shape[1] * P, table.shape[0])
    blocks = {}
    for t, place in enumerate(rows_of(seq_lens, cu, T)):
        if place is not None and 0 <= place[1] < limit:
            b, pos = place
            blocks.setdefault((b, pos // BLOCK), []).append((t, pos))
    for (b, blk), rows in blocks.items():
        page, o = int(pages[b, blk * BLOCK // P]), blk * BLOCK % P
        if not 0 <= page < cache["k_codes"].shape[0]:
            continue
        off = rows[0][1] % BLOCK
        ts, ps = [r[0] for r in rows], np.array([r[1] for r in rows])
        for w, x in (("k", k[ts]), ("v", v[ts])):
            y = x if w == "v" or table is None else rotate(x, table[ps], layout)
            for h in range(H):
                fine = np.abs(y[:, h][np.isfinite(y[:, h])])
                e = exponent(float(fine.max()) if fine.size else 0.0)
                codes, scales = cache[w + "_codes"][page, h], cache[w + "_scales"][page, h]
                if off:
                    old = int(math.frexp(float(scales[o // BLOCK]))[1]) - 1
                    if e > old:
                        codes[o:o + off] = e4m3_encode(e4m3_decode(codes[o:o + off]) * 2.0 ** (old - e))
                    e = max(e, old)
                scales[o // BLOCK] = 2.0 ** e
                z = np.where(np.isfinite(y[:, h]), y[:, h].astype(np.float64), np.nan) * 2.0 ** -e
                codes[o + off:o + off + len(ts)] = e4m3_encode(z)


def attention(cache, q, seq_lens, pages, cu=None, scale=None, window=0):
    """(out, lse, what a tolerance needs) in binary64.  The last, per row and head: sum_j p_j |v_j| (per element),
    the largest scale * sum |q| |k_j|, the largest p_j * value scale, the number of keys."""
    T, HQ, D = q.shape
    n_pages, H, P, _ = cache["k_codes"].shape
    scale = D ** -0.5 if scale is None else scale
    out, lse = np.zeros((T, HQ, D)), np.full((T, HQ), -np.inf)
    mass, reach, peak, keys = np.zeros((T, HQ, D)), np.zeros((T, HQ)), np.zeros((T, HQ)), np.zeros((T, HQ))
    known = {}
    for t, place in enumerate(rows_of(seq_lens, cu, T)):
        if place is None or place[1] < 0:
            continue
        b, pos = place
        if b not in known:
            S = min(int(seq_lens[b]), pages.shape[1] * P)
            ids = pages[b, :-(-S // P)]
            got = []
            for w in ("k", "v"):
                s = np.repeat(cache[w + "_scales"][ids].astype(np.float64), BLOCK, axis=-1)
                x = e4m3_decode(cache[w + "_codes"][ids]) * s[..., None]
                got += [x.transpose(1, 0, 2, 3).reshape(H, -1, D), s.transpose(1, 0, 2).reshape(H, -1)]
            known[b] = (S, got)
        S, (kk, _, vv, vs) = known[b]
        hi = min(pos + 1, S)
        lo = max(0, pos + 1 - window) if window else 0
        if lo >= hi:
            continue
        for h in range(HQ):
            g = h // (HQ // H)
            K, V = kk[g, lo:hi], vv[g, lo:hi]
            x = (K @ q[t, h].astype(np.float64)) * scale
            m = x.max()
            p = np.exp(x - m)
            lse[t, h] = m + math.log(p.sum())
            p /= p.sum()
            out[t, h], mass[t, h] = p @ V, p @ np.abs(V)
            reach[t, h] = (np.abs(K) @ np.abs(q[t, h].astype(np.float64))).max() * scale
            peak[t, h], keys[t, h] = (p * vs[g, lo:hi]).max(), hi - lo
    return out, lse, (mass, reach, peak, keys)
