"""Measured cases of the operators around a paged 8-bit key/value cache.

Three operators that a decode or prompt step of a quantized model runs between
its quantized projections:

* ``rope``     rotary positions of queries or keys,
* ``append``   rotate new keys, quantize keys and values to e4m3 with one
               power-of-two scale per block of 16 tokens and head, store them in
               a paged cache, and rotate the queries of the same tokens,
* ``attend``   causal attention of the new tokens over that cache.

With ``own`` false the operators run in plain torch operations in 32 bits; with
``own`` true they are the framework's calls.

A cache is a dict: k_codes, v_codes float8_e4m3fn [pages, heads, page, dim];
k_scales, v_scales float32 [pages, heads, page / 16], powers of two.
``seq_lens[b]`` counts the tokens of sequence b in the cache, the new ones
included; the new tokens of sequence b are rows cu[b] .. cu[b+1]-1 of q, k and v
(without cu: row b, one token each) and take the last positions.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16            # tokens that share a scale
E_MIN, E_MAX = -40, 40
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _rope(name, tokens, heads, dim, rot, layout, src, dst, span, scaling="none", inverse=False):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "dim": dim, "rot": rot, "layout": layout,
            "src": src, "dst": dst, "span": span, "scaling": scaling, "inverse": inverse}


def _append(name, seqs, new_lo, new_hi, past_lo, past_hi, hq, hkv, dim, page, layout, src, dst, rot, single):
    return {"name": name, "op": "append", "seqs": seqs, "new_lo": new_lo, "new_hi": new_hi, "past_lo": past_lo,
            "past_hi": past_hi, "hq": hq, "hkv": hkv, "dim": dim, "page": page, "layout": layout, "src": src,
            "dst": dst, "rot": rot, "single": single}


def _attend(name, seqs, new_lo, new_hi, past_lo, past_hi, hq, hkv, dim, page, dtype, single, window=0, lse=False):
    return {"name": name, "op": "attend", "seqs": seqs, "new_lo": new_lo, "new_hi": new_hi, "past_lo": past_lo,
            "past_hi": past_hi, "hq": hq, "hkv": hkv, "dim": dim, "page": page, "dtype": dtype, "single": single,
            "window": window, "lse": lse}


def listed():
    return [
        # a decode step's queries, as the quantized projection leaves them (32-bit), far into a long context
        _rope("rope decode", 64, 32, 128, 128, "half", "f32", "f16", 131072, scaling="yarn"),
        # a long prompt's queries, part of the head rotated, neighbouring pairs
        _rope("rope prompt", 16384, 32, 128, 64, "interleaved", "bf16", "bf16", 32768, scaling="linear"),
        # one user, one token: latency is all
        _append("append one token", 1, 1, 1, 777, 777, 32, 8, 128, 64, "half", "f32", "f16", 128, True),
        # a large decode batch
        _append("append decode batch", 256, 1, 1, 1, 500, 64, 8, 128, 16, "half", "f32", "f16", 128, True),
        # prompts of several users in one ragged step, some of them continued in the middle of a block
        _append("append prompts", 7, 500, 4001, 0, 301, 32, 8, 128, 64, "interleaved", "bf16", "bf16", 128, False),
        # one user, short context: latency is all
        _attend("attend one short", 1, 1, 1, 516, 516, 32, 8, 128, 16, "f16", True),
        # one user, a whole book of context
        _attend("attend one long", 1, 1, 1, 131071, 131071, 64, 8, 128, 64, "f16", True),
        # a ragged decode batch
        _attend("attend decode batch", 64, 1, 1, 0, 8191, 64, 8, 128, 32, "bf16", True),
        # every query head with keys of its own, small heads, a sliding window
        _attend("attend own heads", 24, 1, 1, 200, 4099, 32, 32, 64, 16, "f16", True, window=2048),
        # drafts of a few tokens checked at once
        _attend("attend drafts", 8, 3, 6, 2000, 16001, 32, 8, 128, 64, "bf16", False, lse=True),
        # chunks of several prompts over what is already cached
        _attend("attend chunks", 4, 17, 2048, 0, 6001, 64, 8, 128, 64, "f16", False),
        # one whole prompt
        _attend("attend prompt", 1, 8192, 8192, 0, 0, 32, 8, 128, 128, "bf16", False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "attend"])
    layout = rng.choice(["half", "interleaved"])
    dim = rng.choice([64, 128, 128])
    if op == "rope":
        tokens = _log(rng, 1, 16384)
        c = _rope("", tokens, rng.choice([1, 8, 32, 40]), dim, rng.choice([dim, dim // 2, dim // 4]), layout,
                  rng.choice(["f32", "f16", "bf16"]), rng.choice(["f16", "bf16"]), _log(rng, 100, 131072),
                  rng.choice(["none", "linear", "yarn"]), rng.random() < 0.25)
        while c["tokens"] * c["heads"] * c["dim"] > 16384 * 32 * 128:
            c["tokens"] //= 2
    else:
        hkv = rng.choice([1, 2, 4, 8, 8])
        hq = hkv * rng.choice([1, 2, 4, 5, 7, 8])
        page = rng.choice([16, 32, 64, 128])
        single = rng.random() < 0.5
        if single:
            seqs = _log(rng, 1, 256)
            new_lo = new_hi = 1
            past_hi = _log(rng, 3, 500 if op == "append" else 131071)
        else:
            seqs = rng.randint(1, 8)
            new_hi = _log(rng, 2, 4001 if op == "append" else 2048)
            new_lo = rng.randint(1, new_hi)
            past_hi = _log(rng, 1, 301 if op == "append" else 8191)
        past_lo = rng.randint(0, past_hi)
        if op == "append":
            c = _append("", seqs, new_lo, new_hi, past_lo, past_hi, hq, hkv, dim, page, layout,
                        rng.choice(["f32", "f16", "bf16"]), rng.choice(["f16", "bf16"]), rng.choice([dim, dim // 2]),
                        single)
        else:
            c = _attend("", seqs, new_lo, new_hi, past_lo, past_hi, hq, hkv, dim, page, rng.choice(["f16", "bf16"]),
                        single, rng.choice([0, 0, 0, _log(rng, 1, 4096)]), rng.random() < 0.3)
        # no more bytes, cached keys and (query, key) pairs than the largest listed cases have
        keys = 64 * 8192 * 8 * 128
        while c["seqs"] > 1 and (work(c)["bytes"] > keys or c["seqs"] * (c["new_hi"] + c["past_hi"]) * c["hkv"] * c["dim"] > keys):
            c["seqs"] -= 1
        while op == "attend" and c["seqs"] * c["new_hi"] * (c["new_hi"] + c["past_hi"]) * c["hq"] > 8192 * 8192 * 16:
            c["seqs"], c["new_hi"] = max(1, c["seqs"] // 2), max(2 - c["single"], c["new_hi"] // 2)
            c["new_lo"] = min(c["new_lo"], c["new_hi"])
    del c["name"]
    return c


def _spread(case):
    """Tokens before and new tokens of each sequence: spread over the case's ranges, the same for every seed."""
    n = case["seqs"]
    at = [(i * 0.6180339887498949 + (0.0 if n == 1 else 0.5)) % 1.0 for i in range(n)]
    past = [case["past_lo"] + int(round(a * (case["past_hi"] - case["past_lo"]))) for a in at]
    new = [case["new_lo"] + int(round(((a * 7) % 1.0) * (case["new_hi"] - case["new_lo"]))) for a in at]
    return past, new


def _inv_freq(rot, scaling, span):
    """Angles per position (float64 [rot / 2]) and the factor on cosine and sine."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / rot)
    if scaling == "none":
        return f, 1.0
    if scaling == "linear":
        return f / 4.0, 1.0
    # "yarn": factor 8 over an original context of span / 8; fast pairs as they were, slow ones interpolated
    factor, old = 8.0, max(1.0, span / 8.0)
    edge = lambda turns: rot * math.log(old / (turns * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
    lo, hi = max(math.floor(edge(32.0)), 0), min(math.ceil(edge(1.0)), rot - 1)
    ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
    return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0


def _table(n_pos, rot, scaling, span, device):
    f, m = _inv_freq(rot, scaling, span)
    t = torch.arange(n_pos, dtype=torch.float64, device=device)[:, None] * f.to(device)[None, :]
    return (torch.stack([t.cos(), t.sin()], dim=-1) * m).float().contiguous()


def _tokens_of(case, seed, past, new, device):
    """seq_lens, cu (None for single tokens) and page table of a step; pages in an order of the seed's."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    P, n = case["page"], case["seqs"]
    lens = [p + q for p, q in zip(past, new)]
    width = max(-(-x // P) for x in lens)
    pages = torch.zeros((n, width), dtype=torch.int32)
    total = sum(-(-x // P) for x in lens)
    order, at = torch.randperm(total, generator=g, dtype=torch.int32), 0
    for b, x in enumerate(lens):
        k = -(-x // P)
        pages[b, :k] = order[at:at + k]
        at += k
    seq_lens = torch.tensor(lens, dtype=torch.int32, device=device)
    cu = None
    if not case["single"]:
        cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=device)
    return seq_lens, cu, pages.to(device), total


def _new_cache(n_pages, heads, page, dim, g, device):
    """A filled cache: keys whose channels differ in size, as models' keys do; scales as an append leaves them."""
    c = {}
    for w in ("k", "v"):
        x = torch.randn((n_pages * heads * page // BLOCK, BLOCK, dim), generator=g, device=device)
        if w == "k":
            x *= torch.exp(0.8 * torch.randn(dim, generator=g, device=device))
        x *= torch.exp2(torch.randint(-1, 2, (x.shape[0], 1, 1), generator=g, device=device).float())
        e = _exponent(x.abs().amax((1, 2)))
        c[w + "_codes"] = (x * _pow2(-e)[:, None, None]).to(torch.float8_e4m3fn).view(n_pages, heads, page, dim)
        c[w + "_scales"] = _pow2(e).view(n_pages, heads, page // BLOCK)
        del x
    return c


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    s = {"case": case}
    if case["op"] == "rope":
        T, H, D = case["tokens"], case["heads"], case["dim"]
        s["table"] = _table(case["span"], case["rot"], case["scaling"], case["span"], dev)
        s["positions"] = torch.randint(0, case["span"], (T,), generator=g, device=dev, dtype=torch.int32)
        s["x"] = torch.randn((T, H, D), generator=g, device=dev).to(TYPES[case["src"]])
        return s
    past, new = _spread(case)
    T, hq, hkv, D = sum(new), case["hq"], case["hkv"], case["dim"]
    s["seq_lens"], s["cu"], s["pages"], n_pages = _tokens_of(case, seed, past, new, dev)
    s["max_new"] = max(new)
    s["cache"] = _new_cache(n_pages, hkv, case["page"], D, g, dev)
    if case["op"] == "append":
        s["table"] = _table(max(p + q for p, q in zip(past, new)), case["rot"], "none", 1, dev)
        # one fused projection: queries, keys and values side by side
        qkv = torch.randn((T, (hq + 2 * hkv) * D), generator=g, device=dev)
        qkv = qkv.to(TYPES[case["src"]]).view(T, hq + 2 * hkv, D)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        s["q"] = torch.randn((T, hq, D), generator=g, device=dev).to(TYPES[case["dtype"]])
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    c = state["case"]
    if own:
        import awq_activation_aware_b200 as awq

        if c["op"] == "rope":
            return awq.rope(state["x"], state["positions"], state["table"], layout=c["layout"], inverse=c["inverse"],
                            dtype=TYPES[c["dst"]])
        if c["op"] == "append":
            q = awq.kv_append(state["cache"], state["k"], state["v"], state["seq_lens"], state["pages"],
                              cu_tokens=state["cu"], table=state["table"], layout=c["layout"], q=state["q"],
                              q_dtype=TYPES[c["dst"]])
            return {"q": q, **state["cache"]}
        return awq.kv_attention(state["cache"], state["q"], state["seq_lens"], state["pages"], cu_tokens=state["cu"],
                                max_tokens=state["max_new"], window=c["window"], return_lse=c["lse"])
    if c["op"] == "rope":
        cs = state["table"][state["positions"].long()]
        return _rotate(state["x"].float(), cs, c["layout"], c["inverse"]).to(TYPES[c["dst"]])
    if c["op"] == "append":
        return _plain_append(state)
    return _plain_attend(state)


def _pow2(e):
    """2^e in 32 bits, exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponent(amax):
    """The least e in [E_MIN, E_MAX] with amax <= 448 * 2^e."""
    m, x = torch.frexp(amax)
    e = x - 9 + (m > 0.875).to(torch.int32)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)


def _rotate(x, cs, layout, inverse=False):
    """x [T, H, D] in 32 bits, cs [T, rot / 2, 2]."""
    half = cs.shape[1]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    s = -s if inverse else s
    head, rest = x[..., :2 * half], x[..., 2 * half:]
    if layout == "half":
        x1, x2 = head[..., :half], head[..., half:]
        return torch.cat([x1 * c - x2 * s, x2 * c + x1 * s, rest], dim=-1)
    x1, x2 = head[..., 0::2], head[..., 1::2]
    return torch.cat([torch.stack([x1 * c - x2 * s, x2 * c + x1 * s], dim=-1).flatten(-2), rest], dim=-1)


def _places(seq_lens, cu, T):
    """Sequence and position of every new token, and whether it is its sequence's first."""
    t = torch.arange(T, device=seq_lens.device)
    if cu is None:
        return t, seq_lens.long() - 1, torch.ones_like(t, dtype=torch.bool)
    b = torch.searchsorted(cu[1:].long(), t, right=True)
    first = cu.long()[b]
    return b, seq_lens.long()[b] - (cu.long()[b + 1] - first) + t - first, t == first


def _plain_append(s):
    c, cache, cu = s["case"], s["cache"], s["cu"]
    T, P = s["k"].shape[0], c["page"]
    n_pages, H, nb = cache["k_scales"].shape
    b, pos, first = _places(s["seq_lens"], cu, T)
    page, off = s["pages"][b, pos // P].long(), pos % P
    n_new = 1 if cu is None else (cu[1:] - cu[:-1]).long()[b]
    start = s["seq_lens"].long()[b] - n_new
    earlier = (pos // BLOCK) * BLOCK < start                      # the block holds tokens from before
    head = torch.arange(H, device=page.device)
    block = (page[:, None] * H + head) * nb + (off // BLOCK)[:, None]
    cs = s["table"][pos]
    lead = first.nonzero()[:, 0] if cu is not None else torch.arange(T, device=page.device)
    kept = torch.arange(BLOCK, device=page.device)[None, :] < (pos[lead] % BLOCK)[:, None]
    for w, y in (("k", _rotate(s["k"].float(), cs, c["layout"])), ("v", s["v"].float())):
        codes, scales = cache[w + "_codes"], cache[w + "_scales"].view(-1)
        fine = torch.isfinite(y)
        e_new = _exponent(torch.where(fine, y.abs(), torch.zeros_like(y)).amax(-1))
        e_old = torch.where(earlier[:, None], torch.frexp(scales[block])[1] - 1, torch.full_like(e_new, E_MIN))
        every = torch.full((n_pages * H * nb,), E_MIN, dtype=torch.int32, device=page.device)
        every.scatter_reduce_(0, block.flatten(), torch.maximum(e_new, e_old).flatten(), "amax")
        e = every[block]
        # the codes that were there, in the block's new scale
        rows = codes.view(n_pages * H * nb, BLOCK, -1)
        old = rows[block[lead]]
        again = (old.float() * _pow2(e_old[lead] - e[lead])[..., None, None]).to(torch.float8_e4m3fn)
        rows[block[lead]] = torch.where(kept[:, None, :, None], again.view(torch.uint8),
                                        old.view(torch.uint8)).view(torch.float8_e4m3fn)
        y = (y * _pow2(-e)[..., None]).clamp(-448.0, 448.0)
        y = torch.where(fine, y, torch.full_like(y, float("nan"))).to(torch.float8_e4m3fn)
        rows.view(torch.uint8)[block, (off % BLOCK)[:, None]] = y.view(torch.uint8)
        scales[block] = _pow2(e)
    return {"q": _rotate(s["q"].float(), cs, c["layout"]).to(TYPES[c["dst"]]), **cache}


def _plain_attend(s):
    c, cache, q, cu = s["case"], s["cache"], s["q"], s["cu"]
    T, hq, D = q.shape
    hkv, P, B = c["hkv"], c["page"], c["seqs"]
    b, pos, _ = _places(s["seq_lens"], cu, T)
    width = s["max_new"]
    row = torch.zeros_like(b) if cu is None else torch.arange(T, device=q.device) - cu.long()[b]
    qs = torch.zeros((B, width, hq, D), device=q.device)
    qs[b, row] = q.float()
    at = torch.full((B, width), -1, dtype=torch.long, device=q.device)
    at[b, row] = pos
    kv = {}
    for w in ("k", "v"):
        codes = cache[w + "_codes"][s["pages"].long()].float()                      # [B, pages, hkv, P, D]
        codes *= cache[w + "_scales"][s["pages"].long()].repeat_interleave(BLOCK, dim=-1)[..., None]
        kv[w] = codes.transpose(1, 2).flatten(2, 3)                                  # [B, hkv, S, D]
        del codes
    S = kv["k"].shape[2]
    key = torch.arange(S, device=q.device)
    seen = key[None, None, :] <= at[:, :, None]
    if c["window"]:
        seen &= key[None, None, :] > at[:, :, None] - c["window"]
    G = hq // hkv
    qs = qs.view(B, width, hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, hkv, G * width, D)
    x = torch.matmul(qs, kv["k"].transpose(-1, -2)).view(B, hkv, G, width, S)
    x *= 1.0 / math.sqrt(D)
    x.masked_fill_(~seen[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    x -= m
    x.exp_()
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x.view(B, hkv, G * width, S), kv["v"]).view(B, hkv, G, width, D)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    out = out.permute(0, 3, 1, 2, 4).reshape(B, width, hq, D)[b, row].to(q.dtype)
    if not c["lse"]:
        return out
    lse = (m + total.log())[..., 0].permute(0, 3, 1, 2).reshape(B, width, hq)[b, row]
    return out, lse


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    size = {"f16": 2, "bf16": 2, "f32": 4}
    D = case["dim"]
    if case["op"] == "rope":
        T = case["tokens"]
        rows = min(T, case["span"])
        return {"bytes": T * case["heads"] * D * (size[case["src"]] + size[case["dst"]]) + rows * case["rot"] * 4 + 4 * T,
                "flops": 3 * T * case["heads"] * case["rot"]}
    past, new = _spread(case)
    hq, hkv, P = case["hq"], case["hkv"], case["page"]
    T = sum(new)
    if case["op"] == "append":
        blocks = sum((p + n - 1) // BLOCK - p // BLOCK + 1 for p, n in zip(past, new))
        old = sum(1 for p in past if p % BLOCK)
        lens = sorted(set(x for p, n in zip(past, new) for x in range(p, p + n)))
        return {"bytes": T * D * ((hq + 2 * hkv) * size[case["src"]] + hq * size[case["dst"]] + 2 * hkv)
                + 8 * hkv * (blocks + old) + len(lens) * case["rot"] * 4 + 4 * len(new),
                "flops": T * (3 * case["rot"] * (hq + hkv) + 3 * D * 2 * hkv)}
    w = case["window"]
    keys = pairs = 0
    for p, n in zip(past, new):
        lo = max(0, p + 1 - w) if w else 0
        keys += p + n - lo
        pairs += sum(min(x + 1, w) for x in range(p, p + n)) if w else n * p + n * (n + 1) // 2
    return {"bytes": keys * hkv * 2 * (D + 4 / BLOCK) + T * hq * (4 * D + (4 if case["lse"] else 0)) + 4 * sum(
        -(-(p + n) // P) for p, n in zip(past, new)), "flops": 4 * D * hq * pairs}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def _turn64(x, pos, rot, scaling, span, layout, sign):
    """Rotation as a product of complex numbers, angles from the positions themselves."""
    f, m = _inv_freq(rot, scaling, span)
    angle = pos.double()[:, None] * f.to(x.device)[None, :]
    w = torch.polar(torch.full_like(angle, m), sign * angle)[:, None, :]
    y = x.double().clone()
    n = rot // 2
    if layout == "half":
        z = torch.complex(y[..., :n].contiguous(), y[..., n:rot].contiguous()) * w
        y[..., :n], y[..., n:rot] = z.real, z.imag
    else:
        z = torch.view_as_complex(y[..., :rot].contiguous().unflatten(-1, (n, 2))) * w
        y[..., :rot] = torch.view_as_real(z).flatten(-2)
    return y


def _e4m3_64(x):
    """The nearest value with 3 fraction bits and a least exponent of -6, ties to even, at most 448."""
    a = x.abs().clamp_max(448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3)
    return torch.sign(x) * torch.round(a / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _turn64(s["x"], s["positions"], case["rot"], case["scaling"], case["span"], case["layout"],
                       -1.0 if case["inverse"] else 1.0)
    past, new = _spread(case)
    P, D, hq, hkv = case["page"], case["dim"], case["hq"], case["hkv"]
    cache, pages = s["cache"], s["pages"].cpu().tolist()
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    if case["op"] == "append":
        if sum(new) > 30000:
            return None
        pos = torch.cat([torch.arange(p, p + n, device="cuda") for p, n in zip(past, new)])
        k = _turn64(s["k"], pos, case["rot"], "none", 1, case["layout"], 1.0)
        out = {"q": _turn64(s["q"], pos, case["rot"], "none", 1, case["layout"], 1.0)}
        for w, y in (("k", k), ("v", s["v"].double())):
            codes, scales = cache[w + "_codes"].double(), cache[w + "_scales"].double()
            for b, (p, n) in enumerate(zip(past, new)):
                for blk in range(p // BLOCK, (p + n - 1) // BLOCK + 1):
                    lo, hi = max(p, blk * BLOCK), min(p + n, (blk + 1) * BLOCK)
                    part = y[starts[b] + lo - p:starts[b] + hi - p].transpose(0, 1)           # [hkv, rows, D]
                    page, o = pages[b][blk * BLOCK // P], blk * BLOCK % P
                    need = torch.ceil(torch.log2(part.abs().amax((1, 2)) / 448.0)).clamp(E_MIN, E_MAX)
                    scale = torch.exp2(need)
                    if lo > blk * BLOCK:
                        was = scales[page, :, o // BLOCK]
                        scale = torch.maximum(scale, was)
                        rows = codes[page, :, o:o + lo - blk * BLOCK]
                        rows.copy_(_e4m3_64(rows * (was / scale)[:, None, None]))
                    codes[page, :, o + lo - blk * BLOCK:o + hi - blk * BLOCK] = _e4m3_64(part / scale[:, None, None])
                    scales[page, :, o // BLOCK] = scale
            out[w + "_codes"], out[w + "_scales"] = codes, scales
        return out
    out = torch.zeros((sum(new), hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((sum(new), hq), dtype=torch.float64, device="cuda")
    G = hq // hkv
    for b, (p, n) in enumerate(zip(past, new)):
        S = p + n
        ids = torch.tensor(pages[b][:-(-S // P)], device="cuda")
        i = torch.arange(p, S, device="cuda")[:, None]
        j = torch.arange(S, device="cuda")[None, :]
        hidden = j > i
        if case["window"]:
            hidden = hidden | (j <= i - case["window"])
        for h in range(hkv):
            k, v = ((cache[w + "_codes"][ids, h].double() * cache[w + "_scales"][ids, h].double()
                     .repeat_interleave(BLOCK, dim=-1)[..., None]).reshape(-1, D)[:S] for w in ("k", "v"))
            for a in range(h * G, (h + 1) * G):
                x = s["q"][starts[b]:starts[b + 1], a].double() @ k.T / math.sqrt(D)
                x.masked_fill_(hidden, float("-inf"))
                lse[starts[b]:starts[b + 1], a] = torch.logsumexp(x, -1)
                out[starts[b]:starts[b + 1], a] = torch.softmax(x, -1) @ v
    return (out, lse) if case["lse"] else out
