"""Measured cases of the key/value cache operators and of cross attention.

    append   cache_append          new K and V rows into a paged cache, bf16 or quantised to E4M3
    read     cache_read            a batch's rows of a paged cache back into [B, Hkv, N, D] bf16
    decode   forward_decode        attention of the last T tokens of each sequence over its cache
    shared   forward_shared_prefix the same for a batch whose sequences all start with one prefix
    cross    forward_cross,        attention to keys of another length, padded to the batch's
             backward_cross        longest, and its gradients

The cache is [num_pages, Hkv, page, D]; position p of sequence b lies in page block_table[b, p // page] at row
p % page.  An E4M3 cache holds code * 2^e with one e for each token and head (E8M0, [num_pages, Hkv, page]): the
least e >= -120 with amax <= 448 * 2^e; a row that is not finite has the E8M0 NaN, and codes 0.
"""
import math
import random

import torch

own = False

_NEG = float("-inf")
_F8, _E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def listed():
    return [
        # one new token of each sequence of a serving batch: latency counts
        {"name": "append-token-e4m3", "op": "append", "B": 128, "Hkv": 8, "T": 1, "D": 128, "N": 900, "page": 64, "f8": True, "ragged": True},
        # prompts of different lengths just computed, written behind what the cache holds
        {"name": "append-prompt-e4m3", "op": "append", "B": 4, "Hkv": 8, "T": 4096, "D": 128, "N": 100, "page": 64, "f8": True, "ragged": True},
        # a short bf16 cache handed back to the prompt's attention
        {"name": "read-short-bf16", "op": "read", "B": 1, "Hkv": 4, "N": 1000, "D": 64, "page": 16, "f8": False, "ragged": False},
        # a batch's quantised prefixes read back before a second prompt is computed on them
        {"name": "read-batch-e4m3", "op": "read", "B": 16, "Hkv": 8, "N": 4096, "D": 128, "page": 64, "f8": True, "ragged": True},
        # one user's short dialogue: a single token, latency counts
        {"name": "decode-one-short", "op": "decode", "B": 1, "Hq": 32, "Hkv": 8, "T": 1, "D": 128, "N": 500, "page": 16, "f8": False, "ragged": False},
        # a serving batch of uneven lengths on a quantised cache
        {"name": "decode-batch-e4m3", "op": "decode", "B": 64, "Hq": 32, "Hkv": 8, "T": 1, "D": 128, "N": 8192, "page": 64, "f8": True, "ragged": True},
        # few long documents, four drafted tokens to verify at once
        {"name": "decode-long-drafted", "op": "decode", "B": 3, "Hq": 32, "Hkv": 8, "T": 4, "D": 128, "N": 100001, "page": 64, "f8": False, "ragged": True},
        # a few answers sampled from one prompt
        {"name": "shared-few-bf16", "op": "shared", "B": 6, "Hq": 16, "Hkv": 16, "T": 2, "D": 64, "P": 1000, "N": 200, "page": 16, "f8": False, "ragged": True},
        # a large batch behind one long instruction
        {"name": "shared-many-e4m3", "op": "shared", "B": 128, "Hq": 32, "Hkv": 8, "T": 1, "D": 128, "P": 16384, "N": 256, "page": 64, "f8": True, "ragged": True},
        # single tokens of a decoder attending to encoded inputs of different lengths
        {"name": "cross-token", "op": "cross", "B": 16, "Hq": 16, "Hkv": 16, "T": 1, "D": 64, "N": 1500, "ragged": True, "grad": False},
        # a decoder's whole prompt against encoded inputs
        {"name": "cross-prompt", "op": "cross", "B": 8, "Hq": 16, "Hkv": 16, "T": 500, "D": 64, "N": 1500, "ragged": True, "grad": False},
        # a training step of an encoder-decoder: forward and gradients, shared KV heads
        {"name": "cross-train", "op": "cross", "B": 4, "Hq": 32, "Hkv": 8, "T": 2048, "D": 128, "N": 4096, "ragged": True, "grad": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "decode", "shared", "cross"])
    c = {"op": op, "D": rng.choice([32, 64, 96, 128]), "ragged": rng.random() < 0.7}
    hkv = rng.choice([1, 2, 4, 5, 8, 16])
    group = rng.choice([1, 2, 3, 4, 7, 8])
    if op != "cross":
        c.update(Hkv=hkv, page=rng.choice([16, 32, 48, 64, 128, 256]), f8=rng.random() < 0.6)
    if op == "append":
        T = _log(rng, 1, 4000)
        c.update(T=T, N=_log(rng, 1, 2000), B=min(_log(rng, 1, 200), max(1, 16000 // T)))
    elif op == "read":
        N = _log(rng, 1, 20000)
        c.update(N=N, B=min(_log(rng, 1, 64), max(1, 64000 // N)))
    elif op == "decode":
        N = _log(rng, 1, 100000)
        c.update(N=N, T=rng.choice([1, 1, 1, 2, 5, 8]), Hq=hkv * group, B=min(_log(rng, 1, 128), max(1, 300000 // N)))
    elif op == "shared":
        P, B = _log(rng, 1, 16000), _log(rng, 1, 120)
        c.update(P=P, B=B, N=_log(rng, 1, 400), T=rng.choice([1, 1, 2, 4]), Hq=hkv * group)
        while c["B"] * c["Hq"] * c["T"] > 4000:
            c["B"] = max(1, c["B"] // 2)
            if c["B"] == 1:
                break
    else:
        T, N, B = _log(rng, 1, 2000), _log(rng, 1, 4000), _log(rng, 1, 24)
        c.update(T=T, N=N, Hkv=hkv, Hq=hkv * group, grad=T > 16 and rng.random() < 0.6)
        c["B"] = max(1, min(B, int(8e8 / (T * N * c["Hq"]))))
    return c


# ---------------------------------------------------------------- sizes

def _lens(c, n):
    """The batch's lengths, up to n: a ramp whose first is empty where there are enough, or all n."""
    B = c["B"]
    if not c["ragged"] or B == 1:
        return [n] * B
    out = [max(1, n * (i + 1) // B) for i in range(B)]
    if B >= 4:
        out[0] = 0
    return out


def _pages(c, n):
    return -(-n // c["page"])


def work(c):
    D, op = c["D"], c["op"]
    if op == "cross":
        rows, keys = c["B"] * c["Hq"] * c["T"], sum(_lens(c, c["N"])) * c["Hkv"]
        pairs = sum(_lens(c, c["N"])) * c["Hq"] * c["T"]
        if not c["grad"]:
            return {"bytes": rows * (4 * D + 4) + keys * 4 * D, "flops": 4 * pairs * D}
        # forward: q, k, v in, o and lse out; backward: q, k, v, o, lse, do in, dq, dk, dv out
        return {"bytes": rows * (4 * D + 4 + 8 * D + 4) + keys * (4 * D + 8 * D), "flops": 14 * pairs * D}
    row = 2 * (D + 1) if c["f8"] else 4 * D  # K and V of one token and head in the cache
    if op == "append":
        rows = sum(_lens(c, c["T"])) * c["Hkv"]
        return {"bytes": rows * (4 * D + row), "flops": 0}
    if op == "read":
        rows = sum(_lens(c, c["N"])) * c["Hkv"]
        return {"bytes": rows * row + c["B"] * c["Hkv"] * c["N"] * 4 * D, "flops": 0}
    keys, q = sum(_lens(c, c["N"])), c["B"] * c["Hq"] * c["T"]
    flops = 4 * D * c["Hq"] * c["T"] * keys
    if op == "shared":
        flops += 4 * D * q * c["P"]
        keys += c["P"]
    return {"bytes": keys * c["Hkv"] * row + q * (4 * D + 4), "flops": flops}


# ---------------------------------------------------------------- inputs

def _pow2(e):
    """2^e in fp32 for whole e in [-126, 127], exactly."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantise(x):
    """Rows of x (fp32, last axis) as (E4M3 codes, exponents): x ~ code * 2^e."""
    finite = torch.isfinite(x).all(-1)
    x = torch.where(finite[..., None], x, 0.0)
    amax = x.abs().amax(-1)
    m, k = torch.frexp(amax)  # amax = m 2^k, m in [1/2, 1): 448 = 7/8 2^9
    e = (k - 9 + (m > 0.875)).clamp(min=-120)
    e = torch.where(amax > 0, e, torch.full_like(e, -120))
    y = x * _pow2(-e)[..., None]
    top = torch.where(e >= 120, 240.0, 448.0)[..., None]  # 256 * 2^120 is infinite in bf16
    return torch.maximum(torch.minimum(y, top), -top).to(_F8), torch.where(finite, e, torch.full_like(e, 128))


def _e8(e):
    return (e + 127).to(torch.uint8).view(_E8)


def _rows(g, shape):
    """Keys or values as projections give them: channels of different spread."""
    D = shape[-1]
    spread = torch.exp(0.5 * torch.randn(D, generator=g, device="cuda"))
    return (torch.randn(shape, generator=g, device="cuda") * spread).to(torch.bfloat16)


def _cache(c, g, num_pages):
    shape = (num_pages, c["Hkv"], c["page"], c["D"])
    s = {}
    for name in ("k", "v"):
        x = _rows(g, shape)
        s[name + "_cache"], s[name + "_scale"] = x, None
        if c["f8"]:
            codes, e = _quantise(x.float())
            s[name + "_cache"], s[name + "_scale"] = codes, _e8(e)
    return s


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    B, D, op = c["B"], c["D"], c["op"]
    s = {"op": op, "case": c}
    if op == "cross":
        lens = _lens(c, c["N"])
        rng.shuffle(lens)
        s["k_lens"] = _ints(lens)
        s["q"] = torch.randn((B, c["Hq"], c["T"], D), generator=g, device="cuda").to(torch.bfloat16)
        s["k"], s["v"] = (_rows(g, (B, c["Hkv"], c["N"], D)) for _ in range(2))
        s["grad"] = c["grad"]
        if c["grad"]:
            s["dout"] = torch.randn((B, c["Hq"], c["T"], D), generator=g, device="cuda").to(torch.bfloat16)
        return s
    held = _lens({**c, "ragged": c["ragged"] and op != "append"}, c["N"])  # tokens in the cache before the call
    rng.shuffle(held)
    if op == "append":
        held = [rng.randrange(c["N"] + 1) for _ in range(B)]
    per = _pages(c, c["N"] + (c["T"] if op == "append" else 0))
    shared = _pages(c, c["P"]) if op == "shared" else 0
    ids = torch.randperm(B * per + shared, generator=g, device="cuda").to(torch.int32)
    s.update(_cache(c, g, B * per + shared))
    s["block_table"] = ids[: B * per].view(B, per).contiguous()
    s["lens"] = _ints(held)
    if op == "append":
        new = _lens(c, c["T"])
        rng.shuffle(new)
        s["new_lens"] = _ints(new)
        s["k"], s["v"] = (_rows(g, (B, c["Hkv"], c["T"], D)) for _ in range(2))
    elif op == "read":
        s["N"] = c["N"]
    else:
        s["q"] = torch.randn((B, c["Hq"], c["T"], D), generator=g, device="cuda").to(torch.bfloat16)
    if op == "shared":
        s["prefix_table"] = ids[B * per :].contiguous()
        s["prefix_len"] = c["P"]
    return s


# ---------------------------------------------------------------- plain forms

def _written(cache, rows, new, keep):
    """The cache's rows (flat index) replaced by `new` where keep is set; in place."""
    bits = {1: torch.uint8, 2: torch.int16}[cache.element_size()]
    flat = cache.view(bits).view(-1, cache.shape[-1]) if cache.dim() == 4 else cache.view(bits).view(-1)
    new = new.view(bits)
    flat[rows] = torch.where(keep if new.dim() == keep.dim() else keep[..., None], new, flat[rows])
    return cache


def _plain_append(s):
    k = s["k"]
    B, H, T, _ = k.shape
    page = s["k_cache"].shape[2]
    t = torch.arange(T, device=k.device)
    at = s["lens"][:, None].long() + t                                   # [B, T]
    ids = torch.gather(s["block_table"].long(), 1, at // page)
    rows = (ids[:, None] * H + torch.arange(H, device=k.device)[:, None]) * page + (at % page)[:, None]  # [B, H, T]
    keep = (t < s["new_lens"][:, None])[:, None].expand(B, H, T)
    out = {}
    for name in ("k", "v"):
        x = s[name]
        if s[name + "_scale"] is not None:
            x, e = _quantise(x.float())
            out[name + "_scale"] = _written(s[name + "_scale"], rows, _e8(e), keep)
        out[name + "_cache"] = _written(s[name + "_cache"], rows, x, keep)
    return out


def _gathered(cache, scale, table, n):
    """Positions [0, n) of each table row, fp32 [B, Hkv, n, D]."""
    x = cache[table.long()].float()                                      # [B, pages, Hkv, page, D]
    if scale is not None:
        x = x * scale[table.long()].float()[..., None]
    B, P, H, page, D = x.shape
    return x.transpose(1, 2).reshape(B, H, P * page, D)[:, :, :n]


def _plain_read(s):
    n = s["N"]
    seen = torch.arange(n, device="cuda") < s["lens"][:, None]           # [B, n]
    return [torch.where(seen[:, None, :, None], _gathered(s[x + "_cache"], s[x + "_scale"], s["block_table"], n), 0.0)
            .to(torch.bfloat16) for x in ("k", "v")]


def _softmax_v(q, k, v, seen):
    """q [B, Hkv, R, D], k, v [B, Hkv, n, D], seen broadcastable to [B, Hkv, R, n]: o, lse in fp32, empty rows 0, -inf."""
    any_row = seen.any(-2, keepdim=True).transpose(-1, -2)               # keys that no row sees may hold anything
    k, v = torch.where(any_row, k, 0.0), torch.where(any_row, v, 0.0)
    s = torch.where(seen, q @ k.transpose(-1, -2) / math.sqrt(q.shape[-1]), _NEG)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == _NEG, 0.0, m)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total > 0, total, 1.0)
    return o, (m + torch.log(total))[..., 0], p / torch.where(total > 0, total, 1.0)


def _causal_tail(lens, T, n, group):
    """[B, 1, group * T, n]: query t of sequence b stands at position lens[b] - T + t."""
    last = lens[:, None].long() - T + torch.arange(T, device=lens.device)
    return (torch.arange(n, device=lens.device) <= last[..., None])[:, None].repeat(1, 1, group, 1)


def _plain_attend(s):
    q = s["q"]
    B, Hq, T, D = q.shape
    n, Hkv = s["block_table"].shape[1] * s["k_cache"].shape[2], s["k_cache"].shape[1]
    group = Hq // Hkv
    k, v = (_gathered(s[x + "_cache"], s[x + "_scale"], s["block_table"], n) for x in ("k", "v"))
    seen = _causal_tail(s["lens"], T, n, group)
    if s["op"] == "shared":
        P = s["prefix_len"]
        pk, pv = (_gathered(s[x + "_cache"], s[x + "_scale"], s["prefix_table"][None], P) for x in ("k", "v"))
        k, v = (torch.cat([a.expand(B, -1, -1, -1), b], 2) for a, b in ((pk, k), (pv, v)))
        seen = torch.cat([torch.ones((B, 1, group * T, P), dtype=torch.bool, device=q.device), seen], 3)
    o, lse, _ = _softmax_v(q.float().view(B, Hkv, group * T, D), k, v, seen)
    return o.to(torch.bfloat16).view(B, Hq, T, D), lse.view(B, Hq, T)


def _plain_cross(s):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    B, Hq, T, D = q.shape
    Hkv, n = k.shape[1], k.shape[2]
    rows = (B, Hkv, Hq // Hkv * T, D)
    q = q.view(rows)
    seen = (torch.arange(n, device=q.device) < s["k_lens"][:, None])[:, None, None]
    o, lse, p = _softmax_v(q, k, v, seen)
    o = o.to(torch.bfloat16)
    out = [o.view(B, Hq, T, D), lse.view(B, Hq, T)]
    if s["grad"]:
        do = s["dout"].float().view(rows)
        live = seen.transpose(-1, -2)
        k, v = torch.where(live, k, 0.0), torch.where(live, v, 0.0)
        ds = p * (do @ v.transpose(-1, -2) - (do * o.float()).sum(-1, keepdim=True)) / math.sqrt(D)
        out += [(ds @ k).view(B, Hq, T, D), ds.transpose(-1, -2) @ q, p.transpose(-1, -2) @ do]
        out[2:] = [x.to(torch.bfloat16) for x in out[2:]]
    return out


def run(s):
    op = s["op"]
    if own:
        import tiled_attention_forward_03_b200 as attn

        if op == "cross":
            o, lse = attn.forward_cross(s["q"], s["k"], s["v"], k_lens=s["k_lens"])
            if not s["grad"]:
                return [o, lse]
            return [o, lse, *attn.backward_cross(s["q"], s["k"], s["v"], o, lse, s["dout"], k_lens=s["k_lens"])]
        cache = {"k_scale": s["k_scale"], "v_scale": s["v_scale"]}
        if op == "append":
            attn.cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"], s["lens"],
                              new_lens=s["new_lens"], **cache)
            return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale") if s[n] is not None}
        if op == "read":
            return list(attn.cache_read(s["k_cache"], s["v_cache"], s["block_table"], s["lens"], s["N"], **cache))
        if op == "decode":
            return attn.forward_decode(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["lens"], **cache)
        return attn.forward_shared_prefix(s["q"], s["k_cache"], s["v_cache"], s["prefix_table"], s["prefix_len"],
                                          s["block_table"], s["lens"], **cache)
    if op == "append":
        return _plain_append(s)
    if op == "read":
        return _plain_read(s)
    return _plain_cross(s) if op == "cross" else _plain_attend(s)


# ---------------------------------------------------------------- the definitions in 64 bits, sequence by sequence

def _power64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _codes64(x):
    """The value nearest to each x on E4M3's grid (ties to even), |x| <= 448."""
    binade = (x.abs().clamp(min=2.0 ** -6).view(torch.int64) >> 52) - 1023
    step = _power64(binade - 3)
    return torch.round(x / step) * step


def _least_exponent64(top):
    """The least e >= -120 with top <= 448 * 2^e."""
    e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -200) / 448)).clamp(min=-120)
    e = torch.where(top > 448 * _power64(e), e + 1, e)  # the logarithm is rounded
    return torch.where((e > -120) & (top <= 448 * _power64(e - 1)), e - 1, e)


def _positions(s, name, b_table, n):
    """Rows of positions [0, n) behind one table row, fp64 [Hkv, n, D]."""
    cache, scale = s[name + "_cache"], s[name + "_scale"]
    page = cache.shape[2]
    at = torch.arange(n, device="cuda")
    ids = b_table.long()[at // page]
    x = cache.view(torch.uint8)[ids, :, at % page].view(cache.dtype) if scale is not None else cache[ids, :, at % page]
    x = x.double()
    if scale is not None:
        x = x * _power64(scale.view(torch.uint8)[ids, :, at % page].long() - 127)[..., None]
    return x.transpose(0, 1)


def _attend64(q, k, v, lim):
    """One sequence: q [Hq, T, D] (64 bits), k, v [Hkv, n, D], query t sees keys below lim[t]."""
    Hq, T, D = q.shape
    Hkv, n = k.shape[0], k.shape[1]
    o = torch.zeros((Hq, T, D), dtype=torch.float64, device=q.device)
    lse = torch.full((Hq, T), _NEG, dtype=torch.float64, device=q.device)
    ps = {}
    for h in range(Hq):
        if n == 0:
            continue
        x = (q[h] @ k[h * Hkv // Hq].T) * D ** -0.5
        x = x.masked_fill(torch.arange(n, device=q.device)[None] >= lim[:, None], _NEG)
        live = lim > 0
        lse[h, live] = torch.logsumexp(x[live], -1)
        ps[h] = torch.zeros_like(x)
        ps[h][live] = torch.exp(x[live] - lse[h, live][:, None])
        o[h] = ps[h] @ v[h * Hkv // Hq]
    return o, lse, ps


def exact(c, seed):
    s = prepare(c, seed)
    B, op = c["B"], c["op"]
    if op == "append":
        out = {}
        held, new, table = s["lens"].tolist(), s["new_lens"].tolist(), s["block_table"].long()
        for name in ("k", "v"):
            cache = s[name + "_cache"].double()
            scale = _power64(s[name + "_scale"].view(torch.uint8).long() - 127) if c["f8"] else None
            for b in range(B):
                at = held[b] + torch.arange(new[b], device="cuda")
                ids, x = table[b][at // c["page"]], s[name][b, :, : new[b]].double().transpose(0, 1)
                if c["f8"]:
                    e = _least_exponent64(x.abs().amax(-1))
                    scale[ids, :, at % c["page"]] = _power64(e)
                    x = _codes64(x / _power64(e)[..., None])
                cache[ids, :, at % c["page"]] = x
            out[name + "_cache"] = cache
            if c["f8"]:
                out[name + "_scale"] = scale
        return out
    if op == "read":
        out = [torch.zeros((B, c["Hkv"], c["N"], c["D"]), dtype=torch.float64, device="cuda") for _ in range(2)]
        for b, n in enumerate(s["lens"].tolist()):
            for x, name in zip(out, ("k", "v")):
                x[b, :, :n] = _positions(s, name, s["block_table"][b], n)
        return out
    T = c["T"]
    o = torch.empty((B, c["Hq"], T, c["D"]), dtype=torch.float64, device="cuda")
    lse = torch.empty((B, c["Hq"], T), dtype=torch.float64, device="cuda")
    if op == "cross":
        grads = [torch.zeros(s[x].shape, dtype=torch.float64, device="cuda") for x in "qkv"] if c["grad"] else []
        for b, n in enumerate(s["k_lens"].tolist()):
            q, k, v = s["q"][b].double(), s["k"][b, :, :n].double(), s["v"][b, :, :n].double()
            o[b], lse[b], ps = _attend64(q, k, v, torch.full((T,), n, device="cuda"))
            for h in ps if c["grad"] else ():
                g = h * c["Hkv"] // c["Hq"]
                do = s["dout"][b, h].double()
                ds = ps[h] * (do @ v[g].T - (do * o[b, h]).sum(-1, keepdim=True)) * c["D"] ** -0.5
                grads[0][b, h] = ds @ k[g]
                grads[1][b, g, :n] += ds.T @ q[h]
                grads[2][b, g, :n] += ps[h].T @ do
        return [o, lse, *grads]
    P = s.get("prefix_len", 0)
    first = {x: _positions(s, x, s["prefix_table"], P) for x in "kv"} if P else {}
    for b, n in enumerate(s["lens"].tolist()):
        k, v = (_positions(s, x, s["block_table"][b], n) for x in "kv")
        if P:
            k, v = torch.cat([first["k"], k], 1), torch.cat([first["v"], v], 1)
        lim = P + (n - T + 1 + torch.arange(T, device="cuda")).clamp(min=0)
        o[b], lse[b], _ = _attend64(s["q"][b].double(), k, v, lim)
    return o, lse
