"""The serving and position operators of rational-softmax attention as measured work.

Three families, as a decoder layer runs them one after the other:
  norm_rope  the per-head normalisation of queries and keys with the position rotation of one or more axes, from
             the packed projection [B, N, (Hq + 2 Hkv) D]: forward (q, k and v ready for attention), backward (the
             gradient of the projection and of the norm parameters), and append (single tokens written straight
             into a key/value cache);
  decode     one query token per sequence against its own ragged cache and a prefix that the whole batch shares,
             adding each key's attention weight to a running total;
  evict      the cache cut down to its most attended entries and its last ones.

`own` selects between the plain form (elementary torch operations, 32-bit arithmetic, 64-bit angles) and the
framework's calls.  `exact` restates each operator in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# --------------------------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------------------------
def _norm_rope(name, kind, dtype, B, N, Hq, Hkv, D, norm, bias, sections, interleaved, start, capacity=0):
    c = {"kind": kind, "dtype": dtype, "B": B, "N": N, "Hq": Hq, "Hkv": Hkv, "D": D, "norm": norm, "bias": bias,
         "sections": ",".join(str(s) for s in sections), "interleaved": interleaved, "start": start}
    if capacity:
        c["capacity"] = capacity
    return dict(c, name=name) if name else c


def _decode(name, dtype, B, Hq, Hkv, D, capacity, prefix, sigma, tracked):
    c = {"kind": "decode", "dtype": dtype, "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "capacity": capacity,
         "prefix": prefix, "sigma": sigma, "tracked": tracked}
    return dict(c, name=name) if name else c


def _evict(name, dtype, B, Hkv, D, capacity, keep, recent, ragged):
    c = {"kind": "evict", "dtype": dtype, "B": B, "Hkv": Hkv, "D": D, "capacity": capacity, "keep": keep,
         "recent": recent, "ragged": ragged}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one layer of the 768-wide, 12-head example module on two short sequences: a launch-bound training step
        _norm_rope("norm_rope_fwd_b2n128h12d64", "fwd", "bf16", 2, 128, 12, 12, 64, "layer", True, (32,), False, 0),
        # video tokens (time, height, width) of a long context, grouped heads, root-mean-square norm
        _norm_rope("norm_rope_fwd_b4n8192h16kv8d128", "fwd", "bf16", 4, 8192, 16, 8, 128, "rms", False,
                   (16, 24, 24), True, 0),
        # training at the long-sequence attention shape, every head with its own keys: the gradient direction
        _norm_rope("norm_rope_bwd_b4n8192h16d128", "bwd", "bf16", 4, 8192, 16, 16, 128, "layer", True, (64,), False,
                   0),
        # a 32-bit training run with odd sizes, part of each head unrotated, far positions
        _norm_rope("norm_rope_bwd_fp32_b3n1001h6kv2d64", "bwd", "fp32", 3, 1001, 6, 2, 64, "layer", True, (8, 16),
                   False, 1000003),
        # one generated token for each of 64 sequences, written into their caches
        _norm_rope("append_b64h32kv8d128", "append", "bf16", 64, 1, 32, 8, 128, "rms", False, (64,), False, 5000,
                   capacity=256),
        # a single short conversation: latency
        _decode("decode_b1h16d128_c512", "bf16", 1, 16, 16, 128, 512, 0, 1.0, False),
        # a server's ordinary batch behind one long instruction, weights tracked for eviction
        _decode("decode_b32h32kv8d128_c1024_p8192", "bf16", 32, 32, 8, 128, 1024, 8192, 1.0, True),
        # a large batch, long own contexts and a very long shared document
        _decode("decode_b64h32kv8d128_c4096_p32768", "bf16", 64, 32, 8, 128, 4096, 32768, 1.0, True),
        # one long context, all query heads on one key head, wide scores (most weights exactly 0)
        _decode("decode_b2h24kv1d64_c65537", "bf16", 2, 24, 1, 64, 65537, 0, 3.0, False),
        # 32-bit parity runs at odd sizes
        _decode("decode_fp32_b5h12kv4d32_c1003_p777", "fp32", 5, 12, 4, 32, 1003, 777, 1.0, True),
        # long prompts compressed once before generation
        _evict("evict_b4kv8d128_c32768_to_2048", "bf16", 4, 8, 128, 32768, 2048, 64, False),
        # a running batch trimmed back to its budget every 256 tokens
        _evict("evict_b32kv8d128_c4352_to_4096", "bf16", 32, 8, 128, 4352, 4096, 256, True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_sections(rng, pairs, unit):
    """`pairs` pairs over one to three axes, in multiples of `unit` where there are several."""
    axes = rng.choice((1, 1, 2, 3))
    if pairs // unit < axes:
        return (pairs,)
    cuts = sorted(rng.sample(range(1, pairs // unit), axes - 1))
    ends = [u * unit for u in cuts] + [pairs]
    return tuple(b - a for a, b in zip([0] + ends[:-1], ends))


def draw(rng):
    kind = rng.choice(("fwd", "bwd", "append", "decode", "decode", "evict"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "fp32"))
    if kind in ("fwd", "bwd", "append"):
        D = rng.choice((64, 128)) if dtype == "bf16" else rng.choice((16, 32, 64, 128))
        Hkv = rng.choice((1, 2, 3, 4, 8, 16))
        Hq = Hkv * rng.choice((1, 1, 2, 3, 4))
        width = (Hq + 2 * Hkv) * D
        pairs = rng.choice((D // 2, D // 2, max(8, D // 4 // 8 * 8)))
        sections = _draw_sections(rng, pairs, 2)
        norm = rng.choice(("layer", "rms", "none"))
        bias = norm == "layer" and rng.random() < 0.8
        interleaved = rng.random() < 0.5
        start = rng.choice((0, 0, rng.randrange(1 << 20)))
        if kind == "append":
            B = _log(rng, 1, 128)
            N = rng.choice((1, 1, 1, _log(rng, 2, 64)))
            return _norm_rope(None, kind, dtype, B, N, Hq, Hkv, D, norm, bias, sections, interleaved, start,
                              capacity=N + _log(rng, 16, 512))
        # at most the largest listed call's elements
        tokens = _log(rng, 64, max(64, min(32768, 4 * 8192 * 32 * 128 // width // (2 if dtype == "fp32" else 1))))
        B = rng.choice((1, 2, 3, 4))
        return _norm_rope(None, kind, dtype, B, max(1, tokens // B), Hq, Hkv, D, norm, bias, sections, interleaved,
                          start)
    if kind == "decode":
        D = rng.choice((64, 128)) if dtype == "bf16" else rng.choice((16, 32, 64, 128))
        Hkv = rng.choice((1, 2, 4, 8, 16))
        Hq = Hkv * rng.choice((1, 2, 3, 4, 8))
        B = _log(rng, 1, 64)
        most = 4096 * 64 * 8 // (B * Hkv)          # cache entries of the largest listed call, over these rows
        if dtype == "fp32":
            most //= 16
        capacity = _log(rng, 16, max(16, min(65536, most)))
        prefix = rng.choice((0, _log(rng, 1, 16384), _log(rng, 1, 32768) if dtype == "bf16" else _log(rng, 1, 1024)))
        # shared scores stay below the largest listed call's
        prefix = min(prefix, 32768 * 64 * 32 // (B * Hq) // (16 if dtype == "fp32" else 1))
        return _decode(None, dtype, B, Hq, Hkv, D, capacity, prefix, rng.choice((1.0, 1.0, 2.0, 3.0)),
                       rng.random() < 0.6)
    D = rng.choice((64, 128))
    Hkv = rng.choice((1, 2, 4, 8))
    B = _log(rng, 1, 32)
    capacity = _log(rng, 64, max(64, min(65536, 32 * 8 * 4352 // (B * Hkv) // (2 if dtype == "fp32" else 1))))
    keep = _log(rng, 8, capacity)
    return _evict(None, dtype, B, Hkv, D, capacity, keep, rng.choice((0, keep // 16, keep // 2)),
                  rng.random() < 0.5)


# --------------------------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------------------------
def _sections(case):
    return tuple(int(s) for s in case["sections"].split(","))


def _frequencies(pairs):
    """Radians per position of each rotated pair, the usual geometric ladder, in 64 bits."""
    return 10000.0 ** (-torch.arange(pairs, dtype=torch.float64, device="cuda") / pairs)


def _positions(case, axes, B, N):
    """[axes, B, N] positions: a running index for one axis; for two and three, places on a frame's grid (and its
    time), as image and video tokens have them.  Every sequence starts at a place of its own."""
    i = torch.arange(N, device="cuda").view(1, N) + 17 * torch.arange(B, device="cuda").view(B, 1)
    if axes == 1:
        p = [i]
    elif axes == 2:
        p = [i // 32, i % 32]
    else:
        p = [i // 1024, i // 32 % 32, i % 32]
    return (torch.stack(p) + case["start"]).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, sigma=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * sigma + mean).to(dtype)

    s = {"case": case, "kind": case["kind"]}
    B, D, Hkv = case["B"], case["D"], case["Hkv"]
    if case["kind"] in ("fwd", "bwd", "append"):
        N, Hq, sections = case["N"], case["Hq"], _sections(case)
        s["qkv"] = normal(B, N, (Hq + 2 * Hkv) * D, sigma=1.5, mean=0.1)
        s["params"] = {"q_weight": None, "q_bias": None, "k_weight": None, "k_bias": None}
        if case["norm"] != "none":
            s["params"]["q_weight"] = normal(D, sigma=0.1, mean=1.0)
            s["params"]["k_weight"] = normal(D, sigma=0.1, mean=1.0)
        if case["bias"]:
            s["params"]["q_bias"] = normal(D, sigma=0.1)
            s["params"]["k_bias"] = normal(D, sigma=0.1)
        s["sections"] = sections
        s["frequencies"] = _frequencies(sum(sections))
        s["positions"] = _positions(case, len(sections), B, N)
        if case["kind"] == "bwd":
            s["dq"], s["dk"], s["dv"] = normal(B, Hq, N, D), normal(B, Hkv, N, D), normal(B, Hkv, N, D)
        if case["kind"] == "append":
            C = case["capacity"]
            s["k"], s["v"] = normal(B, Hkv, C, D), normal(B, Hkv, C, D)
            s["length"] = torch.randint(0, C - N + 1, (B,), generator=g, device="cuda").to(torch.int32)
        return s
    C = case["capacity"]
    s["k"], s["v"] = normal(B, Hkv, C, D, sigma=case.get("sigma", 1.0)), normal(B, Hkv, C, D)
    if case["kind"] == "decode":
        s["q"] = normal(B, case["Hq"], D, sigma=case["sigma"])
        # ragged: from nothing (one sequence in sixteen) to the whole capacity
        n = torch.randint(1, C + 1, (B,), generator=g, device="cuda")
        empty = torch.rand(B, generator=g, device="cuda") < (1.0 / 16 if B > 1 else 0.0)
        s["length"] = torch.where(empty, torch.zeros_like(n), n).to(torch.int32)
        P = case["prefix"]
        s["prefix_k"] = normal(Hkv, P, D, sigma=case["sigma"]) if P else None
        s["prefix_v"] = normal(Hkv, P, D) if P else None
        s["weight"] = torch.zeros(B, Hkv, C, device="cuda") if case["tracked"] else None
        return s
    # accumulated weights as they come about: many small ones, a few large, and exact ties (entries no query saw)
    w = torch.rand(B, Hkv, C, generator=g, device="cuda") ** 8
    s["weight"] = torch.where(w < 1e-4, torch.zeros_like(w), w)
    low = min(C, max(1, case["keep"] // 2))
    n = torch.randint(low, C + 1, (B,), generator=g, device="cuda")
    s["length"] = (n if case["ragged"] else torch.full_like(n, C)).to(torch.int32)
    K = case["keep"]
    s["out"] = (torch.zeros(B, Hkv, K, D, device="cuda", dtype=dtype),
                torch.zeros(B, Hkv, K, D, device="cuda", dtype=dtype), torch.zeros(B, Hkv, K, device="cuda"))
    return s


# --------------------------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------------------------
EPS = 1e-5


def run(state):
    kind = state["kind"]
    if own:
        return _own(state)
    if kind == "fwd":
        return _plain_norm_rope(state)
    if kind == "bwd":
        return _plain_norm_rope_backward(state)
    if kind == "append":
        return _plain_append(state)
    return _plain_decode(state) if kind == "decode" else _plain_evict(state)


def _own(s):
    import rational_softmax_attention_gb300 as ra

    case, kind = s["case"], s["kind"]
    if kind in ("fwd", "bwd", "append"):
        how = dict(s["params"], norm=case["norm"], eps=EPS, frequencies=s["frequencies"], sections=s["sections"],
                   positions=s["positions"], interleaved=case["interleaved"])
        if kind == "fwd":
            return ra.ra_qk_norm_rope(s["qkv"], case["Hq"], case["Hkv"], **how)
        if kind == "bwd":
            dqkv, dqw, dqb, dkw, dkb = ra.ra_qk_norm_rope_backward(s["qkv"], s["dq"], s["dk"], s["dv"], case["Hq"],
                                                                   case["Hkv"], **how)
            return {"dqkv": dqkv, "dqw": dqw, "dqb": dqb, "dkw": dkw, "dkb": dkb}
        q = ra.ra_cache_append(s["qkv"], s["k"], s["v"], s["length"], case["Hq"], case["Hkv"], **how)
        return q, s["k"], s["v"]
    if kind == "decode":
        o = ra.ra_attention_decode(s["q"], s["k"], s["v"], s["length"], prefix_k=s["prefix_k"],
                                   prefix_v=s["prefix_v"], weight=s["weight"])
        return o, s["weight"]
    return ra.ra_cache_evict(s["k"], s["v"], s["weight"], s["length"], case["keep"], recent=case["recent"],
                             out=s["out"])


def _angles(s):
    """cos and sin [B, 1, N, pairs] of every rotated pair, the angles in 64 bits."""
    sizes = torch.tensor(s["sections"])
    axis = torch.repeat_interleave(torch.arange(len(s["sections"])), sizes)
    pos = s["positions"][axis.tolist()].permute(1, 2, 0)             # [B, N, pairs]
    a = pos.double() * s["frequencies"]
    return torch.cos(a).float().unsqueeze(1), torch.sin(a).float().unsqueeze(1)


def _halves(x, pairs, interleaved):
    """The first and second members of the rotated pairs of x [..., D], and the rest."""
    if interleaved:
        return x[..., 0:2 * pairs:2], x[..., 1:2 * pairs:2], x[..., 2 * pairs:]
    return x[..., :pairs], x[..., pairs:2 * pairs], x[..., 2 * pairs:]


def _whole(x1, x2, rest, interleaved):
    if interleaved:
        return torch.cat([torch.stack([x1, x2], -1).flatten(-2), rest], -1)
    return torch.cat([x1, x2, rest], -1)


def _rotate(x, cos, sin, interleaved):
    x1, x2, rest = _halves(x, cos.shape[-1], interleaved)
    return _whole(x1 * cos - x2 * sin, x2 * cos + x1 * sin, rest, interleaved)


def _normalised(x, norm):
    """x [..., D] without its parameters, and 1 / its standard deviation (or root mean square)."""
    if norm == "none":
        return x, None
    if norm == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _split(case, qkv):
    """q [B, Hq, N, D], k, v [B, Hkv, N, D] as views of the packed projection."""
    x = qkv.view(case["B"], case["N"], -1, case["D"]).transpose(1, 2)
    Hq, Hkv = case["Hq"], case["Hkv"]
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def _plain_norm_rope(s):
    case = s["case"]
    q, k, v = _split(case, s["qkv"])
    cos, sin = _angles(s)

    def one(x, w, b):
        y, _ = _normalised(x.float(), case["norm"])
        if w is not None:
            y = y * w.float()
        if b is not None:
            y = y + b.float()
        return _rotate(y, cos, sin, case["interleaved"]).to(s["qkv"].dtype)

    p = s["params"]
    return one(q, p["q_weight"], p["q_bias"]), one(k, p["k_weight"], p["k_bias"]), v.contiguous()


def _plain_norm_rope_backward(s):
    case = s["case"]
    q, k, _ = _split(case, s["qkv"])
    cos, sin = _angles(s)

    def one(x, dy, w, b):
        dy = _rotate(dy.float(), cos, -sin, case["interleaved"])      # the rotation's transpose
        xhat, r = _normalised(x.float(), case["norm"])
        dw = (dy * xhat).sum((0, 1, 2)) if w is not None else None
        db = dy.sum((0, 1, 2)) if b is not None else None
        if r is None:
            return dy, dw, db
        t = dy * w.float()
        dx = t - xhat * (t * xhat).mean(-1, keepdim=True)
        if case["norm"] == "layer":
            dx = dx - t.mean(-1, keepdim=True)
        return dx * r, dw, db

    p = s["params"]
    dxq, dqw, dqb = one(q, s["dq"], p["q_weight"], p["q_bias"])
    dxk, dkw, dkb = one(k, s["dk"], p["k_weight"], p["k_bias"])
    dqkv = torch.cat([dxq, dxk, s["dv"].float()], 1).transpose(1, 2).reshape(s["qkv"].shape).to(s["qkv"].dtype)
    return {"dqkv": dqkv, "dqw": dqw, "dqb": dqb, "dkw": dkw, "dkb": dkb}


def _plain_append(s):
    case = s["case"]
    q, k, v = _plain_norm_rope(s)
    B, N, Hkv = case["B"], case["N"], case["Hkv"]
    b = torch.arange(B, device="cuda").view(B, 1, 1)
    h = torch.arange(Hkv, device="cuda").view(1, Hkv, 1)
    at = (s["length"].view(B, 1, 1) + torch.arange(N, device="cuda").view(1, 1, N)).long()
    s["k"].index_put_((b, h, at), k)
    s["v"].index_put_((b, h, at), v)
    return q, s["k"], s["v"]


def _plain_decode(s):
    case = s["case"]
    B, Hq, Hkv, D, C, P = (case[n] for n in ("B", "Hq", "Hkv", "D", "capacity", "prefix"))
    G = Hq // Hkv
    q = s["q"].float().view(B, Hkv, G, D)
    seen = torch.arange(C, device="cuda").view(1, 1, 1, C) < s["length"].view(B, 1, 1, 1)
    scores = torch.matmul(q, s["k"].float().transpose(-1, -2)) * D ** -0.5
    scores = torch.where(seen, scores, -math.inf)
    if P:
        rows = q.transpose(0, 1).reshape(Hkv, B * G, D)
        shared = torch.matmul(rows, s["prefix_k"].float().transpose(-1, -2)) * D ** -0.5
        scores = torch.cat([scores, shared.view(Hkv, B, G, P).transpose(0, 1)], -1)
    m = scores.amax(-1, keepdim=True)
    u = ((torch.where(m > -math.inf, m, 0.0) - scores) / 16.0).clamp(max=1.0)
    phi = ((1.0 - u) / (1.0 + u)) ** 8
    total = phi.sum(-1, keepdim=True)
    p = phi / torch.where(total > 0, total, 1.0)
    o = torch.matmul(p[..., :C], torch.where(seen.transpose(-1, -2), s["v"].float(), 0.0))
    if P:
        rows = p[..., C:].transpose(0, 1).reshape(Hkv, B * G, P)
        o = o + torch.matmul(rows, s["prefix_v"].float()).view(Hkv, B, G, D).transpose(0, 1)
    if s["weight"] is not None:
        s["weight"] += p[..., :C].sum(2)
    return o.reshape(B, Hq, D).to(s["q"].dtype), s["weight"]


def _plain_evict(s):
    case = s["case"]
    B, Hkv, C, keep, recent, D = (case[n] for n in ("B", "Hkv", "capacity", "keep", "recent", "D"))
    length = s["length"].view(B, 1, 1)
    slot = torch.arange(C, device="cuda").view(1, 1, C)
    w = torch.where(slot >= length - recent, math.inf, s["weight"])     # the last ones stay
    w = torch.where(slot < length, w, -math.inf)
    best = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep]
    count = torch.clamp(s["length"], max=keep)
    there = torch.arange(keep, device="cuda").view(1, 1, keep) < count.view(B, 1, 1)
    best = torch.sort(torch.where(there, best, C), dim=-1).values
    at = torch.where(there, best, 0)
    wide = at.unsqueeze(-1).expand(B, Hkv, keep, D)
    ko, vo, wo = s["out"]
    ko.copy_(torch.where(there.unsqueeze(-1), torch.gather(s["k"], 2, wide), ko))
    vo.copy_(torch.where(there.unsqueeze(-1), torch.gather(s["v"], 2, wide), vo))
    wo.copy_(torch.where(there, torch.gather(s["weight"], 2, at), wo))
    return ko, vo, wo, count, torch.where(there, best, -1).to(torch.int32)


# --------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------------------------------------------
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    B, D, Hkv = case["B"], case["D"], case["Hkv"]
    if case["kind"] in ("fwd", "bwd", "append"):
        N, Hq = case["N"], case["Hq"]
        axes = len(_sections(case))
        heads = Hq + 2 * Hkv
        rows = B * N
        pos = 4 * axes * rows
        if case["kind"] == "bwd":      # q and k parts of the projection, the incoming gradients, the outgoing one
            return {"bytes": rows * D * e * ((Hq + Hkv) + 2 * heads) + pos, "flops": 20 * rows * (Hq + Hkv) * D}
        return {"bytes": 2 * rows * heads * D * e + pos, "flops": 10 * rows * (Hq + Hkv) * D}
    if case["kind"] == "decode":       # half of the capacity is filled on the average
        Hq, C, P = case["Hq"], case["capacity"], case["prefix"]
        keys = B * Hkv * (C + 1) // 2
        n = 2 * (keys + Hkv * P) * D * e + 2 * B * Hq * D * e + (8 * keys if case["tracked"] else 0)
        return {"bytes": n, "flops": 4 * B * Hq * ((C + 1) // 2 + P) * D}
    C, keep = case["capacity"], case["keep"]
    mean = (max(1, keep // 2) + C) // 2 if case["ragged"] else C
    kept = min(mean, keep)
    return {"bytes": B * Hkv * (4 * mean + kept * (4 * D * e + 4 + 4)), "flops": 0}


# --------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------------------------------------------
def _exact_head(case, s, x, w, b):
    """One of q and k, [B, N, H, D] in 64 bits: normalised, then each pair turned as a complex number."""
    if case["norm"] == "layer":
        d = x - x.sum(-1, keepdim=True) / case["D"]
        x = d / torch.sqrt((d ** 2).sum(-1, keepdim=True) / case["D"] + EPS)
    elif case["norm"] == "rms":
        x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / case["D"] + EPS)
    x = x if w is None else x * w
    x = x if b is None else x + b
    r = sum(s["sections"])
    turn = [s["positions"][axis].double()[..., None] * f for axis, f in enumerate(s["frequencies"].split(s["sections"]))]
    turn = torch.cat(turn, -1)[:, :, None, :]
    pairs = x[..., :2 * r].unflatten(-1, (r, 2)) if case["interleaved"] else \
        x[..., :2 * r].unflatten(-1, (2, r)).transpose(-1, -2)
    z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.ones_like(turn), turn)
    z = torch.view_as_real(z)
    z = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, x[..., 2 * r:]], -1)


def _exact_norm_rope(case, s, qkv, params):
    B, N, Hq, Hkv, D = (case[n] for n in ("B", "N", "Hq", "Hkv", "D"))
    x = qkv.unflatten(-1, (Hq + 2 * Hkv, D))
    q = _exact_head(case, s, x[:, :, :Hq], params["q_weight"], params["q_bias"])
    k = _exact_head(case, s, x[:, :, Hq:Hq + Hkv], params["k_weight"], params["k_bias"])
    return q.movedim(2, 1), k.movedim(2, 1), x[:, :, Hq + Hkv:].movedim(2, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] in ("fwd", "append"):
        params = {n: None if t is None else t.double() for n, t in s["params"].items()}
        q, k, v = _exact_norm_rope(case, s, s["qkv"].double(), params)
        if case["kind"] == "fwd":
            return q, k, v
        kc, vc = s["k"].double(), s["v"].double()
        for b, n in enumerate(s["length"].tolist()):
            kc[b, :, n:n + case["N"]] = k[b]
            vc[b, :, n:n + case["N"]] = v[b]
        return q, kc, vc
    if case["kind"] == "bwd":
        # by automatic differentiation of the definition, a few sequences' tokens at a time
        total = {n: None if t is None else torch.zeros(case["D"], dtype=torch.float64, device="cuda")
                 for n, t in s["params"].items()}
        dqkv = torch.empty(s["qkv"].shape, dtype=torch.float64, device="cuda")
        step = 2048
        for b in range(case["B"]):
            for n in range(0, case["N"], step):
                part = slice(n, n + step)
                part_s = dict(s, positions=s["positions"][:, b:b + 1, part])
                part_case = dict(case, B=1, N=min(step, case["N"] - n))
                x = s["qkv"][b:b + 1, part].double().requires_grad_(True)
                params = {m: None if t is None else t.double().requires_grad_(True) for m, t in s["params"].items()}
                got = _exact_norm_rope(part_case, part_s, x, params)
                loss = sum((y * s[m][b:b + 1, :, part].double()).sum() for y, m in zip(got, ("dq", "dk", "dv")))
                loss.backward()
                dqkv[b:b + 1, part] = x.grad
                for m, t in params.items():
                    if t is not None:
                        total[m] += t.grad
        return {"dqkv": dqkv, "dqw": total["q_weight"], "dqb": total["q_bias"], "dkw": total["k_weight"],
                "dkb": total["k_bias"]}
    if case["kind"] == "decode":
        B, Hq, Hkv, D, C, P = (case[n] for n in ("B", "Hq", "Hkv", "D", "capacity", "prefix"))
        G = Hq // Hkv
        o = torch.zeros(B, Hkv, G, D, dtype=torch.float64, device="cuda")
        weight = torch.zeros(B, Hkv, C, dtype=torch.float64, device="cuda") if case["tracked"] else None
        pk = s["prefix_k"].double() if P else torch.zeros(Hkv, 0, D, dtype=torch.float64, device="cuda")
        pv = s["prefix_v"].double() if P else pk
        for b, n in enumerate(s["length"].tolist()):
            if n + P == 0:
                continue
            keys = torch.cat([pk, s["k"][b, :, :n].double()], 1)
            values = torch.cat([pv, s["v"][b, :, :n].double()], 1)
            z = s["q"][b].double().view(Hkv, G, D) @ keys.movedim(1, 2) / math.sqrt(D)
            gap = z.max(-1, keepdim=True).values - z
            f = torch.where(gap < 16.0, (16.0 - gap) / (16.0 + gap), torch.zeros_like(gap)) ** 8
            f = f / f.sum(-1, keepdim=True)
            o[b] = f @ values
            if weight is not None:
                weight[b, :, :n] = f[..., P:].sum(1)
        return o.view(B, Hq, D), weight
    # eviction only chooses and copies: the chosen entries, one row at a time
    ko, vo, wo = (t.double() for t in s["out"])
    lengths, keep, recent = s["length"].tolist(), case["keep"], case["recent"]
    for b, n in enumerate(lengths):
        last = min(recent, n)
        m = min(n, keep)
        for h in range(case["Hkv"]):
            order = torch.argsort(-s["weight"][b, h, :n - last].double(), stable=True)[:m - last]
            at = torch.cat([order.sort().values, torch.arange(n - last, n, device="cuda")])
            ko[b, h, :m] = s["k"][b, h, at].double()
            vo[b, h, :m] = s["v"][b, h, at].double()
            wo[b, h, :m] = s["weight"][b, h, at].double()
    return ko, vo, wo, None, None
