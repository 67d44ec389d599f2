"""The paged 4-bit cache of rational-softmax attention as measured work.

A cache whose keys and values lie in pages of a pool, four bits an element with a scale and a minimum for every 64
elements; sequences own pages through a table, and share them until they part.  Five operators, as a server runs them:
  write    keys and values quantised into their sequences' pages, and given back as the values that are held;
  read     the held values of any range of tokens, dense;
  decode   one query token per sequence against its pages;
  step     the table's rows replaced by their parents' (beams reordered, sequences forked and freed), then room made for
           the next token: free pages handed out, shared ones copied before they are written;
  compact  the pages in use moved together into another pool.

The layout.  pool: bytes [pages, key heads, 2 (keys, values), page, row]; row = D / 2 + D / 16.  The bytes of a page's
head are the codes [page][D / 2], then bf16 [page][2 G]: the scales of a token's G = D / 64 groups, then their minima.
Dimension 64 g + 8 w + n is nibble n of a token's 32-bit word w G + g; with D = 128 a token whose number in the page has
bit 1 set holds the two halves of its codes in the other order.  table: int32 [sequences, most pages], -1 where there is
no page; uses: int32 [pages], in how many rows of the table a page stands.

`own` selects between the plain form (elementary torch operations in 32 bits) and the framework's calls.  `exact`
restates what is computed in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# --------------------------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------------------------
def _write(name, dtype, B, N, Hkv, D, page, capacity):
    c = {"kind": "write", "dtype": dtype, "B": B, "N": N, "Hkv": Hkv, "D": D, "page": page, "capacity": capacity}
    return dict(c, name=name) if name else c


def _read(name, dtype, B, N, Hkv, D, page, capacity):
    return dict(_write(name, dtype, B, N, Hkv, D, page, capacity), kind="read")


def _decode(name, dtype, B, Hq, Hkv, D, page, capacity, shared, sigma):
    c = {"kind": "decode", "dtype": dtype, "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page, "capacity": capacity,
         "shared": shared, "sigma": sigma}
    return dict(c, name=name) if name else c


def _step(name, B, beams, Hkv, D, page, capacity, pages, tokens):
    c = {"kind": "step", "B": B, "beams": beams, "Hkv": Hkv, "D": D, "page": page, "capacity": capacity,
         "pages": pages, "tokens": tokens}
    return dict(c, name=name) if name else c


def _compact(name, B, Hkv, D, page, capacity, pages):
    c = {"kind": "compact", "B": B, "Hkv": Hkv, "D": D, "page": page, "capacity": capacity, "pages": pages}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one generated token of each of 64 sequences: a launch-bound step
        _write("write_b64kv8d128", "bf16", 64, 1, 8, 128, 64, 4096),
        # four prompts, whose own attention goes on with the values that the cache holds
        _write("write_b4n4096kv8d128", "bf16", 4, 4096, 8, 128, 64, 8192),
        # a further part of a prompt behind long documents: everything held, dense
        _read("read_b4n16384kv8d128", "bf16", 4, 16384, 8, 128, 64, 16384),
        # a 32-bit run at odd sizes with small pages, from the middle of the sequences
        _read("read_fp32_b3n777kv2d64_p16", "fp32", 3, 777, 2, 64, 16, 1003),
        # a single short conversation: latency
        _decode("decode_b1h32kv8d128_c512", "bf16", 1, 32, 8, 128, 64, 512, 0, 1.0),
        # a server's ordinary batch, forked from one instruction whose pages all share
        _decode("decode_b32h32kv8d128_c2048_s512", "bf16", 32, 32, 8, 128, 64, 2048, 512, 1.0),
        # a large batch of long contexts
        _decode("decode_b64h32kv8d128_c16384", "bf16", 64, 32, 8, 128, 64, 16384, 0, 1.0),
        # 32-bit parity runs at odd sizes with small pages, wide scores
        _decode("decode_fp32_b5h12kv4d64_c1003_p16", "fp32", 5, 12, 4, 64, 16, 1003, 100, 2.0),
        # sixteen beams of one sequence reordered after every token
        _step("step_b16beam16kv8d128", 16, 16, 8, 128, 64, 4096, 256, 1),
        # a busy server: some sequences end, others fork, the rest go on
        _step("step_b256kv8d128", 256, 4, 8, 128, 64, 4096, 8192, 1),
        # a small cache after most of its sequences have ended
        _compact("compact_b16kv2d64_p32", 16, 2, 64, 32, 1000, 1024),
        # a large pool given back
        _compact("compact_b64kv8d128", 64, 8, 128, 64, 8192, 16384),
    ]


def _log(rng, lo, hi):
    hi = max(lo, hi)
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("write", "read", "decode", "decode", "step", "compact"))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    D = rng.choice((64, 128))
    page = rng.choice((16, 32, 64, 64, 128, 256))
    Hkv = rng.choice((1, 2, 3, 4, 8))
    if kind in ("write", "read"):
        B = _log(rng, 1, 128)
        most = (4 * 4096 if kind == "write" else 4 * 16384) * 8 * 128 // (Hkv * D) // (2 if dtype == "fp32" else 1)
        N = rng.choice((1, _log(rng, 1, most // B), _log(rng, 1, most // B)))
        return (_write if kind == "write" else _read)(None, dtype, B, N, Hkv, D, page, N + _log(rng, 1, 2048))
    if kind == "decode":
        B = _log(rng, 1, 64)
        Hq = Hkv * rng.choice((1, 2, 4, 5, 8, 12, 16))
        most = 64 * 32 * 16384 * 128 // (B * max(Hq, 4 * Hkv) * D) // (16 if dtype == "fp32" else 1)
        capacity = _log(rng, 1, min(131072, most))
        return _decode(None, dtype, B, Hq, Hkv, D, page, capacity, rng.choice((0, 0, capacity // 3)),
                       rng.choice((1.0, 1.0, 2.0, 3.0)))
    part = Hkv * 2 * page * (D // 2 + D // 16)
    if kind == "step":
        B = _log(rng, 1, 256)
        capacity = _log(rng, 16, 16384)
        tokens = rng.choice((1, 1, _log(rng, 1, 300)))
        # enough for every sequence's pages and those of the new tokens in most draws, too few in some
        need = B * ((capacity + page - 1) // page + (tokens + page - 1) // page + 2)
        pages = min(int(need * rng.choice((0.7, 1.0, 1.5))) + 2, 8192 * 73728 // part, 1 << 18)
        return _step(None, B, rng.choice((1, 2, 4, 8)), Hkv, D, page, capacity, pages, tokens)
    pages = _log(rng, 16, min(1 << 17, 16384 * 73728 // part))
    B = min(_log(rng, 1, 128), pages)
    return _compact(None, B, Hkv, D, page, _log(rng, page, 8192), pages)


# --------------------------------------------------------------------------------------------------------------
# the layout
# --------------------------------------------------------------------------------------------------------------
def _swapped(page, device):
    return ((torch.arange(page, device=device) >> 1) & 1).bool()


def _up(x):
    """Non-negative 32-bit values up to the next that 16 bits hold."""
    return ((x.view(torch.int32) + 0xFFFF) & -65536).view(torch.float32)


def _down(x):
    b = x.view(torch.int32)
    return torch.where(b < 0, (b + 0xFFFF) & -65536, b & -65536).view(torch.float32)


def _codes(x):
    """x [.., D] in 32 bits -> (codes [.., G, 64] int32, scales and minima [.., G] in 32 bits).  The scale is the least
    16-bit number whose fifteenfold covers the span, a code the nearest, ties to even: in 64 bits, next to borders."""
    x = x.unflatten(-1, (-1, 64))
    lo = _down(x.amin(-1) + 0.0)                       # + 0.0: no minus zero
    span = x.amax(-1).double() - lo.double()
    s = _up((span / 15.0).float())                     # one rounding to 32 bits, which may pass a 16-bit number
    below = ((s.view(torch.int32) - 65536).clamp(min=0)).view(torch.float32)
    s = torch.where(below.double() * 15.0 >= span, below, s)
    s = torch.where(s.double() * 15.0 < span, (s.view(torch.int32) + 65536).view(torch.float32), s)
    good = torch.isfinite(span.float()) & torch.isfinite(s)
    lo = torch.where(good, lo, math.nan)
    s = torch.where(good & (s >= 2.0 ** -100), s, 0.0)
    wide = torch.where(s > 0, s, 1.0).double().unsqueeze(-1)
    u = torch.round((x.double() - lo.double().unsqueeze(-1)) / wide)
    return torch.where((s > 0).unsqueeze(-1), u, 0.0).to(torch.int32), s, lo


def _pack(x, slot):
    """Rows x [.., D] in 32 bits, of tokens whose numbers in their pages are slot [..] -> (codes [.., D / 2] bytes,
    scales and minima [.., D / 16] bytes)."""
    D = x.shape[-1]
    u, s, lo = _codes(x)
    u = u.unflatten(-1, (8, 8)).transpose(-2, -3).flatten(-3).unflatten(-1, (D // 2, 2))     # words w G + g
    b = (u[..., 0] | (u[..., 1] << 4)).to(torch.uint8)
    if D == 128:
        b = torch.where(((slot >> 1) & 1).bool().unsqueeze(-1), torch.cat([b[..., 32:], b[..., :32]], -1), b)
    return b, torch.cat([s, lo], -1).to(torch.bfloat16).contiguous().view(torch.uint8)


def _parts(pool):
    """A pool's (codes [pages, H, 2, page, D / 2], scales and minima as bf16 [pages, H, 2, page, 2 G]) as views."""
    page, row = pool.shape[3:]
    D = row * 16 // 9
    flat = pool.flatten(3)
    return (flat[..., :page * (D // 2)].unflatten(-1, (page, D // 2)),
            flat[..., page * (D // 2):].view(torch.bfloat16).unflatten(-1, (page, D // 32)))


def _unpack(codes, meta, slot, wide=torch.float32):
    """The values [.., D] that codes [.., D / 2] and meta [.., 2 G] of tokens `slot` stand for."""
    D = codes.shape[-1] * 2
    if D == 128:
        codes = torch.where(((slot >> 1) & 1).bool().unsqueeze(-1), torch.cat([codes[..., 32:], codes[..., :32]], -1), codes)
    u = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).unflatten(-1, (8, D // 64, 8)).transpose(-2, -3)
    s, lo = meta.to(wide).chunk(2, -1)
    return (lo[..., None, None] + s[..., None, None] * u.to(wide)).flatten(-3)


# --------------------------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------------------------
def _row(D):
    return D // 2 + D // 16


def _filled_pool(g, pages, Hkv, page, D, sigma):
    """A pool whose every slot holds quantised normal keys and values, keys with a mean of their own in every
    dimension; pages that no sequence owns hold what earlier sequences left."""
    pool = torch.empty(pages, Hkv, 2, page, _row(D), dtype=torch.uint8, device="cuda")
    codes, meta = _parts(pool)
    mean = torch.randn(Hkv, 2, 1, D, generator=g, device="cuda") * 0.5
    mean[:, 1] = 0.0
    spread = torch.tensor([sigma, 1.0], device="cuda").view(2, 1, 1)
    slot = torch.arange(page, device="cuda")
    step = max(1, (1 << 26) // (Hkv * 2 * page * D))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = (torch.randn(n, Hkv, 2, page, D, generator=g, device="cuda") + mean) * spread
        b, m = _pack(x, slot)
        codes[p:p + n] = b
        meta[p:p + n] = m.view(torch.bfloat16)
    return pool


def _cut(n, page):
    return (n + page - 1) // page


def _table(g, lengths, M, page, pages, shared=0):
    """Rows of pages in no order, the first `shared` tokens' ones the same in all rows; and the pages' uses."""
    B = lengths.numel()
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    at = torch.arange(M, device="cuda").view(1, M)
    held = at < _cut(lengths, page).view(B, 1)
    common = min(shared // page, M)
    place = torch.where(at < common, at, common + torch.arange(B, device="cuda").view(B, 1) * (M - common) + at - common)
    table = torch.where(held, order[place.clamp(max=pages - 1)], -1).to(torch.int32)
    return table, torch.bincount(table[held].long(), minlength=pages).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    kind, B, Hkv, D, page = case["kind"], case["B"], case["Hkv"], case["D"], case["page"]
    M = _cut(case["capacity"], page)
    s = {"case": case, "kind": kind}
    if kind in ("write", "read", "decode"):
        dtype = DTYPES[case["dtype"]]
        common = min(case.get("shared", 0) // page, M)
        pages = common + B * (M - common)
        if kind == "decode":
            C = case["capacity"]
            # ragged: behind the shared part from nothing on; now and then an empty sequence
            n = torch.randint(min(case["shared"], C - 1) + 1, C + 1, (B,), generator=g, device="cuda")
            empty = torch.rand(B, generator=g, device="cuda") < (1.0 / 16 if B > 1 else 0.0)
            s["length"] = torch.where(empty, 0, n).to(torch.int32)
            s["table"], _ = _table(g, s["length"], M, page, pages, common * page)
            s["pool"] = _filled_pool(g, pages, Hkv, page, D, case["sigma"])
            s["q"] = (torch.randn(B, case["Hq"], D, generator=g, device="cuda") * case["sigma"]).to(dtype)
            return s
        N, C = case["N"], case["capacity"]
        s["start"] = torch.randint(0, C - N + 1, (B,), generator=g, device="cuda").to(torch.int32)
        s["length"] = (s["start"] + N).to(torch.int32)
        s["table"], _ = _table(g, s["length"], M, page, pages)
        if kind == "write":
            s["pool"] = torch.randint(0, 256, (pages, Hkv, 2, page, _row(D)), generator=g, device="cuda", dtype=torch.uint8)
            mean = torch.randn(Hkv, 1, D, generator=g, device="cuda") * 0.5
            s["k"] = (torch.randn(B, Hkv, N, D, generator=g, device="cuda") + mean).to(dtype)
            s["v"] = torch.randn(B, Hkv, N, D, generator=g, device="cuda").to(dtype)
        else:
            s["pool"] = _filled_pool(g, pages, Hkv, page, D, 1.0)
        return s
    P, C = case["pages"], case["capacity"]
    s["pool"] = torch.randint(0, 256, (P, Hkv, 2, page, _row(D)), generator=g, device="cuda", dtype=torch.uint8)
    if kind == "step":
        # what the pool has room for, with pages to spare for the copies
        M += _cut(case["tokens"], page)
        most = max(1, min(C, (P - 2) // (B + 1) * page))
        n = torch.randint(max(1, most // 2), most + 1, (B,), generator=g, device="cuda").to(torch.int32)
        s["length"] = n
        s["table"], s["uses"] = _table(g, n, M, page, P)
        # every group of `beams` neighbours goes on from members of its own; with fewer than eight beams one sequence in
        # sixteen ends instead
        b = torch.arange(B, device="cuda")
        k = case["beams"]
        parent = torch.minimum(b // k * k + torch.randint(0, k, (B,), generator=g, device="cuda"), torch.tensor(B - 1, device="cuda"))
        if k < 8:
            parent = torch.where(torch.rand(B, generator=g, device="cuda") < 0.5, b, parent)
            parent = torch.where(torch.rand(B, generator=g, device="cuda") < 1.0 / 16, -1, parent)
        s["parent"] = parent.to(torch.int32)
        s["count"] = torch.where(parent >= 0, case["tokens"], 0).to(torch.int32)
        return s
    # half of the sequences have ended: their pages are free, here and there in the pool
    most = max(1, min(C, P // B * page))
    n = torch.randint(max(1, most // 2), most + 1, (B,), generator=g, device="cuda")
    n = torch.where(torch.rand(B, generator=g, device="cuda") < 0.5, n, 0).to(torch.int32)
    n[0] = most
    s["table"], s["uses"] = _table(g, n, M, page, P)
    s["out"] = torch.zeros(max(1, (P + 1) // 2 + P // 8), Hkv, 2, page, _row(D), dtype=torch.uint8, device="cuda")
    return s


# --------------------------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------------------------
def run(state):
    if own:
        return _own(state)
    return {"write": _plain_write, "read": _plain_read, "decode": _plain_decode, "step": _plain_step,
            "compact": _plain_compact}[state["kind"]](state)


def _own(s):
    import rational_softmax_attention_gb300 as ra

    case, kind = s["case"], s["kind"]
    if kind == "write":
        k, v = ra.ra_page_write(s["k"], s["v"], s["pool"], s["table"], s["start"], held=True)
        return k, v, s["pool"]
    if kind == "read":
        return ra.ra_page_read(s["pool"], s["table"], s["length"], case["N"], start=s["start"], dtype=DTYPES[case["dtype"]])
    if kind == "decode":
        return ra.ra_attention_decode_paged(s["q"], s["pool"], s["table"], s["length"])
    if kind == "step":
        ra.ra_page_fork(s["table"], s["length"], s["uses"], s["parent"])
        granted = ra.ra_page_reserve(s["pool"], s["table"], s["length"], s["uses"], case["tokens"], count=s["count"])
        return s["table"], s["length"], s["uses"], granted, s["pool"]
    table, uses, live = ra.ra_page_compact(s["pool"], s["table"], s["uses"], s["out"])
    return table, uses, live, s["out"]


def _places(s):
    """(page, slot in it), each [B, N], of tokens start .. start + N - 1."""
    case = s["case"]
    at = s["start"].long().view(-1, 1) + torch.arange(case["N"], device="cuda").view(1, -1)
    return torch.gather(s["table"], 1, at // case["page"]).long(), at % case["page"]


def _plain_write(s):
    page, slot = _places(s)
    codes, meta = _parts(s["pool"])
    held = []
    for i, x in enumerate((s["k"], s["v"])):
        x = x.float().transpose(1, 2)                                      # [B, N, H, D]
        b, m = _pack(x, slot.unsqueeze(-1))
        codes[page, :, i, slot] = b
        meta[page, :, i, slot] = m.view(torch.bfloat16)
        u, sc, lo = _codes(x)
        y = (lo.unsqueeze(-1) + sc.unsqueeze(-1) * u.float()).flatten(-2)
        held.append(y.transpose(1, 2).to(s["k"].dtype).contiguous())
    return held[0], held[1], s["pool"]


def _plain_read(s):
    page, slot = _places(s)
    codes, meta = _parts(s["pool"])
    out = []
    for i in range(2):
        y = _unpack(codes[page, :, i, slot], meta[page, :, i, slot], slot.unsqueeze(-1))
        out.append(y.transpose(1, 2).to(DTYPES[s["case"]["dtype"]]).contiguous())
    return tuple(out)


def _plain_decode(s):
    case = s["case"]
    B, Hq, Hkv, D, page = (case[n] for n in ("B", "Hq", "Hkv", "D", "page"))
    M = s["table"].shape[1]
    C, G = M * page, Hq // Hkv
    codes, meta = _parts(s["pool"])
    at = s["table"].clamp(min=0).long()
    slot = torch.arange(page, device="cuda")
    seen = torch.arange(C, device="cuda").view(1, 1, 1, C) < s["length"].view(B, 1, 1, 1)

    def held(i):                                                           # [B, H, C, D]
        y = _unpack(codes[at, :, i], meta[at, :, i], slot)
        return y.transpose(1, 2).reshape(B, Hkv, C, D)

    z = torch.matmul(s["q"].float().view(B, Hkv, G, D), held(0).transpose(-1, -2)) * D ** -0.5
    z = torch.where(seen, z, -math.inf)
    m = z.amax(-1, keepdim=True)
    d = ((torch.where(m > -math.inf, m, 0.0) - z) / 16.0).clamp(max=1.0)
    phi = ((1.0 - d) / (1.0 + d)) ** 8
    total = phi.sum(-1, keepdim=True)
    p = phi / torch.where(total > 0, total, 1.0)
    o = torch.matmul(p, torch.where(seen.transpose(-1, -2), held(1), 0.0))
    return o.reshape(B, Hq, D).to(s["q"].dtype)


def _counted(table, uses, by):
    """uses, plus `by` for every place in the table that holds a page."""
    there = table >= 0
    ones = torch.where(there, by, 0).flatten().to(torch.int32)
    return uses.scatter_add(0, table.clamp(min=0).flatten().long(), ones)


def _plain_step(s):
    case = s["case"]
    page, tokens = case["page"], case["tokens"]
    table, length, parent = s["table"], s["length"], s["parent"].long()
    B, M = table.shape
    # the rows of their parents
    ends = parent < 0
    rows = torch.where(ends.view(B, 1), -1, table[parent.clamp(min=0)]).to(torch.int32)
    uses = _counted(rows, _counted(table, s["uses"], -1), 1)
    length.copy_(torch.where(ends, 0, length[parent.clamp(min=0)]))
    # the pages that the new tokens touch, [B, K]
    K = (tokens + page - 2) // page + 1
    n = s["count"].clamp(0, tokens).long()
    first = length.long() // page
    at = first.view(B, 1) + torch.arange(K, device="cuda").view(1, K)
    touched = (n > 0).view(B, 1) & (at * page < (length.long() + n).view(B, 1)) & (at < M)
    old = torch.where(touched, torch.gather(rows, 1, at.clamp(max=M - 1)), -1).long()
    wanted = touched & ((old < 0) | (uses[old.clamp(min=0)] > 1))
    rank = torch.cumsum(wanted.flatten(), 0).view(B, K) - 1
    free = torch.argsort((uses != 0).to(torch.int8), stable=True)
    got = wanted & (rank < (uses == 0).sum())
    new = free[rank.clamp(0, free.numel() - 1)]
    # the first page of a sequence that is not at a page's start keeps its content
    copies = got[:, 0] & (old[:, 0] >= 0) & (length % page != 0)
    # (a sequence without a copy repeats the first one's, or page 0's on itself)
    other, some = copies.to(torch.int8).argmax().view(1), copies.any()
    to = torch.where(copies, new[:, 0], torch.where(some, new[other, 0], 0))
    s["pool"][to] = s["pool"][torch.where(copies, old[:, 0], torch.where(some, old[other, 0], 0))]
    uses = uses.scatter_add(0, old.clamp(min=0).flatten(), -(got & (old >= 0)).flatten().to(torch.int32))
    uses = uses.scatter_add(0, torch.where(got, new, 0).flatten(), got.flatten().to(torch.int32))
    # one place past the row's end takes what is not written
    rows = torch.cat([rows, rows[:, :1]], 1)
    rows.scatter_(1, torch.where(got, at, M), torch.where(got, new, 0).to(torch.int32))
    table.copy_(rows[:, :M])
    s["uses"].copy_(uses)
    room = torch.where(wanted & ~got, at * page - length.long().view(B, 1), M * page).amin(1).clamp(min=0)
    granted = torch.minimum(torch.minimum(n, room), (M * page - length.long()).clamp(min=0)).to(torch.int32)
    return table, length, s["uses"], granted, s["pool"]


def _plain_compact(s):
    pool, out, uses = s["pool"], s["out"], s["uses"]
    P2 = out.shape[0]
    live = uses > 0
    rank = (torch.cumsum(live, 0) - 1).to(torch.int32)
    order = torch.argsort((~live).to(torch.int8), stable=True)[:P2]
    count = live.sum().to(torch.int32).view(1)
    there = torch.arange(order.numel(), device="cuda") < count
    out[:order.numel()] = torch.where(there.view(-1, 1, 1, 1, 1), pool[order], out[:order.numel()])
    new_uses = torch.zeros(P2, dtype=torch.int32, device="cuda")
    new_uses[:order.numel()] = torch.where(there, uses[order], 0)
    at = rank[s["table"].clamp(min=0).long()]
    table = torch.where((s["table"] >= 0) & (at < P2), at, -1)
    return table, new_uses, count, out


# --------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------------------------------------------
def work(case):
    kind, B, Hkv, D, page = case["kind"], case["B"], case["Hkv"], case["D"], case["page"]
    row = _row(D)
    if kind in ("write", "read"):
        e = 2 if case["dtype"] == "bf16" else 4
        rows = 2 * B * case["N"] * Hkv
        wide = rows * D * e * (2 if kind == "write" else 1)      # write: the rows come in, and go out as they are held
        return {"bytes": wide + rows * row, "flops": (4 if kind == "write" else 2) * rows * D}
    if kind == "decode":       # the parts of the sequences that are their own are half full on the average
        e, Hq, C = 2 if case["dtype"] == "bf16" else 4, case["Hq"], case["capacity"]
        common = min(case["shared"], C)
        n = common + (C - common + 1) / 2
        if B > 1:
            n *= 15 / 16
        tokens = B * n - (B - 1) * (common // page * page) * (15 / 16 if B > 1 else 1.0)
        return {"bytes": 2 * max(tokens, 1.0) * Hkv * row + 2 * B * Hq * D * e + 4 * B * _cut(n, page),
                "flops": 4 * B * Hq * n * D}
    part = Hkv * 2 * page * row
    M = _cut(case["capacity"], page)
    if kind == "step":         # a table read and written, the pages' uses, and a copied page for most that fork
        forks = B * (0.95 if case["beams"] >= 8 else 0.45 * (1 - 1 / case["beams"]))
        return {"bytes": 8 * B * M + 8 * case["pages"] + 2 * forks * part, "flops": 0}
    live = min(case["pages"], B // 2 * _cut(min(case["capacity"], case["pages"] // B * page) * 3 / 4, page))
    return {"bytes": 2 * max(live, 1) * part + 8 * B * M + 8 * case["pages"], "flops": 0}


# --------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------------------------------------------
def _exact_rows(pool, D, pages, slots, head, which):
    """The values [n, D] in 64 bits of one head's tokens at (pages, slots), dimension by dimension from the layout."""
    page = pool.shape[3]
    flat = pool[:, head, which].reshape(pool.shape[0], -1)
    d = torch.arange(D, device="cuda")
    G = D // 64
    word = (d % 64 // 8) * G + d // 64
    byte = word * 4 + d % 8 // 2
    if D == 128:
        byte = byte.view(1, D) ^ (((slots.view(-1, 1) >> 1) & 1) * 32)
    code = flat[pages.view(-1, 1), slots.view(-1, 1) * (D // 2) + byte].long()
    u = torch.where(d % 2 == 1, code // 16, code % 16).double()
    at = page * (D // 2) + slots.view(-1, 1) * (4 * G) + 2 * (d // 64).view(1, D)

    def half(at):
        b = flat[pages.view(-1, 1), at].int() | (flat[pages.view(-1, 1), at + 1].int() << 8)
        return (b << 16).view(torch.float32).double()

    return half(at + 2 * G) + half(at) * u


def _exact_held(x):
    """What [.., D] is held as, in 64 bits."""
    x = x.double().unflatten(-1, (-1, 64))
    low = x.amin(-1, keepdim=True)

    def grid(y):         # the distance of neighbouring values with eight significant bits
        return ((torch.frexp(y).exponent.long() - 8 + 1023) << 52).view(torch.float64)

    lo = torch.floor(low / grid(low)) * grid(low)
    span = x.amax(-1, keepdim=True) - lo
    s = span / torch.full_like(span, 15.0)
    s = torch.ceil(s / grid(s)) * grid(s)
    u = torch.where(s > 0, torch.round((x - lo) / torch.where(s > 0, s, 1.0)), 0.0)
    return (lo + s * u).flatten(-2)


def exact(case, seed):
    kind = case["kind"]
    if kind in ("step", "compact"):          # choices and copies: whole numbers alone
        return None
    s = prepare(case, seed)
    B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    if kind == "write":
        return _exact_held(s["k"]), _exact_held(s["v"]), None
    table = s["table"].long()
    if kind == "read":
        out = torch.empty(2, B, Hkv, case["N"], D, dtype=torch.float64, device="cuda")
        for b, n in enumerate(s["start"].tolist()):
            t = torch.arange(n, n + case["N"], device="cuda")
            for h in range(Hkv):
                for i in range(2):
                    out[i, b, h] = _exact_rows(s["pool"], D, table[b, t // page], t % page, h, i)
        return out[0], out[1]
    Hq = case["Hq"]
    G = Hq // Hkv
    o = torch.zeros(B, Hkv, G, D, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["length"].tolist()):
        if n == 0:
            continue
        t = torch.arange(n, device="cuda")
        for h in range(Hkv):
            keys = _exact_rows(s["pool"], D, table[b, t // page], t % page, h, 0)
            z = s["q"][b, h * G:(h + 1) * G].double() @ keys.T / math.sqrt(D)
            gap = z.max(-1, keepdim=True).values - z
            f = torch.where(gap < 16.0, (16.0 - gap) / (16.0 + gap), torch.zeros_like(gap)) ** 8
            f = f / f.sum(-1, keepdim=True)
            o[b, h] = f @ _exact_rows(s["pool"], D, table[b, t // page], t % page, h, 1)
    return o.view(B, Hq, D)
