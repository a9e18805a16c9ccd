"""The operators on a sequence's text K/V, as a benchmark: appending to the paged text cache, reading it
back, and attention of drafted tokens over it.

The text cache keeps one layer's text K and V in pages of `page` tokens.  A token's head_dim values in one
head are held as bfloat16 ("bf16"), as E4M3 codes ("mxfp8") or as E2M1 codes, two to a byte ("mxfp4"); the
coded formats have one power-of-two scale for each 32 values (E8M0, 2^(byte - 127), 255 for a group that
holds an infinity or a NaN).  The scale is the smallest power of two that brings the group's largest
magnitude within the code's largest value, so scaling is exact and the only rounding is to the code's grid.

A batch is rows: sequence s owns rows row_starts[s] .. row_starts[s+1], its newest tokens, which stand at
the cache positions kv_lens[s] - n .. kv_lens[s] - 1.  Row i of the n may attend to every token before them
and to those of the n whose bits are set in its tree word.
"""
import math
import random

import torch

own = False

E4M3_MAX, E2M1_MAX = 448.0, 6.0
CODE_BITS = {"bf16": 16, "mxfp8": 8, "mxfp4": 4}


# ------------------------------------------------------------------------------------------ cases ---
def listed():
    return [
        # one generated token for each of 8 requests: the smallest call of a decode step (4 K/V heads x 256)
        dict(name="append_step", op="append", fmt="mxfp8", heads=4, dim=256, page=64, seqs=8, rows=1, ctx=701,
             io="bf16"),
        # drafted trees of 16 requests on a cache kept in bf16 (4 K/V heads x 128, float32 activations)
        dict(name="append_tree_f32", op="append", fmt="bf16", heads=4, dim=128, page=16, seqs=16, rows=23, ctx=333,
             io="f32"),
        # four long ragged prompts written at once at 4 bits (8 K/V heads x 128)
        dict(name="append_prompts", op="append", fmt="mxfp4", heads=8, dim=128, page=64, seqs=4, rows=12001, ctx=12001,
             io="bf16"),
        # the shared prefix of a conversation read back for the next turn's prompt
        dict(name="read_prefix", op="read", fmt="mxfp8", heads=4, dim=256, page=64, seqs=2, rows=9973, ctx=9973,
             io="bf16"),
        # the last few tokens of each request read back for a rescoring pass
        dict(name="read_window", op="read", fmt="mxfp4", heads=8, dim=128, page=32, seqs=8, rows=37, ctx=1500,
             io="f32"),
        # the first generated token after a one-token text prompt: pure latency
        dict(name="decode_first", op="attention", fmt="bf16", heads=1, dim=64, page=16, seqs=1, group=1, rows=1, ctx=2,
             io="bf16", merge=True),
        # single-token decode of 16 requests, 7 query heads to a K/V head, merged with the visual tokens' partial
        dict(name="decode_batch", op="attention", fmt="bf16", heads=4, dim=128, page=64, seqs=16, group=7, rows=1,
             ctx=4090, io="bf16", merge=True),
        # single-token decode of one request with a very long text (4 K/V heads x 256)
        dict(name="decode_long", op="attention", fmt="mxfp8", heads=4, dim=256, page=64, seqs=1, group=2, rows=1,
             ctx=130001, io="bf16", merge=True),
        # the same float32 queries that the visual attention takes, a short tree on a bf16 cache
        dict(name="tree_f32", op="attention", fmt="bf16", heads=2, dim=64, page=16, seqs=3, group=4, rows=12, ctx=311,
             io="f32", merge=True),
        # medium trees of 8 requests (the 4B-class head layout, 8-bit cache)
        dict(name="tree_medium", op="attention", fmt="mxfp8", heads=4, dim=256, page=64, seqs=8, group=2, rows=16,
             ctx=2047, io="bf16", merge=True),
        # short trees of 32 requests on a 4-bit cache: the cache's size decides
        dict(name="tree_batch", op="attention", fmt="mxfp4", heads=8, dim=128, page=64, seqs=32, group=4, rows=6,
             ctx=6001, io="bf16", merge=False),
        # the widest trees (the 32B-class head layout): matrix products decide
        dict(name="tree_wide", op="attention", fmt="mxfp8", heads=8, dim=128, page=128, seqs=4, group=8, rows=63,
             ctx=8111, io="bf16", merge=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "attention", "attention", "attention"])
    case = dict(op=op, fmt=rng.choice(["bf16", "mxfp8", "mxfp4"]), heads=rng.choice([1, 2, 3, 4, 5, 8]),
                dim=rng.choice([32, 64, 96, 128, 128, 160, 192, 256]), page=rng.choice([16, 32, 64, 128]),
                io=rng.choice(["bf16", "bf16", "f32"]))
    seqs = case["seqs"] = _log(rng, 1, 32)
    width = case["heads"] * case["dim"]
    if op == "attention":
        case["rows"] = _log(rng, 1, 64)
        case["group"] = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
        case["merge"] = rng.random() < 0.5
        # at most the listed extremes' cache elements and multiply-adds
        most = min(130000, (32 << 20) * 2 // (seqs * width))
        most = min(most, int(8e9) // (seqs * width * case["rows"] * case["group"]) + 1)
        case["ctx"] = _log(rng, 1, max(2, most)) + case["rows"]
    else:
        most = max(2, min(20000, (16 << 20) // (seqs * width)))
        case["rows"] = _log(rng, 1, most)
        case["ctx"] = case["rows"] + (_log(rng, 1, max(2, most // 2)) - 1 if rng.random() < 0.7 else 0)
    return case


def _lengths(case):
    """(rows, cache length with those rows) of every sequence: ragged, down to half of the case's own."""
    n, ctx, seqs = case["rows"], case["ctx"], case["seqs"]
    got = []
    for s in range(seqs):
        rows = n - (s * n) // (2 * seqs)
        before = (ctx - n) - (s * (ctx - n)) // (2 * seqs)
        got.append((rows, before + rows))
    return got


def work(case):
    lens = _lengths(case)
    heads, dim, bits = case["heads"], case["dim"], CODE_BITS[case["fmt"]]
    row_bytes = dim * bits // 8 + (0 if bits == 16 else dim // 32)   # one token and head of K or of V in the cache
    io = 4 if case["io"] == "f32" else 2
    rows = sum(r for r, _ in lens)
    if case["op"] != "attention":
        plain = 2 * rows * heads * dim * io
        held = 2 * rows * heads * row_bytes
        # append: rows in, codes out, and the values that the codes stand for out
        return {"bytes": held + plain * (2 if case["op"] == "append" else 1), "flops": 0}
    qh = heads * case["group"]
    cache = 2 * heads * row_bytes * sum(t for _, t in lens)
    rowio = rows * qh * (2 * dim * io + 8) + (rows * qh * (4 * dim + 8) if case["merge"] else 0)
    return {"bytes": cache + rowio, "flops": 4 * dim * qh * sum(r * t for r, t in lens)}


# ----------------------------------------------------------------------------------------- inputs ---
def _kv(gen, shape, dtype, outliers):
    """Activations as K and V have them: unit spread, K with a few channels several times larger."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    if outliers:
        x *= 1 + 5 * (torch.rand(shape[-2:], generator=gen, device="cuda") < 0.03)
    return x.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype = torch.float32 if case["io"] == "f32" else torch.bfloat16
    heads, dim, page, fmt = case["heads"], case["dim"], case["page"], case["fmt"]
    lens = _lengths(case)
    rows = [r for r, _ in lens]
    total = sum(rows)
    width = max(-(-t // page) for _, t in lens)
    used = sum(-(-t // page) for _, t in lens)
    n_pages = used + 3
    perm = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at, perm_host = 0, perm.cpu()
    for s, (_, t) in enumerate(lens):
        k = -(-t // page)
        table[s, :k] = perm_host[at:at + k]
        at += k
    starts = torch.zeros(len(lens) + 1, dtype=torch.int32)
    starts[1:] = torch.cumsum(torch.tensor(rows), 0)
    state = dict(case, table=table.cuda(), row_starts=starts.cuda(), max_rows=max(rows),
                 kv_lens=torch.tensor([t for _, t in lens], dtype=torch.int32, device="cuda"),
                 max_kv_len=max(t for _, t in lens), n_rows=total, dtype=dtype)
    row_bytes = dim * CODE_BITS[fmt] // 8
    for name in ("k", "v"):
        pool = torch.empty((n_pages, heads, page, row_bytes), dtype=torch.uint8, device="cuda")
        scales = torch.empty((n_pages, heads, page, dim // 32), dtype=torch.uint8, device="cuda")
        if case["op"] == "append":
            pool.random_(0, 256, generator=gen)      # pages hold what earlier requests left in them
            scales.random_(0, 255, generator=gen)
        else:
            for p in range(0, n_pages, 256):           # a cache as appending fills it, some pages at a time
                q = min(256, n_pages - p)
                x = _kv(gen, (q, page, heads, dim), torch.float32, name == "k").transpose(1, 2)
                pool[p:p + q], scales[p:p + q] = _encode(x, fmt)
        state[name + "_pages"], state[name + "_scales"] = pool, scales
    if case["op"] == "attention":
        qh = heads * case["group"]
        state["q"] = (1.5 * torch.randn((total, qh, dim), generator=gen, device="cuda")).to(dtype)
        # a random tree for each sequence: node j hangs under an earlier node; its word holds its ancestors and itself
        words, r = [], random.Random(int(seed))
        for n in rows:
            mine = []
            for j in range(n):
                up = mine[r.randrange(max(0, j - 6), j)] if j else 0
                mine.append(up | (1 << j))
            words += mine
        signed = [w - (1 << 64) if w >> 63 else w for w in words]
        state["tree"] = torch.tensor(signed, dtype=torch.int64, device="cuda")
        state["prior"] = None
        if case["merge"]:
            o = torch.randn((total, qh, dim), generator=gen, device="cuda") * 0.1
            m = 4 + 0.5 * torch.randn((total, qh), generator=gen, device="cuda")
            l = 50 + 400 * torch.rand((total, qh), generator=gen, device="cuda")
            state["prior"] = (o, m, l)
    elif case["op"] == "append":
        state["k"] = _kv(gen, (total, heads, dim), dtype, True)
        state["v"] = _kv(gen, (total, heads, dim), dtype, False)
    if own:   # the handle and the workspace that a user's program keeps
        from dct_transform_coding_b200 import tactkv as T
        state["cache"] = T.TextCache(fmt, state["k_pages"], state["v_pages"],
                                     None if fmt == "bf16" else state["k_scales"],
                                     None if fmt == "bf16" else state["v_scales"])
        state["workspace"] = T.text_workspace(state["cache"], n_seqs=len(lens), n_rows=total, max_rows=max(rows),
                                              q_heads=heads * case.get("group", 1), max_kv_len=state["max_kv_len"])
    return state


# ------------------------------------------------------------------------------------ plain forms ---
def _pow2(e):
    """2^e as float32, exactly (a power function rounds): the exponent field of a float64."""
    return ((e.long() + 1023) << 52).view(torch.float64).float()


def _encode(x, fmt):
    """Codes and scale bytes of x [..., dim] (float32), each group of 32 on its own."""
    if fmt == "bf16":
        return x.to(torch.bfloat16).contiguous().view(torch.uint8), torch.zeros((), dtype=torch.uint8, device=x.device)
    top, shift = (0.875, 9) if fmt == "mxfp8" else (0.75, 3)        # 448 = 0.875 * 2^9, 6 = 0.75 * 2^3
    g = x.reshape(*x.shape[:-1], -1, 32)
    amax = g.abs().amax(-1)
    bad = ~torch.isfinite(amax)
    mant, ex = torch.frexp(torch.where(bad, 1.0, amax))
    e = torch.clamp(ex - shift + (mant > top), -127, 127)
    e = torch.where(amax == 0, -127, e)
    u = torch.where(bad[..., None], 0.0, g * _pow2(-e[..., None]))
    scales = torch.where(bad, 255, e + 127).to(torch.uint8)
    if fmt == "mxfp8":
        codes = u.to(torch.float8_e4m3fn).view(torch.uint8).reshape(x.shape)
    else:
        a = u.abs()   # round to nearest on 0, 1/2, 1, 3/2, 2, 3, 4, 6; a tie goes to the even code
        n = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte()
             + (a >= 3.5).byte() + (a > 5).byte())
        n = (n + 8 * torch.signbit(u).byte()).reshape(*x.shape[:-1], -1, 2)
        codes = n[..., 0] + 16 * n[..., 1]
    return codes, scales


def _decode(codes, scales, fmt):
    """The float32 values that codes [..., row bytes] and scale bytes [..., dim / 32] stand for."""
    if fmt == "bf16":
        return codes.contiguous().view(torch.bfloat16).float()
    if fmt == "mxfp8":
        u = codes.view(torch.float8_e4m3fn).float()
    else:
        levels = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
        u = levels[torch.stack((codes & 15, codes >> 4), -1).int().flatten(-2)]
    g = u.reshape(*u.shape[:-1], -1, 32)
    e = scales.int()[..., None] - 127
    return torch.where(e == 128, math.nan, g * _pow2(e)).reshape(u.shape)


def _row_places(s):
    """(page, offset in it) of every row."""
    starts, lens = s["row_starts"].long(), s["kv_lens"].long()
    row = torch.arange(s["n_rows"], device=starts.device)
    seq = torch.searchsorted(starts[1:], row, right=True)
    pos = lens[seq] - (starts[seq + 1] - row)
    return s["table"][seq, pos // s["page"]].long(), pos % s["page"], seq, row - starts[seq]


def _append(s):
    page, off, _, _ = _row_places(s)
    values = []
    for name in ("k", "v"):
        codes, scales = _encode(s[name].float(), s["fmt"])
        s[name + "_pages"][page, :, off] = codes
        if s["fmt"] != "bf16":
            s[name + "_scales"][page, :, off] = scales
        values.append(_decode(codes, scales, s["fmt"]).to(s["dtype"]))
    return values


def _read(s):
    page, off, _, _ = _row_places(s)
    return [_decode(s[n + "_pages"][page, :, off], s[n + "_scales"][page, :, off], s["fmt"]).to(s["dtype"])
            for n in ("k", "v")]


def _attend(s):
    heads, dim, G = s["heads"], s["dim"], s["group"]
    _, _, seq, node = _row_places(s)
    lens, starts = s["kv_lens"].long(), s["row_starts"].long()
    S, R, n = len(lens), s["max_rows"], starts[1:] - starts[:-1]
    T = s["table"].shape[1] * s["page"]
    table = s["table"].clamp(min=0).long()
    t = torch.arange(T, device=lens.device)
    held = t < lens[:, None]                                                             # [S, T]
    kv = []
    for name in ("k", "v"):
        x = _decode(s[name + "_pages"][table], s[name + "_scales"][table], s["fmt"])      # [S, pages, heads, page, dim]
        x = x.permute(0, 2, 1, 3, 4).reshape(S, heads, T, dim)
        kv.append(torch.where(held[:, None, :, None], x, 0.0))
    q = torch.zeros((S, R, heads * G, dim), device=lens.device)
    q[seq, node] = s["q"].float()
    words = torch.zeros((S, R), dtype=torch.int64, device=lens.device)
    words[seq, node] = s["tree"]
    j = t - (lens - n)[:, None]                                                           # [S, T]: the node at t, or < 0
    bit = (words[:, :, None] >> j.clamp(0, 63)[:, None, :]) & 1
    seen = held[:, None, :] & ((j < 0)[:, None, :] | (bit == 1))                          # [S, R, T]
    q = q.reshape(S, R, heads, G, dim).permute(0, 2, 1, 3, 4).reshape(S, heads, R * G, dim)
    score = (q @ kv[0].transpose(-1, -2)).mul_(1 / math.sqrt(dim)).view(S, heads, R, G, T)
    score.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = score.amax(-1)
    p = score.sub_(torch.where(m == -math.inf, 0.0, m)[..., None]).exp_()
    l = p.sum(-1)
    o = (p.view(S, heads, R * G, T) @ kv[1]).view(S, heads, R, G, dim)
    o, m, l = (x.transpose(1, 2).flatten(2, 3)[seq, node] for x in (o, m, l))             # [rows, q heads(, dim)]
    if s["prior"] is not None:
        po, pm, pl = s["prior"]
        top = torch.maximum(m, pm)
        safe = torch.where(top == -math.inf, 0.0, top)
        a, b = torch.exp(m - safe), torch.exp(pm - safe) * pl
        o, l, m = o * a[..., None] + po * b[..., None], l * a + b, top
    o = torch.where(l[..., None] == 0, 0.0, o / l[..., None])
    return [o.to(s["dtype"]), m, l]


def run(s):
    if own:
        from dct_transform_coding_b200 import tactkv as T
        rows = (s["table"], s["kv_lens"], s["row_starts"])
        if s["op"] == "append":
            k, v = T.text_append(s["cache"], s["k"], s["v"], *rows, values=True, workspace=s["workspace"])
        elif s["op"] == "read":
            return T.text_read(s["cache"], *rows, n_rows=s["n_rows"], dtype=s["dtype"], workspace=s["workspace"])
        else:
            return T.text_attention(s["q"], s["cache"], *rows, max_rows=s["max_rows"], max_kv_len=s["max_kv_len"],
                                    tree=s["tree"], prior=s["prior"], workspace=s["workspace"])
    elif s["op"] == "append":
        k, v = _append(s)
    else:
        return _read(s) if s["op"] == "read" else _attend(s)
    pools = ("k_pages", "v_pages") + (() if s["fmt"] == "bf16" else ("k_scales", "v_scales"))
    return [k, v] + [s[name] for name in pools]


# ------------------------------------------------------------------------------ the definition in 64 bits ---
def _two(e):
    """2^e in float64 from a table of Python's own powers (e: whole numbers within -400 .. 400)."""
    return torch.tensor([2.0 ** k for k in range(-400, 401)], dtype=torch.float64, device=e.device)[e.long() + 400]


def _floor_log2(x):
    """floor(log2(x)) of float64 x >= 2^-300, the logarithm's own rounding put right."""
    e = torch.floor(torch.log2(x))
    e = torch.where(_two(e) > x, e - 1, e)
    return torch.where(_two(e + 1) <= x, e + 1, e)


def _grid64(x, fmt):
    """x (float64) [..., 32 * groups] rounded onto its groups' code grids."""
    lowest, frac, top = (-6, 3, E4M3_MAX) if fmt == "mxfp8" else (0, 1, E2M1_MAX)
    g = x.reshape(*x.shape[:-1], -1, 32)
    amax = g.abs().amax(-1, keepdim=True)
    e = _floor_log2(amax.clamp(min=2.0 ** -300)) - _floor_log2(torch.tensor(top, dtype=torch.float64, device=x.device))
    e = torch.where(amax > top * _two(e), e + 1, e).clamp(-127, 127)
    u = g / _two(e)
    step = _two(_floor_log2(u.abs().clamp(min=2.0 ** -300)).clamp(min=lowest) - frac)
    return (torch.round(u / step) * step * _two(e)).reshape(x.shape)


def _values64(codes, scales, fmt):
    """The values of cache bytes, field by field."""
    if fmt == "bf16":
        return codes.contiguous().view(torch.bfloat16).double()
    c = codes.int() if fmt == "mxfp8" else torch.stack((codes.int() % 16, codes.int() // 16), -1).flatten(-2)
    sign_at, frac, bias = (7, 3, 7) if fmt == "mxfp8" else (3, 1, 1)
    ex = (c % (1 << sign_at)) >> frac
    mant = (c % (1 << frac)).double() / (1 << frac)
    u = torch.where(ex == 0, mant * 2.0 ** (1 - bias), (1 + mant) * _two(ex - bias))
    u = torch.where((c >> sign_at) == 1, -u, u)
    return u * _two(scales.int() - 127).repeat_interleave(32, -1)


def _pages_of(s, name, i, first, last):
    """The cache bytes of positions first .. last - 1 of sequence i: codes and scales, [heads, tokens, ...]."""
    ids = s["table"][i, first // s["page"]:(last - 1) // s["page"] + 1].long()
    skip = first % s["page"]
    return [s[name + part][ids].transpose(0, 1).flatten(1, 2)[:, skip:skip + last - first] for part in ("_pages", "_scales")]


def exact(case, seed):
    s = prepare(case, seed)
    fmt, lens, starts = s["fmt"], s["kv_lens"].tolist(), s["row_starts"].tolist()
    if s["op"] == "append":
        pools = 2 if fmt == "bf16" else 4
        both = [s[n].double() if fmt == "bf16" else _grid64(s[n].double(), fmt) for n in ("k", "v")]
        if fmt == "bf16":   # the cache's own rounding, to 8 significant bits
            step = [_two(_floor_log2(x.abs().clamp(min=2.0 ** -126)) - 7) for x in both]
            both = [torch.round(x / w) * w for x, w in zip(both, step)]
        return both + [None] * pools
    n = [b - a for a, b in zip(starts, starts[1:])]
    if s["op"] == "read":
        return [torch.cat([_values64(*_pages_of(s, name, i, lens[i] - n[i], lens[i]), fmt).transpose(0, 1)
                           for i in range(len(lens))]) for name in ("k", "v")]
    outs = []
    heads, G, dim = s["heads"], s["group"], s["dim"]
    for i, length in enumerate(lens):
        lo, hi = starts[i], starts[i + 1]
        K, V = (_values64(*_pages_of(s, name, i, 0, length), fmt) for name in ("k", "v"))
        before = length - n[i]
        words = s["tree"][lo:hi].tolist()
        seen = torch.tensor([[w >> j & 1 == 1 for j in range(n[i])] for w in words], device="cuda")
        got = []
        for h in range(heads * G):
            z = s["q"][lo:hi, h].double() @ K[h // G].T / dim ** 0.5
            z[:, before:][~seen] = -math.inf
            if s["prior"] is not None:   # the prior's tokens as one more, of weight l and value out
                po, pm, pl = (x[lo:hi, h].double() for x in s["prior"])
                m = torch.maximum(z.amax(1), pm)
                p, w = torch.exp(z - m[:, None]), pl * torch.exp(pm - m)
                l = p.sum(1) + w
                o = (p @ V[h // G] + w[:, None] * po) / l[:, None]
            else:
                m = z.amax(1)
                p = torch.exp(z - m[:, None])
                l = p.sum(1)
                o = p @ V[h // G] / l[:, None]
            got.append((o, m, l))
        outs.append([torch.stack(x, 1) for x in zip(*got)])
    return [torch.cat(x) for x in zip(*outs)]
