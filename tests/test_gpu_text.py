"""The text cache on the GPU against plain float64 (text_plain.py): appending, reading, attention, and a decode
step that joins them with the visual tokens' compressed attention.

Tolerances.  Codes, scale bytes and read values are exact.  In attention a score is summed by D / 16 matrix
instructions, each of which adds to a float32 with an error of at most one unit, 2^-23 of a sum that never exceeds
S = sum |q k| / sqrt(D); the query's lower terms, the change to log2 and the scaling add less than four more, so
  dz = (D / 16 + 4) 2^-23 S
bounds a score's error, and exp(z) is off by 2 dz (its own error and the maximum's).  Exponentials and sums of
at most 2^12 float32 terms (pairwise over lanes, warps and parts) stay within 2^-16.  So
  |out error| <= h_out |out| + (h_p + 2 dz + 2^-16) A + 2^-22 max|V|,   A = sum p |V| / sum p,
with h = eps / 2 of a type: h_out of the output, h_p of the probabilities as they multiply V (bfloat16 caches: 2^-8;
coded ones: half precision, 2^-11; float32 queries: split, below 2^-20); 2^-22 max|V| covers what half precision
drops below 2^-24 of its largest value.  |m error| <= dz + 2^-22 |m|, and |l error| <= (2 dz + 2^-16) l.
"""
import math

import numpy as np
import pytest
import torch

import text_plain as P
from oracle import tactkv_oracle as O
from dct_transform_coding_b200.workloads import make_unit

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from dct_transform_coding_b200 import tactkv as T

DEV = "cuda:0"
FMTS = ["bf16", "mxfp8", "mxfp4"]
# Calls bounded to 128 tokens and longer ones take different kernels (bfloat16 queries, head_dim 64, 128, 192, 256).
BOUNDS = [None, 2000]
IO = {"bf16": torch.bfloat16, "f32": torch.float32}


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Setup:
    """A filled cache of random pages, the batch arrays of sequences with (rows, length), and their values."""

    def __init__(self, fmt, heads, D, page, seqs, seed=0, extra_rows=0, scale=1.0, n_pages=None):
        gen = torch.Generator().manual_seed(seed)
        self.fmt, self.heads, self.D, self.page, self.seqs = fmt, heads, D, page, seqs
        width = max([1] + [-(-t // page) for _, t in seqs])
        used = sum(-(-t // page) for _, t in seqs)
        n_pages = n_pages or used + 2
        perm = torch.randperm(n_pages, generator=gen).tolist()
        self.table = [[-1] * width for _ in seqs]
        at = 0
        for row, (_, t) in zip(self.table, seqs):
            for i in range(-(-t // page)):
                row[i], at = perm[at], at + 1
        self.n_rows = sum(n for n, _ in seqs) + extra_rows
        self.cache = T.text_cache(fmt, n_pages, heads, D, page_tokens=page, device=DEV)
        self.gen = gen
        self.batch = (ints(self.table).reshape(len(seqs), width), ints([t for _, t in seqs]),
                      ints(np.concatenate(([0], np.cumsum([n for n, _ in seqs]))).tolist()))
        # every sequence's tokens, written through the same entry point
        total = sum(t for _, t in seqs)
        if total:
            k, v = (torch.randn((total, heads, D), generator=gen) * scale for _ in range(2))
            k[:, :, 1] *= 6
            ends = ints(np.concatenate(([0], np.cumsum([t for _, t in seqs]))).tolist())
            T.text_append(self.cache, k.to(DEV), v.to(DEV), self.batch[0], self.batch[1], ends, check=True)

    def values(self):
        """K and V of every sequence, [heads, length, D] float64."""
        pools = [P.held(self.cache, self.fmt, n) for n in ("k", "v")]
        return [[P.gather(pool, row, self.page, t) for pool in pools] for row, (_, t) in zip(self.table, self.seqs)]

    def starts(self):
        return self.batch[2].tolist()


def check_attention(s, G, io, tree=None, prior=False, q_scale=1.0, max_kv_len=None, call=None):
    dtype = IO[io]
    qh = s.heads * G
    q = (torch.randn((s.n_rows, qh, s.D), generator=s.gen) * q_scale).to(dtype)
    words = None
    if tree == "random":
        words = []
        for n, _ in s.seqs:
            mine = []
            for j in range(n):
                up = int(torch.randint(-1, j, (1,), generator=s.gen)) if j else -1
                mine.append(up)
            words.append(mine)
        words = T.text_tree(words, device=DEV)
        words = torch.cat((words, torch.zeros(s.n_rows - words.numel(), dtype=torch.int64, device=DEV)))
    elif tree is not None:
        words = tree
    pr = None
    if prior:
        pr = (torch.randn((s.n_rows, qh, s.D), generator=s.gen), 2 * torch.randn((s.n_rows, qh), generator=s.gen),
              50 * torch.rand((s.n_rows, qh), generator=s.gen))
        pr[1][0, 0], pr[2][0, 0], pr[0][0, 0] = -math.inf, 0.0, 0.0           # a prior that saw nothing
    out = torch.full((s.n_rows, qh, s.D), 77.0, dtype=dtype, device=DEV)
    got = (call or T.text_attention)(q.to(DEV), s.cache, *s.batch, max_rows=max([1] + [n for n, _ in s.seqs]),
                                     max_kv_len=max_kv_len, tree=words,
                                     prior=None if pr is None else tuple(x.to(DEV) for x in pr), out=out)
    torch.cuda.synchronize()
    verify(s, q, words, pr, got, io)
    return got


def verify(s, q, words, pr, got, io):
    out, m, l = (x.double().cpu().numpy() for x in got)
    h_out = torch.finfo(IO[io]).eps / 2
    h_p = 2.0 ** -20 if io == "f32" else (2.0 ** -8 if s.fmt == "bf16" else 2.0 ** -11)
    q = q.double().numpy()
    for i, ((n, t), (K, V)) in enumerate(zip(s.seqs, s.values())):
        lo = s.starts()[i]
        w = None if words is None else [x & (2 ** 64 - 1) for x in words[lo:lo + n].tolist()]
        p = None if pr is None else [x[lo:lo + n].double().numpy() for x in pr]
        ro, rm, rl, mag, S = P.attend(q[lo:lo + n], K, V, P.visible(n, t, w), p)
        sl = slice(lo, lo + n)
        big = np.max(np.abs(V[np.isfinite(V)]), initial=0.0)
        nan = np.isnan(rl)
        assert np.array_equal(np.isnan(l[sl]), nan)
        assert np.array_equal(np.isneginf(m[sl]), np.isneginf(rm))
        dz = (s.D / 16 + 4) * 2.0 ** -23 * S
        tol = h_out * np.abs(ro) + (h_p + 2 * dz + 2.0 ** -16)[..., None] * mag + 2.0 ** -22 * big
        with np.errstate(invalid="ignore"):
            bad = ~(np.abs(out[sl] - ro) <= tol) & np.isfinite(ro)
        bad[nan] = False
        assert not bad.any(), (i, np.argwhere(bad)[:4], out[sl][bad][:4], ro[bad][:4], tol[bad][:4])
        fin = np.isfinite(rm) & ~nan
        assert np.array_equal(np.isfinite(out[sl])[~nan], np.isfinite(ro)[~nan])
        assert (np.abs(m[sl][fin] - rm[fin]) <= dz[fin] + 2.0 ** -22 * np.abs(rm[fin])).all()
        assert (np.abs(l[sl] - rl)[~nan] <= ((2 * dz + 2.0 ** -16) * rl)[~nan]).all()
    end = s.starts()[-1]
    assert (got[0][end:] == 77.0).all()                  # rows behind the last sequence


# -------------------------------------------------------------------------------------- append, read ---
def special_rows(D, n):
    """Rows whose groups hold zeros, ties, the extremes of either type, infinities and NaN."""
    gen = torch.Generator().manual_seed(5)
    x = torch.randn((n, D), generator=gen).to(torch.bfloat16).float()
    x[0] = 0.0
    x[0, 1] = -0.0
    x[1] = torch.arange(D) * 0.25 - 4                    # many ties on either grid
    x[2] = 2.0 ** -133 * (torch.arange(D) % 13)          # bfloat16's subnormals
    x[3] = 3.3895e38 * (1 - 2 * (torch.arange(D) % 2))   # near its largest value
    x[4, 3] = math.inf
    x[5, D - 1] = math.nan
    x[6] = 448.0
    x[6, 0] = 450.0
    x[7] = 6.0
    x[7, 0] = 6.03125
    x[8] = torch.ldexp(torch.ones(D), -(torch.arange(D) % 40))
    return x


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("heads,D", [(1, 32), (3, 96), (2, 256), (5, 160)])
def test_append_and_read_are_exact(fmt, io, heads, D):
    n, page, dtype = 21, 16, IO[io]
    x = torch.stack([special_rows(D, n).roll(h, 0) for h in range(heads)], 1)
    if io == "f32":
        x[10:] += 1e-4 * torch.rand((n - 10, heads, D), generator=torch.Generator().manual_seed(1))
    k, v = x.to(dtype), (-x.flip(0)).to(dtype)
    cache = T.text_cache(fmt, 3, heads, D, page_tokens=page, device=DEV)
    for pool in (cache.k_pages, cache.v_pages) + ((cache.k_scales, cache.v_scales) if fmt != "bf16" else ()):
        pool.fill_(0x5A)
    batch = (ints([[2, 0]]), ints([n + 3]), ints([0, n]))
    kv, vv = T.text_append(cache, k.to(DEV), v.to(DEV), *batch, values=True, check=True)
    kr, vr = T.text_read(cache, *batch, n_rows=n, dtype=torch.float32, check=True)
    for name, src, val, rd in (("k", k, kv, kr), ("v", v, vv, vr)):
        want, scales = P.quantise(src.double().numpy(), fmt)
        with np.errstate(over="ignore"):
            as_f32 = torch.from_numpy(want).float()
        assert torch.equal(rd.cpu().nan_to_num(1.5), as_f32.nan_to_num(1.5))
        assert torch.equal(rd.cpu().isnan(), as_f32.isnan())
        assert torch.equal(val.cpu().nan_to_num(1.5), as_f32.to(dtype).nan_to_num(1.5))
        pool = getattr(cache, name + "_pages").cpu()
        tokens = [(2, t) if t < page else (0, t - page) for t in range(3, n + 3)]
        rows = torch.stack([pool[p, :, t] for p, t in tokens])
        if fmt != "bf16":
            got = np.stack([getattr(cache, name + "_scales").cpu().numpy()[p, :, t] for p, t in tokens])
            assert np.array_equal(got, scales)
            neg = torch.signbit(src) & torch.isfinite(as_f32)
            raw = rows if fmt == "mxfp8" else torch.stack((rows & 15, rows >> 4), -1).flatten(-2)
            bit = 7 if fmt == "mxfp8" else 3
            assert torch.equal((raw >> bit == 1)[torch.isfinite(as_f32)], neg[torch.isfinite(as_f32)])
        # no byte of another token
        mask = torch.ones(pool.shape[0], pool.shape[2], dtype=torch.bool)
        for p, t in tokens:
            mask[p, t] = False
        assert (pool.transpose(1, 2)[mask] == 0x5A).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("view", ["fused", "heads_first", "odd_base"])
def test_append_and_read_through_strides(fmt, dtype, view):
    heads, D, n = 3, 64, 19
    gen = torch.Generator(DEV).manual_seed(3)
    if view == "fused":                                   # one product's [rows, (q | k | v)] output
        x = torch.randn((n, 4 * heads, D), generator=gen, device=DEV).to(dtype)
        k, v = x[:, heads:2 * heads], x[:, 3 * heads:]
    elif view == "heads_first":
        k, v = (torch.randn((heads, n, D), generator=gen, device=DEV).to(dtype).transpose(0, 1) for _ in range(2))
    else:                                                 # two elements off a 16-byte boundary, rows of an even length
        x = torch.randn((2, n * (heads * D + 2) + 2), generator=gen, device=DEV).to(dtype)
        k, v = (y[2:].reshape(n, heads * D + 2)[:, :heads * D].unflatten(1, (heads, D)) for y in x)
        assert k.data_ptr() % 16
    caches = [T.text_cache(fmt, 4, heads, D, page_tokens=16, device=DEV) for _ in range(2)]
    batch = (ints([[1, 3], [0, -1]]), ints([17, 6]), ints([0, 14, 19]))
    a = T.text_append(caches[0], k, v, *batch, values=True, check=True)
    b = T.text_append(caches[1], k.contiguous(), v.contiguous(), *batch, values=True, check=True)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    assert torch.equal(caches[0].k_pages, caches[1].k_pages) and torch.equal(caches[0].v_pages, caches[1].v_pages)
    out = tuple(torch.full_like(x, 9.0) if view == "heads_first" else x.clone() for x in (k, v))
    if view == "odd_base":
        y = torch.zeros((2, n * (heads * D + 2) + 2), device=DEV, dtype=dtype)
        out = tuple(z[2:].reshape(n, heads * D + 2)[:, :heads * D].unflatten(1, (heads, D)) for z in y)
    got = T.text_read(caches[0], *batch, n_rows=n, dtype=dtype, out=out, check=True)
    for x, y in zip(got, a):
        assert torch.equal(x, y)
    if view == "odd_base":
        assert not y.dtype.is_complex and (out[0].storage_offset() == 2)


def test_rows_behind_the_last_sequence_and_errors():
    """Padded rows are left alone; rows that do not fit are skipped by append, zeroed by read, and reported."""
    heads, D, n = 2, 32, 8
    k = torch.randn((n, heads, D), device=DEV).bfloat16()
    for bad in ("length", "page", "page_big", "order", "short", "none"):
        cache = T.text_cache("mxfp8", 3, heads, D, page_tokens=16, device=DEV)
        table, lens, starts = [[0, -1], [1, 2]], [5, 20], [0, 2, 6]
        if bad == "length":
            lens[0] = 33                                  # more than two pages hold
        elif bad == "page":
            lens[0] = 17                                  # on the page -1
        elif bad == "page_big":
            table[0][0] = 3
        elif bad == "short":
            lens[0] = 1                                   # fewer tokens than rows
        elif bad == "order":
            starts = [0, 7, 6]
        batch = (ints(table), ints(lens), ints(starts))
        ws = T.text_workspace(cache, n_seqs=2, n_rows=n)
        out = tuple(torch.full((n, heads, D), 3.0, device=DEV).bfloat16() for _ in range(2))
        T.text_append(cache, k, k, *batch, workspace=ws)
        st = T.tactkv_device_status(ws.data_ptr(), ws.numel(), 0)
        assert st == (T.TACTKV_OK if bad == "none" else T.TACTKV_INVALID_ARG), bad
        T.text_read(cache, *batch, n_rows=n, out=out, workspace=ws)
        assert T.tactkv_device_status(ws.data_ptr(), ws.numel(), 0) == st
        if bad == "none":
            assert (out[0][:6] != 3.0).any(dim=(1, 2)).all()
        elif bad != "order":
            # a length of 17 puts one of the two rows on a good page
            assert not (out[0][1:2] if bad == "page" else out[0][:2]).any()
            assert (out[0][2:6] != 0).any(dim=(1, 2)).all()
        assert (out[0][7:] == 3.0).all() and (bad == "order" or (out[0][6:] == 3.0).all())


# ----------------------------------------------------------------------------------------- attention ---
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 224, 256])
def test_attention_head_dims(fmt, io, D):
    s = Setup(fmt, 2, D, 16, [(5, 40), (1, 1), (3, 150)], seed=D)
    check_attention(s, 3, io, tree="random", prior=True)


@pytest.mark.parametrize("fmt,io", [("bf16", "bf16"), ("mxfp8", "bf16"), ("mxfp4", "f32")])
@pytest.mark.parametrize("G,page,seqs,extra", [
    (1, 16, [(1, 1)], 0),
    (1, 64, [(1, n) for n in (1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129)], 3),
    (16, 32, [(1, 700), (4, 4), (0, 33), (2, 1000)], 2),
    (7, 128, [(64, 64), (64, 65), (33, 300), (0, 0), (17, 17)], 0),
    (2, 1024, [(63, 1500), (1, 3000)], 1),
    (3, 16, [(2, 5000)], 0),                              # split into parts
])
def test_attention_lengths_and_groups(fmt, io, G, page, seqs, extra):
    s = Setup(fmt, 2, 64, page, seqs, seed=G, extra_rows=extra)
    check_attention(s, G, io, tree="random", prior=False)
    check_attention(s, G, io, tree=None, prior=True)


@pytest.mark.parametrize("fmt,io", [("bf16", "bf16"), ("bf16", "f32"), ("mxfp8", "bf16"), ("mxfp4", "bf16")])
@pytest.mark.parametrize("D,G,rows", [(64, 8, 30), (128, 8, 63), (256, 2, 64), (128, 16, 16)])
def test_attention_wide_trees(fmt, io, D, G, rows):
    """Many rows to a K/V head, odd lengths, and sequences of other sizes in the same call."""
    s = Setup(fmt, 1, D, 64, [(rows, 777), (rows // 2, rows // 2 + 1), (1, 130), (rows - 3, 2051)], seed=rows, extra_rows=5)
    check_attention(s, G, io, tree="random", prior=True)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("prior", [False, True])
@pytest.mark.parametrize("rows", [3, 40])
@pytest.mark.parametrize("bound", BOUNDS)
def test_rows_that_see_nothing(fmt, prior, rows, bound):
    s = Setup(fmt, 2, 64, 16, [(rows, rows), (2, 20)], seed=8)
    words = torch.zeros(rows + 2, dtype=torch.int64, device=DEV)
    words[1] = 1
    out, m, l = check_attention(s, 8, "bf16", tree=words, prior=prior, max_kv_len=bound)
    if not prior:
        assert not out[0].any() and torch.isneginf(m[0]).all() and not l[0].any()
        assert not out[rows - 1].any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [6, 50])
@pytest.mark.parametrize("D,before,bound", [(64, 45, None), (64, 45, 2000), (128, 45, 2000), (256, 700, None), (192, 250, None)])
def test_infinities_and_nan_reach_only_the_rows_that_see_them(fmt, io, rows, D, before, bound):
    """K and V of drafted tokens, and whatever stands behind the last token, hold infinities and NaN."""
    s = Setup(fmt, 1, D, 32, [(rows, before + rows), (rows, 31 + rows)], seed=4)
    k, v = (torch.randn((2 * rows, 1, D)) for _ in range(2))
    k[2, 0, 5], v[3, 0, 40], v[4, 0, 0] = math.nan, math.inf, math.nan
    T.text_append(s.cache, k.to(DEV), v.to(DEV), *s.batch, check=True)
    for i, (_, t) in enumerate(s.seqs):                   # the rest of the last page
        page, off = s.table[i][(t - 1) // 32], (t - 1) % 32 + 1
        for pool in (s.cache.k_pages, s.cache.v_pages):
            pool[page, :, off:] = 0xFF                    # NaN in bfloat16 and in E4M3
        if fmt != "bf16":
            s.cache.k_scales[page, :, off:] = 255
            s.cache.v_scales[page, :, off:] = 255
    words = [1 << j for j in range(rows)]                 # every row sees itself alone
    words[5] |= 1 << 0
    out, m, l = check_attention(s, 4, io, tree=torch.tensor(words * 2, dtype=torch.int64, device=DEV),
                                max_kv_len=bound)
    assert torch.isnan(out[2]).all() and torch.isfinite(out[[0, 1, 5]]).all()
    assert not torch.isfinite(out[3, :, 40]).any() and torch.isnan(out[4, :, 0]).all()
    if fmt == "bf16":
        assert torch.isfinite(out[3, :, :40]).all() and torch.isfinite(out[4, :, 1:]).all()
    else:                                                 # the group reads back as NaN, the others as they were
        assert torch.isfinite(out[3, :, :32]).all() and torch.isfinite(out[4, :, 32:]).all()
        assert torch.isfinite(out[3, :, 64:]).all()
    assert torch.isfinite(out[rows:rows + 2]).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("scale,q_scale", [(1e-20, 1e18), (3e4, 1e-4), (1.0, 20.0), (1e15, 1e-17)])
@pytest.mark.parametrize("bound", BOUNDS)
def test_far_ranges(fmt, scale, q_scale, bound):
    """K and V, and the queries against them, far from 1; and scores sharp enough for a one-hot softmax."""
    s = Setup(fmt, 2, 64, 16, [(4, 90), (1, 33)], seed=2, scale=scale)
    check_attention(s, 2, "bf16", q_scale=q_scale, max_kv_len=bound)
    check_attention(s, 2, "f32", q_scale=q_scale, max_kv_len=bound)


def test_scales_of_very_different_size_in_one_sequence():
    """Tokens whose V is 2^20 times another's: the largest scale seen so far moves late."""
    s = Setup("mxfp8", 1, 128, 16, [(1, 600)], seed=6)
    k, v = (torch.randn((600, 1, 128)) for _ in range(2))
    v *= torch.ldexp(torch.ones(600), torch.arange(600) // 30)[:, None, None]
    T.text_append(s.cache, k.to(DEV), v.to(DEV), s.batch[0], s.batch[1], ints([0, 600]), check=True)
    check_attention(s, 4, "bf16")
    check_attention(s, 4, "f32")


def test_offsets_beyond_32_bits():
    """Pools of over 2^32 bytes each, the sequence's pages at their end."""
    n_pages, page, heads, D = 2200, 1024, 4, 256
    k = torch.empty((n_pages, heads, page, D * 2), dtype=torch.uint8, device=DEV)
    v = torch.empty_like(k)
    assert k.numel() > 2 ** 32
    cache = T.TextCache("bf16", k, v)
    table, t, n = [n_pages - 1, n_pages - 3, n_pages - 2], 2100, 2100
    x = torch.randn((n, heads, D), generator=torch.Generator(DEV).manual_seed(1), device=DEV).bfloat16()
    batch = (ints([table]), ints([t]), ints([0, n]))
    T.text_append(cache, x, -x, *batch, check=True)
    kr, vr = T.text_read(cache, *batch, n_rows=n, check=True)
    assert torch.equal(kr, x) and torch.equal(vr, -x)
    q = torch.randn((1, heads, D), generator=torch.Generator(DEV).manual_seed(2), device=DEV).bfloat16()
    out, m, l = T.text_attention(q, cache, batch[0], batch[1], ints([0, 1]), max_rows=1, check=True)
    s = torch.einsum("qhd,thd->ht", q.double(), x.double()) / 16
    ref = torch.einsum("ht,thd->hd", torch.softmax(s, 1), -x.double())
    mag = torch.einsum("ht,thd->hd", torch.softmax(s, 1), x.double().abs())
    assert ((out[0].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -15) * mag).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("before", [0, 640])
def test_attention_reports_bad_rows_and_pages(fmt, before):
    """Rows that do not fit see no text token, a bad page's tokens are left out, other sequences are as ever.  (before:
    so many more tokens in front, for the kernel of long sequences.)"""
    heads, D = 1, 64
    for bad in ("page", "length", "rows", "max_len", "none"):
        s = Setup(fmt, heads, D, 16, [(2, before + 40), (1, before + 20)], seed=1)
        table, lens, max_rows, max_len = s.batch[0].clone(), s.batch[1].clone(), 2, before + 48
        if bad == "page":
            table[0, 1] = s.cache.n_pages
            table[0, before // 16] = -5
        elif bad == "length":
            lens[0] = 1
        elif bad == "rows":
            max_rows = 1
        elif bad == "max_len":
            max_len = before + 39
        q = torch.randn((3, 2, D), device=DEV).bfloat16()
        ws = T.text_workspace(s.cache, n_seqs=2, n_rows=3, max_rows=2, q_heads=2, max_kv_len=before + 48)
        out, m, l = T.text_attention(q, s.cache, table, lens, s.batch[2], max_rows=max_rows, max_kv_len=max_len, workspace=ws)
        assert T.tactkv_device_status(ws.data_ptr(), ws.numel(), 0) == (T.TACTKV_OK if bad == "none" else T.TACTKV_INVALID_ARG)
        ref = T.text_attention(q, s.cache, *s.batch, max_rows=2, max_kv_len=before + 48)
        assert torch.equal(out[2], ref[0][2])             # the other sequence
        if bad == "none":
            assert torch.equal(out, ref[0])
        elif bad == "page":                               # two pages' tokens are left out
            K, V = s.values()[0]
            seen = P.visible(2, before + 40, None)
            seen[:, 16:32] = False
            seen[:, before:before + 16] = False
            o, _, rl, mag, S = P.attend(q[:2].double().cpu().numpy(), K, V, seen)
            dz = (D / 16 + 4) * 2.0 ** -23 * S
            assert np.all(np.abs(l[:2].cpu().numpy() - rl) <= (2 * dz + 2.0 ** -16) * rl)
            tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2 * dz + 2.0 ** -16)[..., None] * mag + 2.0 ** -22 * np.max(np.abs(V))
            assert np.all(np.abs(out[:2].double().cpu().numpy() - o) <= tol)
        else:
            assert not out[:2].any() and torch.isneginf(m[:2]).all() and not l[:2].any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,G,rows,page", [(64, 2, 5, 16), (128, 4, 4, 256), (128, 8, 9, 64), (192, 5, 4, 32), (256, 4, 4, 128)])
def test_long_sequences_in_parts(fmt, D, G, rows, page):
    """Sequences that are split over blocks, ragged, beside short ones; the same bits every time."""
    s = Setup(fmt, 2, D, page, [(rows, 6000), (1, 1), (rows, 2900), (2, 129), (0, 50), (rows, 300)], seed=D + page, extra_rows=2)
    first = check_attention(s, G, "bf16", tree="random", prior=True)
    q = torch.randn((s.n_rows, 2 * G, D), device=DEV).bfloat16()
    runs = [T.text_attention(q, s.cache, *s.batch, max_rows=rows, out=torch.zeros_like(q)) for _ in range(4)]
    assert first[0].shape == q.shape
    for r in runs[1:]:
        end = s.starts()[-1]
        assert all(torch.equal(a[:end], b[:end]) for a, b in zip(runs[0], r))


def test_many_sequences():
    """More sequences than blocks fit the GPU at once, lengths from 1 to 700, and one row each."""
    lens = [1 + (i * 37) % 700 for i in range(500)]
    for fmt in FMTS:
        s = Setup(fmt, 1, 64, 64, [(1, t) for t in lens], seed=3, extra_rows=1)
        check_attention(s, 4, "bf16", prior=True)


@pytest.mark.parametrize("fmt,D", [("bf16", 128), ("mxfp8", 256), ("mxfp4", 256), ("mxfp8", 96)])
def test_offsets_past_32_bits(fmt, D):
    """A pool of more than 2^32 bytes (2^31 elements at the least), its last pages and first ones in use, against a
    small pool with the same contents."""
    heads, page, pages = 8, 64, 5 + 2 ** 32 // (8 * 64 * D * {"bf16": 2, "mxfp8": 1, "mxfp4": 1}[fmt])
    small = Setup(fmt, heads, D, page, [(4, 333)], seed=1, n_pages=6)
    row = T.text_cache(fmt, 1, heads, D, page_tokens=page, device=DEV)
    shape = (pages, *row.k_pages.shape[1:])
    pools = [torch.empty(shape, dtype=torch.uint8, device=DEV) for _ in range(2)]
    if fmt != "bf16":
        pools += [torch.empty((pages, *row.k_scales.shape[1:]), dtype=torch.uint8, device=DEV) for _ in range(2)]
    big = T.TextCache(fmt, *pools)
    order = [pages - 1, 0, pages - 3, 2, pages - 2, 1]
    table = ints([order])
    k, v = T.text_read(small.cache, small.batch[0], small.batch[1], ints([0, 333]), n_rows=333, dtype=torch.float32)
    T.text_append(big, k, v, table, small.batch[1], ints([0, 333]), check=True)
    q = torch.randn((4, 2 * heads, D), device=DEV).bfloat16()
    want = T.text_attention(q, small.cache, *small.batch, max_rows=4, check=True)
    got = T.text_attention(q, big, table, *small.batch[1:], max_rows=4, check=True)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    again = T.text_read(big, table, small.batch[1], ints([0, 333]), n_rows=333, dtype=torch.float32, check=True)
    assert torch.equal(again[0], k) and torch.equal(again[1], v)


@pytest.mark.parametrize("layout", ["token", "head", "gaps", "expanded"])
def test_read_into_strided_outputs(layout):
    s = Setup("mxfp4", 3, 64, 16, [(5, 40), (2, 7)], seed=8)
    n = s.n_rows
    k, v = T.text_read(s.cache, *s.batch, n_rows=n)
    make = {"token": lambda: torch.empty((n, 3, 64), device=DEV, dtype=torch.bfloat16),
            "head": lambda: torch.empty((3, n, 64), device=DEV, dtype=torch.bfloat16).transpose(0, 1),
            "gaps": lambda: torch.empty((n, 3, 2, 64), device=DEV, dtype=torch.bfloat16)[:, :, 0],
            "expanded": lambda: torch.empty((n, 1, 64), device=DEV, dtype=torch.bfloat16).expand(n, 3, 64)}[layout]
    out = (make(), make())
    if layout == "expanded":                              # every head would be written to the same place
        with pytest.raises(T.TactkvError):
            T.text_read(s.cache, *s.batch, n_rows=n, out=out)
        return
    T.text_read(s.cache, *s.batch, n_rows=n, out=out)
    assert torch.equal(out[0], k) and torch.equal(out[1], v)


# ------------------------------------------------------------------------------------- as it is used ---
def test_other_stream_and_captured_graph():
    """Calls on a stream of their own, and a captured step replayed on other lengths, pages and rows."""
    s = Setup("mxfp8", 2, 64, 16, [(2, 60), (2, 200)], seed=9)
    q = torch.randn((4, 4, 64), device=DEV).bfloat16()
    k = torch.randn((4, 2, 64), device=DEV).bfloat16()
    stream = torch.cuda.Stream(DEV)
    stream.wait_stream(torch.cuda.current_stream())
    table, lens, starts = (x.clone() for x in s.batch)
    ws = T.text_workspace(s.cache, n_seqs=2, n_rows=4, max_rows=3, q_heads=4, max_kv_len=256)
    torch.cuda.synchronize()

    def step():
        T.text_append(s.cache, k, k, table, lens, starts, workspace=ws, stream=stream)
        return T.text_attention(q, s.cache, table, lens, starts, max_rows=3, max_kv_len=256, workspace=ws, stream=stream)

    first = step()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, got))
    lens.copy_(ints([57, 177]))                           # a replay on other lengths and rows
    starts.copy_(ints([0, 1, 4]))
    k.normal_(), q.normal_()
    graph.replay()
    torch.cuda.synchronize()
    replayed = [x.clone() for x in got]
    want = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, replayed))
    s.seqs = [(1, 57), (3, 177)]
    s.batch = (table, lens, starts)
    verify(s, q.cpu(), None, None, want, "bf16")


@pytest.mark.parametrize("fmt", FMTS)
def test_captured_graph_of_split_sequences(fmt):
    """A captured call whose sequences are split over blocks, replayed on other lengths."""
    s = Setup(fmt, 2, 128, 64, [(3, 3000), (2, 2500)], seed=2)
    q = torch.randn((5, 8, 128), device=DEV).bfloat16()
    table, lens, starts = (x.clone() for x in s.batch)
    ws = T.text_workspace(s.cache, n_seqs=2, n_rows=5, max_rows=3, q_heads=8, max_kv_len=3008)
    kw = dict(max_rows=3, max_kv_len=3008, workspace=ws)
    T.text_attention(q, s.cache, table, lens, starts, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [T.text_attention(q, s.cache, table, lens, starts, **kw) for _ in range(3)]
    for new in ([3000, 2500], [700, 2499], [129, 64]):
        lens.copy_(ints(new))
        graph.replay()
        torch.cuda.synchronize()
        replayed = [[x.clone() for x in g] for g in got]
        want = T.text_attention(q, s.cache, table, lens, starts, **kw)
        torch.cuda.synchronize()
        for g in replayed:
            assert all(torch.equal(a, b) for a, b in zip(want, g))
    assert T.tactkv_device_status(ws.data_ptr(), ws.numel(), 0) == T.TACTKV_OK


def test_two_calls_at_once():
    """Two streams, a workspace each, the same cache: the results of calls one after another."""
    s = Setup("mxfp4", 2, 128, 32, [(3, 900), (2, 1500)], seed=3)
    q = [torch.randn((5, 8, 128), device=DEV).bfloat16() for _ in range(2)]
    want = [T.text_attention(x, s.cache, *s.batch, max_rows=3) for x in q]
    streams = [torch.cuda.Stream(DEV) for _ in q]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [T.text_attention(x, s.cache, *s.batch, max_rows=3, stream=st) for x, st in zip(q, streams)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_step_with_visual_and_text_tokens(fmt):
    """A request's decode step as a user runs it: the visual K/V compressed, the text prompt appended, then
    a tree of drafted tokens appended, attended over both and, once the accepted path is known, written again at
    its place.  Against one softmax over the visual tokens (decompressed by the oracle) and the text's."""
    S, H, W, heads, D, G, bits = 8, 8, 8, 2, 64, 4, 2
    vis = [make_unit(S, H, W, heads, D, rho=(0.9, 0.85, 0.85), nu=4.0, seed=i, device=DEV)[None] for i in range(2)]
    pay = [T.compress(x, S, H, W, bits, layers=[0], kvs=[i]) for i, x in enumerate(vis)]
    cache = T.text_cache(fmt, 8, heads, D, page_tokens=16, device=DEV)
    table = ints([[5, 2, 7]])
    gen = torch.Generator(DEV).manual_seed(2)

    def rows(n):
        return [torch.randn((n, heads, D), generator=gen, device=DEV).bfloat16() for _ in range(2)]

    prompt = rows(29)
    T.text_append(cache, *prompt, table, ints([29]), ints([0, 29]), check=True)
    parents = [-1, 0, 0, 1, 2, 4]
    n = len(parents)
    draft = rows(n)
    T.text_append(cache, *draft, table, ints([29 + n]), ints([0, n]), check=True)
    q = torch.randn((n, heads * G, D), generator=gen, device=DEV)
    # the visual part: every drafted token is one more unit over the same payloads
    prior = T.attention_decode(q, pay[0].expand(n, -1), pay[1].expand(n, -1), S, H, W, bits, heads=heads, head_dim=D,
                               layers=[0] * n, check=True)
    out, m, l = T.text_attention(q, cache, table, ints([29 + n]), ints([0, n]), max_rows=n,
                                 tree=T.text_tree([parents], device=DEV), prior=prior, check=True)
    from_oracle = [O.decompress_unit(p[0].cpu().numpy().tobytes()) for p in pay]
    text = [P.gather(P.held(cache, fmt, name), table[0].tolist(), 16, 29 + n) for name in ("k", "v")]
    K, V = [np.concatenate((np.asarray(a).reshape(S * H * W, heads, D).transpose(1, 0, 2), b), axis=1)
            for a, b in zip(from_oracle, text)]
    words = [int(w) for w in T.text_tree([parents], device="cpu")]
    seen = np.concatenate((np.ones((n, S * H * W), bool), P.visible(n, 29 + n, words)), axis=1)
    ro, rm, rl, _, _ = P.attend(q.double().cpu().numpy(), K, V, seen)
    # the visual partial's own tolerance: 1e-4 of the largest output, and on m and l
    assert np.max(np.abs(out.double().cpu().numpy() - ro)) <= 2e-4 * np.max(np.abs(ro))
    assert np.allclose(m.cpu().numpy(), rm, rtol=1e-4, atol=1e-4) and np.allclose(l.cpu().numpy(), rl, rtol=1e-3)
    # nodes 0, 2, 4 are accepted: their rows are written again behind the prompt
    path = [0, 2, 4]
    T.text_append(cache, *[x[path] for x in draft], table, ints([32]), ints([0, 3]), check=True)
    kr, vr = T.text_read(cache, table, ints([32]), ints([0, 32]), n_rows=32, check=True)
    for got, a, b in ((kr, prompt[0], draft[0]), (vr, prompt[1], draft[1])):
        want, _ = P.quantise(torch.cat((a, b[path])).double().cpu().numpy(), fmt)
        assert np.array_equal(got.double().cpu().numpy(), want)
