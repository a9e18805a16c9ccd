"""The text cache's attention where magnitudes differ by more than half precision holds, on the GPU against float64.

Tolerances.  As in test_gpu_text.py a score is off by at most dz = (D / 16 + 4) 2^-23 S, S = sum |q k| / sqrt(D), its
exponential by 2 dz, and exponentials and float32 sums stay within 2^-16.  The probabilities multiply V as bfloat16 terms,
each of which leaves at most half a step, 2^-8, of the one before: one term for bfloat16 caches (h_p = 2^-8), two for coded
ones (2^-16), three for float32 queries (2^-24).  A coded value is a bfloat16 exactly.  So
  |out error| <= h_out |out| + (h_p + 2 dz + 2^-16) A,   A = sum p |V| / sum p over the tokens that the row sees,
with no term for values that the row does not see, for other columns', or for tokens of no weight.  (2^-126 stands for what
float32 drops below its smallest value.)
"""
import math

import numpy as np
import pytest
import torch

import text_plain as P

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from dct_transform_coding_b200 import tactkv as T
    from test_gpu_text import Setup, ints

DEV = "cuda:0"
FMTS = ["bf16", "mxfp8", "mxfp4"]
IO = {"bf16": torch.bfloat16, "f32": torch.float32}
# (type, head_dim, tokens before the drafted ones, max_kv_len): short calls, head_dims that are not a multiple of 64, and
# float32 queries take one kernel, the last four the other.  700 tokens of one sequence are split over blocks.
CALLS = [("bf16", 64, 45, None), ("bf16", 96, 300, None), ("f32", 64, 45, None), ("f32", 128, 45, 2000), ("f32", 256, 700, None),
         ("bf16", 64, 45, 2000), ("bf16", 128, 45, 2000), ("bf16", 256, 700, None), ("bf16", 192, 250, None)]


def compare(fmt, D, io, got, ref, what=""):
    """(out, m, l) of some rows against attend()'s, elementwise, with the tolerance above; every finite value of it."""
    (out, m, l), (ro, rm, rl, A, S) = got, ref
    h_out = torch.finfo(IO[io]).eps / 2
    h_p = 2.0 ** -24 if io == "f32" else (2.0 ** -8 if fmt == "bf16" else 2.0 ** -16)
    dz = (D / 16 + 4) * 2.0 ** -23 * S
    fin = np.isfinite(rl)
    assert np.array_equal(np.isfinite(l), fin), what
    assert np.array_equal(np.isneginf(m), np.isneginf(rm)), what
    some = np.isfinite(rm)
    assert (np.abs(m[some] - rm[some]) <= dz[some] + 2.0 ** -22 * np.abs(rm[some])).all(), what
    assert (np.abs(l - rl)[fin] <= ((2 * dz + 2.0 ** -16) * rl)[fin]).all(), what
    tol = h_out * np.abs(ro) + (h_p + 2 * dz + 2.0 ** -16)[..., None] * A + 2.0 ** -126
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(out - ro) <= tol) & np.isfinite(ro)
    assert not bad.any(), (what, np.argwhere(bad)[:4], out[bad][:4], ro[bad][:4], tol[bad][:4])
    assert np.array_equal(np.isfinite(out), np.isfinite(ro)), what


def strict(s, q, words, got, io):
    out, m, l = (x.double().cpu().numpy() for x in got)
    q = q.double().cpu().numpy()
    for i, ((n, t), (K, V)) in enumerate(zip(s.seqs, s.values())):
        lo = s.starts()[i]
        w = None if words is None else [int(x) & (2 ** 64 - 1) for x in words[lo:lo + n]]
        sl = slice(lo, lo + n)
        compare(s.fmt, s.D, io, (out[sl], m[sl], l[sl]), P.attend(q[sl], K, V, P.visible(n, t, w)), i)


def fill(s, k, v):
    """Every sequence's tokens, in order, written over what the setup wrote."""
    ends = np.concatenate(([0], np.cumsum([t for _, t in s.seqs]))).tolist()
    T.text_append(s.cache, k.to(DEV), v.to(DEV), s.batch[0], s.batch[1], ints(ends), check=True)


def attend(s, q, words=None, bound=None, **kw):
    tree = None if words is None else torch.tensor(words, dtype=torch.int64, device=DEV)
    return T.text_attention(q.to(DEV), s.cache, *s.batch, max_rows=max(n for n, _ in s.seqs), max_kv_len=bound, tree=tree,
                            check=True, **kw)


# ------------------------------------------------------------------- values that a row does not see or weigh ---
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("far", [30, 100])
@pytest.mark.parametrize("io,D,before,bound", CALLS)
def test_large_values_of_unseen_drafts_reach_no_row(fmt, io, far, D, before, bound):
    """Drafted tokens whose V is 2^30 or 2^100 times the others', each seen by its own row alone."""
    rows, G = 6, 4
    s = Setup(fmt, 1, D, 32, [(rows, before + rows)], seed=4)
    t = before + rows
    k, v = (torch.randn((t, 1, D), generator=s.gen) for _ in range(2))
    v[before + 2] *= 2.0 ** far
    v[before + 4] *= 2.0 ** (far - 7)
    fill(s, k, v)
    words = [1 << j for j in range(rows)]
    words[5] |= 1
    q = torch.randn((rows, G, D), generator=s.gen).to(IO[io])
    strict(s, q, words, attend(s, q, words, bound), io)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("io,D,before,bound", CALLS)
def test_large_values_of_no_weight(fmt, io, D, before, bound):
    """A token that every row sees, with V 2^40 times the others' and a probability below e^-60."""
    rows, G = 3, 2
    s = Setup(fmt, 1, D, 16, [(rows, before + rows)], seed=5)
    t = before + rows
    k, v = (torch.randn((t, 1, D), generator=s.gen) for _ in range(2))
    q = torch.randn((rows, G, D), generator=s.gen)
    q[..., 0] = 4.0
    k[7, 0] = 0.0
    k[7, 0, 0] = -30.0 * math.sqrt(D)                     # a score of -120
    v[7] *= 2.0 ** 40
    fill(s, k, v)
    q = q.to(IO[io])
    strict(s, q, None, attend(s, q, None, bound), io)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("step", [-20, -30, 12])
@pytest.mark.parametrize("io,D,before,bound", CALLS)
def test_groups_of_a_token_far_apart(fmt, io, step, D, before, bound):
    """Each group of 32 columns of V is 2^step times the one before; the queries live in the smallest group of K."""
    rows, G = 4, 2
    s = Setup(fmt, 1, D, 16, [(rows, before + rows)], seed=6)
    t = before + rows
    k, v = (torch.randn((t, 1, D), generator=s.gen) for _ in range(2))
    factor = torch.ldexp(torch.ones(D), (torch.arange(D) // 32).clamp(max=3) * step)
    v *= factor
    k *= factor
    small = factor == factor.min()
    q = torch.where(small, torch.randn((rows, G, D), generator=s.gen) / factor, 0.0)
    fill(s, k, v)
    q = q.to(IO[io])
    strict(s, q, None, attend(s, q, None, bound), io)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("io,D,before,bound", CALLS)
def test_values_near_the_largest(fmt, io, D, before, bound):
    """V of one sign up to 2.5e38, whose sums pass float32's range, and a late token of most of the weight whose score is
    not far enough above the others' for the running maximum to follow it at once."""
    rows, G = 3, 2
    s = Setup(fmt, 1, D, 16, [(rows, before + rows)], seed=7)
    t = before + rows
    k, v = (torch.randn((t, 1, D), generator=s.gen) for _ in range(2))
    v = 2.5e38 * (0.5 + 0.5 * torch.rand((t, 1, D), generator=s.gen))
    q = torch.randn((rows, G, D), generator=s.gen)
    q[..., 0] = 4.0
    k[..., 0] = 0.0
    k[t - rows - 1] = 0.0
    k[t - rows - 1, 0, 0] = 2.0 * math.sqrt(D)            # a score of 8 beside others of about 1
    fill(s, k, v)
    q = q.to(IO[io])
    strict(s, q, None, attend(s, q, None, bound), io)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,before,bound", [(64, 45, None), (128, 300, 2000)])
def test_queries_near_the_largest(fmt, D, before, bound):
    """float32 queries above bfloat16's largest value, against a group of K near its smallest."""
    rows, G = 3, 2
    s = Setup(fmt, 1, D, 16, [(rows, before + rows)], seed=8)
    k, v = (torch.randn((before + rows, 1, D), generator=s.gen) for _ in range(2))
    k[..., :32] *= 1e-37
    fill(s, k, v)
    q = torch.randn((rows, G, D), generator=s.gen)
    q[..., 3] = 3.4e38
    q[0, 1, 9] = -3.4e38
    strict(s, q, None, attend(s, q, None, bound), "f32")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("with_prior", [False, True])
@pytest.mark.parametrize("io,D,before,bound", CALLS)
def test_maxima_of_infinite_scores(fmt, with_prior, io, D, before, bound):
    """m is the scores' maximum, +inf or NaN among them; l and out of such a row are NaN, other rows are as ever."""
    rows, G = 6, 2
    s = Setup(fmt, 1, D, 16, [(rows, before + rows)], seed=9)
    t = before + rows
    k, v = (torch.randn((t, 1, D), generator=s.gen) for _ in range(2))
    k[..., 3] = 1.0 + torch.rand((t, 1), generator=s.gen)
    k[..., 4] = torch.where(torch.arange(t) % 40 == 39, 1.0, -1.0)[:, None]
    fill(s, k, v)
    q = torch.randn((rows, G, D), generator=s.gen)
    q[0, :, 3] = math.inf                                 # every score +inf
    q[1, :, 3] = -math.inf                                # every score -inf
    q[2, 1, 4] = math.inf                                 # some +inf, the others -inf
    q[3, 0, 7] = math.nan
    q = q.to(IO[io])
    prior = None
    if with_prior:
        prior = (torch.randn((rows, G, D), generator=s.gen), torch.randn((rows, G), generator=s.gen),
                 1 + torch.rand((rows, G), generator=s.gen))
    got = attend(s, q, None, bound, prior=None if prior is None else tuple(x.to(DEV) for x in prior))
    K, V = s.values()[0]
    ro, rm, rl, _, _ = P.attend(q.double().numpy(), K, V, P.visible(rows, t, None),
                                None if prior is None else [x.double().numpy() for x in prior])
    out, m, l = (x.double().cpu().numpy() for x in got)
    assert np.isposinf(rm[0]).all() and np.isposinf(rm[2, 1]) and np.isnan(rm[3, 0])
    for test in (np.isnan, np.isposinf, np.isneginf):
        assert np.array_equal(test(m), test(rm))
    assert np.array_equal(np.isnan(l), np.isnan(rl)) and np.array_equal(np.isnan(out), np.isnan(ro))
    fin = np.isfinite(rm)
    assert np.allclose(m[fin], rm[fin], rtol=1e-3, atol=1e-3) and np.allclose(out[fin], ro[fin], rtol=2e-2, atol=2e-2)


# ------------------------------------------------------------------------------------ many tiles in one block ---
class Crowd:
    """160 sequences over one K/V head that read the same pages, so many that none is split and a block walks through all
    of its tokens, 128 at a time; their lengths differ."""

    def __init__(self, fmt, D, rows, G, T_max, page=64, seed=1):
        self.s = s = Setup(fmt, 1, D, page, [(rows, T_max)], seed=seed)
        self.rows, self.G, self.n, self.T = rows, G, 160, T_max
        self.lens = [T_max - 61 * (i % 9) for i in range(self.n)]
        self.starts = ints([rows * i for i in range(self.n + 1)])
        self.k, self.v = (torch.randn((T_max, 1, D), generator=s.gen) for _ in range(2))
        self.q = torch.randn((rows * self.n, G, D), generator=s.gen).bfloat16()

    def run(self, words=None, bad_pages=()):
        """Attention of every sequence; three of each length's are checked, with bad_pages' tokens unseen."""
        s, rows = self.s, self.rows
        fill(s, self.k, self.v)
        table = s.batch[0].repeat(self.n, 1)
        for i, page in enumerate(bad_pages):
            table[:, page] = (-1, s.cache.n_pages, 1 << 30, -(1 << 31))[i % 4]
        ws = T.text_workspace(s.cache, n_seqs=self.n, n_rows=rows * self.n, max_rows=rows, q_heads=self.G, max_kv_len=self.T)
        tree = None if words is None else torch.tensor(words * self.n, dtype=torch.int64, device=DEV)
        got = T.text_attention(self.q.to(DEV), s.cache, table, ints(self.lens), self.starts, max_rows=rows, max_kv_len=self.T,
                               tree=tree, workspace=ws)
        status = T.tactkv_device_status(ws.data_ptr(), ws.numel(), 0)
        assert status == (T.TACTKV_INVALID_ARG if bad_pages else T.TACTKV_OK)
        out, m, l = (x.double().cpu().numpy() for x in got)
        K, V = s.values()[0]
        for i in list(range(9)) + [77, self.n - 1]:
            t, sl = self.lens[i], slice(rows * i, rows * (i + 1))
            seen = P.visible(rows, t, None if words is None else [w & (2 ** 64 - 1) for w in words])
            for page in bad_pages:
                seen[:, page * s.page:(page + 1) * s.page] = False
            ref = P.attend(self.q[sl].double().numpy(), K[:, :t], V[:, :t], seen)
            compare(s.fmt, s.D, "bf16", (out[sl], m[sl], l[sl]), ref, i)


# (head_dim, rows, query heads to a K/V head): units of 16, 32 and 64 rows; the first on the other kernel
CROWDS = [(96, 4, 4), (64, 2, 5), (64, 8, 8), (128, 4, 4), (128, 3, 8), (128, 7, 8), (192, 4, 4), (192, 5, 6), (256, 1, 16), (256, 5, 4)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,rows,G", CROWDS)
@pytest.mark.parametrize("kind", ["grow", "shrink", "climb"])
def test_values_and_scores_that_change_from_tile_to_tile(fmt, D, rows, G, kind):
    """V that grows or shrinks by 2^9 with each tile; scores that rise, so that the references move in most tiles."""
    c = Crowd(fmt, D, rows, G, 1500)
    tile = torch.arange(1500) // 128
    if kind == "climb":
        c.q[..., 0] = 4.0
        c.k[:, 0, 0] = torch.arange(1500) * (20.0 / 1500) * math.sqrt(D)      # scores from 0 to 80
    else:
        c.v *= torch.ldexp(torch.ones(1500), (9 if kind == "grow" else -9) * tile)[:, None, None]
    c.run()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,rows,G", CROWDS)
@pytest.mark.parametrize("drafts", ["plain", "odd"])
def test_bad_pages_in_many_tiles(fmt, D, rows, G, drafts):
    """Pages out of range in tiles 0, 3, 17 and the last one; drafted tokens, each its own row's alone, with infinities and
    NaN in their V."""
    c = Crowd(fmt, D, rows, G, 2650 + rows)
    words = [1 << j for j in range(rows)]
    if drafts == "odd":
        c.lens = [c.T] * c.n                              # (a shorter sequence's drafts would be a longer one's past)
        c.v[c.T - 1, 0, 33] = math.inf
        c.v[c.T - rows, 0, 5] = math.nan
    c.run(words, bad_pages=(0, 7, 34, 40))


# ------------------------------------------------------------------------------------- arguments as they come ---
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_from_an_odd_element(fmt, dtype):
    """k and v as views that start at an odd element of their storage, or have strides that differ."""
    n, heads, D = 5, 2, 64
    s = Setup(fmt, heads, D, 16, [(n, 20)], seed=3)
    k, v = (torch.randn((n, heads, D), generator=s.gen).to(DEV).to(dtype) for _ in range(2))
    want = T.text_append(s.cache, k, v, *s.batch, values=True, check=True)

    def odd(x):
        flat = torch.empty(x.numel() + 1, dtype=dtype, device=DEV)[1:]
        return flat.view(x.shape).copy_(x)

    assert odd(k).data_ptr() % (2 * k.element_size())
    for a, b in ((odd(k), odd(v)), (k, odd(v)), (odd(k), v), (k.transpose(0, 1).contiguous().transpose(0, 1), v)):
        got = T.text_append(s.cache, a, b, *s.batch, values=True, check=True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(ValueError):
        T.text_read(s.cache, *s.batch, n_rows=n, out=(odd(k), odd(v)))
