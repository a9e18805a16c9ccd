"""The text cache's host side without a GPU: sizes, refusals and the tree words (no kernel is launched)."""
import pytest

import text_plain as P
import numpy as np


@pytest.fixture(scope="module")
def T():
    from dct_transform_coding_b200 import tactkv
    return tactkv


def cache(T, **kw):
    d = dict(format=T.TACTKV_TEXT_MXFP8, heads=2, head_dim=64, page_tokens=16, n_pages=4, k_pages=4096, v_pages=8192,
             k_scales=16384, v_scales=32768)
    d.update(kw)
    return bytes(T.tactkv_text_cache(**d))


def batch(T, **kw):
    d = dict(page_table=4096, kv_lens=4096, row_starts=4096, n_seqs=1, n_rows=1, max_pages=2)
    d.update(kw)
    return bytes(T.tactkv_text_batch(**d))


BAD_CACHE = [
    (dict(format=3), "TACTKV_INVALID_ARG"), (dict(format=-1), "TACTKV_INVALID_ARG"), (dict(heads=0), "TACTKV_INVALID_ARG"),
    (dict(n_pages=0), "TACTKV_INVALID_ARG"), (dict(head_dim=48), "TACTKV_UNSUPPORTED_SHAPE"),
    (dict(head_dim=288), "TACTKV_UNSUPPORTED_SHAPE"), (dict(heads=1025), "TACTKV_UNSUPPORTED_SHAPE"),
    (dict(page_tokens=8), "TACTKV_UNSUPPORTED_SHAPE"), (dict(page_tokens=48), "TACTKV_UNSUPPORTED_SHAPE"),
    (dict(page_tokens=2048), "TACTKV_UNSUPPORTED_SHAPE"), (dict(n_pages=1 << 31), "TACTKV_UNSUPPORTED_SHAPE"),
]
BAD_POOLS = [
    (dict(k_pages=None), "TACTKV_INVALID_ARG"), (dict(v_scales=None), "TACTKV_INVALID_ARG"),
    (dict(v_pages=8200), "TACTKV_ALIGNMENT"), (dict(k_scales=16388), "TACTKV_ALIGNMENT"),
]
BAD_BATCH = [
    (dict(n_seqs=-1), "TACTKV_INVALID_ARG"), (dict(n_rows=-1), "TACTKV_INVALID_ARG"), (dict(max_pages=-1), "TACTKV_INVALID_ARG"),
    (dict(page_table=None), "TACTKV_INVALID_ARG"), (dict(kv_lens=None), "TACTKV_INVALID_ARG"),
    (dict(row_starts=None), "TACTKV_INVALID_ARG"), (dict(kv_lens=4098), "TACTKV_ALIGNMENT"),
    (dict(n_rows=1 << 30), None),
]


def append(T, c, b, k=4096, v=4096, ts=128, hs=64, kv=None, vv=None, flags=0, ws=4096, n=1 << 20):
    return T._lib.tactkv_text_append(c, b, k, v, ts, hs, kv, vv, flags, ws, n, 0)


def read(T, c, b, k=4096, v=4096, ts=128, hs=64, flags=0, ws=4096, n=1 << 20):
    return T._lib.tactkv_text_read(c, b, k, v, ts, hs, flags, ws, n, 0)


def attend(T, c, b, qh=4, rows=1, length=32, q=4096, qt=256, qhs=64, tree=None, prior=(None, None, None), out=4096,
           m=4096, l=4096, flags=0, ws=4096, n=1 << 30):
    return T._lib.tactkv_text_attention(c, b, qh, rows, length, q, qt, qhs, tree, *prior, out, m, l, flags, ws, n, 0)


@pytest.mark.parametrize("kw,status", BAD_CACHE + BAD_POOLS)
def test_cache_refusals(T, kw, status):
    for call in (append, read, attend):
        assert call(T, cache(T, **kw), batch(T)) == getattr(T, status)
    size = T._lib.tactkv_text_workspace_bytes(cache(T, **kw), 1, 1, 4, 1, 32)
    assert (size == 0) == ((kw, status) in BAD_CACHE)


@pytest.mark.parametrize("kw,status", BAD_BATCH)
def test_batch_refusals(T, kw, status):
    if status is None:                       # more rows than a launch can hold
        assert append(T, cache(T, heads=32), batch(T, **kw)) == T.TACTKV_UNSUPPORTED_SHAPE
        assert read(T, cache(T, heads=32), batch(T, **kw)) == T.TACTKV_UNSUPPORTED_SHAPE
        return
    for call in (append, read, attend):
        assert call(T, cache(T), batch(T, **kw)) == getattr(T, status)


def test_nothing_to_do(T):
    for call in (append, read, attend):
        assert call(T, cache(T), batch(T, n_seqs=0, page_table=None)) == T.TACTKV_OK
        assert call(T, cache(T), batch(T, n_rows=0)) == T.TACTKV_OK


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), "TACTKV_INVALID_ARG"), (dict(v=None), "TACTKV_INVALID_ARG"), (dict(ts=0), "TACTKV_INVALID_ARG"),
    (dict(flags=1), "TACTKV_INVALID_ARG"), (dict(flags=64), "TACTKV_INVALID_ARG"), (dict(k=4098), "TACTKV_ALIGNMENT"),
    (dict(v=4100, flags=2), "TACTKV_ALIGNMENT"), (dict(ts=129), "TACTKV_ALIGNMENT"), (dict(hs=63), "TACTKV_ALIGNMENT"),
    (dict(ws=0), "TACTKV_WORKSPACE"), (dict(ws=4104), "TACTKV_WORKSPACE"), (dict(n=100), "TACTKV_WORKSPACE"),
])
def test_append_and_read_refusals(T, kw, status):
    assert append(T, cache(T), batch(T), **kw) == getattr(T, status)
    assert read(T, cache(T), batch(T), **kw) == getattr(T, status)


@pytest.mark.parametrize("ts,hs,rows,ok", [
    (128, 64, 3, True), (128, 62, 3, False), (126, 64, 3, False), (64, 192, 3, True), (64, 190, 3, False), (62, 500, 3, False),
    (128, 0, 1, False), (2, 64, 1, True), (128, -64, 3, True), (128, -62, 3, False), (256, 128, 3, True), (1 << 62, 1 << 61, 3, True),
])
def test_read_refuses_places_that_meet(T, ts, hs, rows, ok):
    """Two heads of 64.  (Calls that are not refused would launch: the GPU's tests make them.)"""
    places = {(r, h): r * ts + h * hs for r in range(rows) for h in range(2)}
    at = sorted(places.values())
    assert ok == all(b - a >= 64 for a, b in zip(at, at[1:]))          # the parameters themselves
    if not ok:
        assert read(T, cache(T), batch(T, n_rows=rows), ts=ts, hs=hs) == T.TACTKV_INVALID_ARG


def test_append_values_refusals(T):
    assert append(T, cache(T), batch(T), kv=4096) == T.TACTKV_INVALID_ARG
    assert append(T, cache(T), batch(T), vv=4096) == T.TACTKV_INVALID_ARG
    assert append(T, cache(T), batch(T), kv=4096, vv=4104) == T.TACTKV_ALIGNMENT


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), "TACTKV_INVALID_ARG"), (dict(out=None), "TACTKV_INVALID_ARG"), (dict(m=None), "TACTKV_INVALID_ARG"),
    (dict(l=None), "TACTKV_INVALID_ARG"), (dict(qh=0), "TACTKV_INVALID_ARG"), (dict(rows=0), "TACTKV_INVALID_ARG"),
    (dict(length=-1), "TACTKV_INVALID_ARG"), (dict(prior=(4096, None, None)), "TACTKV_INVALID_ARG"),
    (dict(prior=(4096, 4096, None)), "TACTKV_INVALID_ARG"), (dict(prior=(None, 4096, 4096)), "TACTKV_INVALID_ARG"),
    (dict(qh=3), "TACTKV_UNSUPPORTED_SHAPE"), (dict(qh=34), "TACTKV_UNSUPPORTED_SHAPE"),
    (dict(rows=65), "TACTKV_UNSUPPORTED_SHAPE"), (dict(length=(1 << 30) + 1), "TACTKV_UNSUPPORTED_SHAPE"),
    (dict(q=4104), "TACTKV_ALIGNMENT"), (dict(qt=260), "TACTKV_ALIGNMENT"), (dict(qhs=68), "TACTKV_ALIGNMENT"),
    (dict(out=4100), "TACTKV_ALIGNMENT"), (dict(tree=4100), "TACTKV_ALIGNMENT"),
    (dict(prior=(4104, 4096, 4096)), "TACTKV_ALIGNMENT"), (dict(flags=8), "TACTKV_INVALID_ARG"),
    (dict(ws=0), "TACTKV_WORKSPACE"), (dict(n=256), "TACTKV_WORKSPACE"),
])
def test_attention_refusals(T, kw, status):
    assert attend(T, cache(T), batch(T), **kw) == getattr(T, status)


def test_attention_refuses_more_bfloat16_tokens_than_coordinates(T):
    big = dict(format=0, n_pages=1 << 25, page_tokens=1024, heads=2)
    assert attend(T, cache(T, **big), batch(T)) == T.TACTKV_UNSUPPORTED_SHAPE
    assert attend(T, cache(T, **big), batch(T, n_rows=0)) == T.TACTKV_UNSUPPORTED_SHAPE


def test_workspace_sizes(T):
    c = cache(T)
    size = lambda *a: T._lib.tactkv_text_workspace_bytes(c, *a)  # noqa: E731
    assert size(8, 100, 0, 1, 0) == 256                          # append and read: the status word
    assert size(8, 8, 4, 1, 100) > 256
    assert size(-1, 0, 0, 0, 0) == 0 and size(0, 0, -1, 0, 0) == 0
    need = size(8, 8, 4, 1, 1 << 20)
    assert attend(T, c, batch(T, n_seqs=8, n_rows=8), length=1 << 20, n=need - 1) == T.TACTKV_WORKSPACE
    assert T._lib.tactkv_text_workspace_bytes(None, 1, 1, 1, 1, 1) == 0


def test_packed_batch_is_the_structure(T):
    b = T.tactkv_text_batch(11, 22, 33, 4, 5, 6)
    assert T._TEXT_BATCH.pack(11, 22, 33, 4, 5, 6) == bytes(b)[:T._TEXT_BATCH.size]
    assert bytes(b)[T._TEXT_BATCH.size:].strip(b"\0") == b""


def test_tree_words(T):
    w = T.text_tree([[-1, 0, 0, 1], [-1, -1]], device="cpu")
    assert w.tolist() == [1, 3, 5, 11, 1, 2]
    chain = T.text_tree([list(range(-1, 63))], device="cpu")
    assert chain[63].item() == -1 and chain[62].item() == 2 ** 63 - 1
    for bad in ([0], [-1, 1], [-2], list(range(-1, 64))):
        with pytest.raises(ValueError):
            T.text_tree([bad], device="cpu")


def test_pools_are_checked(T):
    import torch
    with pytest.raises(ValueError):                              # on the CPU
        T.TextCache("bf16", torch.zeros((2, 1, 16, 64), dtype=torch.uint8), torch.zeros((2, 1, 16, 64), dtype=torch.uint8))
    with pytest.raises(KeyError):
        T.TextCache("int8", None, None)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_plain_grids(fmt):
    """The test's own quantiser: every code is a fixed point, and nothing between two codes is nearer to a third."""
    codes = sorted({P.code_value(c, fmt) for c in range(256 if fmt == "mxfp8" else 16)} - {np.nan},
                   key=lambda v: (np.isnan(v), v))
    codes = np.array([v for v in codes if not np.isnan(v)])
    x = np.zeros((len(codes), 32))
    x[:, 0], x[:, 1] = codes[-1], codes
    got, scales = P.quantise(x, fmt)
    assert np.array_equal(got[:, 1], codes) and (scales == 127).all()
    mid = (codes[1:] + codes[:-1]) / 2
    x = np.zeros((len(mid), 32))
    x[:, 0], x[:, 1], x[:, 2] = codes[-1], np.nextafter(mid, -np.inf), np.nextafter(mid, np.inf)
    got, _ = P.quantise(x, fmt)
    assert np.array_equal(got[:, 1], codes[:-1]) and np.array_equal(got[:, 2], codes[1:])


def test_numbers_beyond_32_bits(T):
    """Bounds that a C int cannot hold are refused instead of being taken modulo 2^32."""
    c = type("Cache", (), {"ptr": cache(T)})()
    assert T.tactkv_text_workspace_bytes(c, 1, 1, 4, 1, 64) > 0
    for big in ((1 << 32) + 64, 1 << 32, -(1 << 32) + 64):
        assert T.tactkv_text_workspace_bytes(c, 1, 1, 4, 1, big) == 0
        assert T.tactkv_text_workspace_bytes(c, big, 1, 4, 1, 64) == 0
        for kw in (dict(max_rows=1, max_kv_len=big), dict(max_rows=big, max_kv_len=64)):
            with pytest.raises(T.TactkvError):
                T.text_attention(None, c, None, None, None, **kw)
