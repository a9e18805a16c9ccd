"""The text attention's waits when they run out: a build of the tcgen05 kernel whose waits give up after a few polls.

Every wait of that kernel is bounded; one that expires ends its block's work, records TACTKV_TIMEOUT, and leaves the block
only when no copy or product of it is under way.  Here the limit is so short that waits expire at their first poll, or
somewhere along the tiles; the context stays usable and the next call with an ample limit is right.
"""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from dct_transform_coding_b200 import tactkv as T
    from test_gpu_text import Setup, ints

DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")


@pytest.fixture(scope="module", params=[128, 256])
def built(request, tmp_path_factory):
    if shutil.which(NVCC) is None:
        pytest.skip("needs nvcc")
    lib = str(tmp_path_factory.mktemp("text_waits") / f"text_waits_{request.param}.so")
    csrc = os.path.join(ROOT, "dct_transform_coding_b200", "csrc")
    subprocess.run([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-std=c++17", "-shared", "-Xcompiler", "-fPIC",
                    f"-DTACTKV_TEXT_D={request.param}", "-I", os.path.join(ROOT, "include"), "-I", csrc,
                    os.path.join(ROOT, "tests", "text_waits.cu"), "-o", lib], check=True)
    run = ctypes.CDLL(lib).text_waits_run
    run.argtypes = [ctypes.c_uint32] + [ctypes.c_void_p] * 2 + [ctypes.c_int] * 3 + [ctypes.c_void_p] * 5
    return request.param, run


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("rows,G", [(2, 8), (4, 8), (8, 8)])
def test_waits_that_run_out(built, fmt, rows, G):
    D, run = built
    n, tokens = 300, 1100
    s = Setup(fmt, 1, D, 64, [(rows, tokens)], seed=2)
    table, lens = s.batch[0].repeat(n, 1), ints([tokens - i % 300 for i in range(n)])
    starts = ints([rows * i for i in range(n + 1)])
    q = torch.randn((rows * n + 2, G, D), generator=s.gen).bfloat16().to(DEV)      # two rows behind the last sequence
    want = T.text_attention(q, s.cache, table, lens, starts, max_rows=rows, max_kv_len=tokens,
                            out=torch.full_like(q, 77.0), check=True)
    batch = T.tactkv_text_batch(table.data_ptr(), lens.data_ptr(), starts.data_ptr(), n, rows * n + 2, table.shape[1])
    seen = set()
    for polls in (1, 2, 4, 8, 16, 32, 64, 128, 256, 512, 1024, 1 << 16, 1, 1 << 16):
        out, status = torch.full_like(q, 77.0), torch.zeros(64, dtype=torch.int32, device=DEV)
        m = torch.full(q.shape[:2], 77.0, device=DEV)
        l = m.clone()
        torch.cuda.synchronize()
        assert run(polls, s.cache.ptr, ctypes.addressof(batch), G, rows, tokens, q.data_ptr(), out.data_ptr(), m.data_ptr(),
                   l.data_ptr(), status.data_ptr()) == 0
        got = int(status[0])
        seen.add(got)
        assert got in (T.TACTKV_OK, T.TACTKV_TIMEOUT) and not status[1:].any()
        assert (out[rows * n:] == 77.0).all() and (m[rows * n:] == 77.0).all() and (l[rows * n:] == 77.0).all()
        if polls == 1:
            assert got == T.TACTKV_TIMEOUT
        if polls == 1 << 16:
            assert got == T.TACTKV_OK
        if got == T.TACTKV_OK:
            assert torch.equal(out, want[0])
            assert torch.equal(m[:rows * n], want[1][:rows * n]) and torch.equal(l[:rows * n], want[2][:rows * n])
    assert seen == {T.TACTKV_OK, T.TACTKV_TIMEOUT}
    again = T.text_attention(q, s.cache, table, lens, starts, max_rows=rows, max_kv_len=tokens, check=True)
    assert all(torch.equal(a[:rows * n], b[:rows * n]) for a, b in zip(again, want))
