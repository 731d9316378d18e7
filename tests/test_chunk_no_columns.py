"""Chunks over a table of no columns, whose memory may be at NULL: every length
counts as 0, so every row is zeros; and packed rows are told from a cache by more
than that pointer.  On the CPU by the kernels' own function, compiled here."""
import ctypes
import os
import subprocess

import pytest
import torch

import elementwise_row_rmsnorm_gb300 as gbe
from chunk_ref import filled, i32, rand
from elementwise_row_rmsnorm_gb300 import _build

F8, BF, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def sequence(tmp_path_factory):
    so = tmp_path_factory.mktemp("chunk") / "chunk_host.so"
    subprocess.run([_build.nvcc(), *_build.ARCH, *_build.NVCC_FLAGS, "-shared", "-o", str(so),
                    os.path.join(HERE, "chunk_host.cu"), "-lcudart_static"], check=True, capture_output=True)
    f = ctypes.CDLL(str(so)).chunk_sequence
    i64, p = ctypes.c_int64, ctypes.c_void_p
    f.argtypes = [ctypes.c_int, p, p, p, i64, i64, i64, ctypes.c_int, i64, p]
    f.restype = None

    def call(packed, starts, lens, T, table=None, max_pages=0, page_size=16, b=0):
        s, n, out = ((ctypes.c_int * len(x))(*x) for x in (starts, lens, [0, 0, 0]))
        f(packed, s, table, n, len(starts) - 1, T, max_pages, page_size, b, out)
        return tuple(out)
    return call


def test_a_cache_without_columns_holds_no_keys(sequence):
    for lens in ([100], [-1], [0], [2 ** 31 - 1]):
        assert sequence(0, [3, 10], lens, 20) == (3, 7, 0)
    assert sequence(0, [3, 10], [100], 20, table=1 << 40, max_pages=2) == (3, 7, 32)
    assert sequence(0, [3, 10], [30], 20, table=1 << 40, max_pages=2) == (3, 7, 30)


def test_packed_rows_are_their_own_keys(sequence):
    assert sequence(1, [3, 10, 10], [0], 20) == (3, 7, 7)
    assert sequence(1, [3, 10, 10], [0], 20, b=1) == (10, 0, 0)
    assert sequence(1, [-5, 2 ** 31 - 1], [0], 20) == (0, 20, 20)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kind", [(F32, F32), (F32, F8), (BF, BF), (BF, F8)])
@pytest.mark.parametrize("D", [64, 136])
def test_zeros(dtype, kind, D):
    P, H, Hq, T = 16, 2, 8, 40
    cache, _ = filled([70], P, H, D, dtype, kind, 5)
    wide = rand((T, Hq * D + 1), dtype, 6)
    for shift in (0, 1):  # (1: off the 16-byte grid)
        q = wide[:, shift:shift + Hq * D].unflatten(1, (Hq, D))
        for table in (torch.empty(3, 0, dtype=torch.int32, device="cuda"),
                      torch.zeros(9, dtype=torch.int32, device="cuda")[:0].view(3, 0)):
            assert gbe.attn_chunk_workspace(3, T, Hq, cache, 0) == 0
            for window, sinks in ((0, 0), (5, 2)):
                out = torch.full_like(wide, 9.0)
                view = out[:, shift:shift + Hq * D].unflatten(1, (Hq, D))
                gbe.gbe_attn_chunk(q, view, cache, i32([2, 35, 35, 38]), table, i32([70, 9, -4]), 0.1, window, sinks)
                assert bool((view[2:38] == 0).all())
                assert bool((view[:2] == 9.0).all()) and bool((view[38:] == 9.0).all())
                one = gbe.attn_decode_window(q[:3].contiguous(), cache, table, i32([70, 9, -4]), window, sinks)
                assert bool((one == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kind", [(F32, F32), (F32, F8), (BF, BF), (BF, F8)])
@pytest.mark.parametrize("D", [64, 136])
def test_a_cache_of_no_pages(dtype, kind, D):
    """Every token lies on a page that is not there."""
    P, H, Hq, T = 16, 2, 8, 40
    cache = gbe.kv_cache(0, H, P, D, kind)
    table, lens = torch.zeros(2, 200, dtype=torch.int32, device="cuda"), i32([3000, 9])
    q = rand((T, Hq, D), dtype, 6)
    for window, sinks in ((0, 0), (5, 2)):
        out = gbe.attn_chunk(q, cache, i32([0, 35, T]), table, lens, 0.1, window, sinks)
        assert bool((out == 0).all())
        assert bool((gbe.attn_decode_window(q[:2], cache, table, lens, window, sinks) == 0).all())
