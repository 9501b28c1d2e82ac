"""Limits of the decoding-step entry points that the host refuses, without a
GPU: every call here ends before a HIP call."""
import ctypes
import os

import pytest

from lossless_weight_compression_amd import enc

P = 4096          # a well-aligned address that nothing reads


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(enc.LIB_PATH):
        from lossless_weight_compression_amd import build
        build.build(verbose=False)
    return enc.lib()


@pytest.mark.parametrize("row_bytes", [2 ** 31 + 16, 2 ** 32 - 4096, 2 ** 32 - 16])
def test_rows_whose_copy_would_pass_32_bits(L, row_bytes):
    c = enc.EncCache()
    c.d_data = c.d_table = c.d_lens = c.d_refs = P
    c.plane_stride, c.n_planes, c.n_pages, c.page_size, c.row_bytes = 2 ** 36, 2, 4, 1, row_bytes
    c.max_seqs, c.max_pages = 4, 4
    ref = ctypes.byref(c)
    assert L.enc_cache_commit(ref, P, 1, P, 2 ** 36, 2 ** 34, P, P, 2, P, P, 1 << 40, None) == -2
    assert L.enc_cache_fork(ref, P, P, 1, None) == -2
    assert L.enc_cache_truncate(ref, P, P, 1, None) == -2
    assert L.enc_cache_workspace_bytes(ref, 1, 2) == 0
    c.row_bytes = 2 ** 31
    assert L.enc_cache_workspace_bytes(ref, 1, 2) > 0
