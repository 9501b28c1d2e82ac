"""Host-side checks, without a GPU, of the entry points that decoding several
continuations adds: struct layouts, workspace sizes, and refusals before any
launch (each with its status). Pointers here are never followed."""
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


def test_block_norm_layout():
    assert ctypes.sizeof(enc.EncBlockNormArgs) == 144


def norm(**kw):
    a = enc.EncBlockNormArgs()
    for n in ("d_y", "d_h", "d_gate", "d_w_post", "d_w_pre", "d_h_out", "d_out"):
        setattr(a, n, P)
    for n in ("y_token", "h_token", "gate_row", "h_out_token", "out_token"):
        setattr(a, n, 4096)
    a.tokens, a.width, a.gate_every = 4, 4096, 1
    a.y_dtype, a.h_dtype, a.g_dtype, a.w_dtype, a.out_dtype, a.flags = 3, 3, 1, 1, 1, 1
    a.eps, a.h_scale, a.y_scale = 1e-6, 1.0, 1.0
    for n, v in kw.items():
        setattr(a, n, v)
    return a


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw,status", [
    (dict(width=0), -1), (dict(width=32769), -2), (dict(flags=4), -1), (dict(eps=-1.0), -1), (dict(eps=NAN), -1),
    (dict(eps=INF), -1), (dict(h_scale=NAN), -1), (dict(y_scale=INF), -1), (dict(tokens=2 ** 31), -2), (dict(d_h=0), -1),
    (dict(d_h_out=0, d_out=0, d_w_pre=0), -1), (dict(d_y=0), -1), (dict(d_y=0, flags=0, d_w_post=0), -1),
    (dict(flags=0), -1), (dict(d_out=0), -1), (dict(gate_every=0), -1), (dict(y_dtype=0), -2), (dict(h_dtype=4), -2),
    (dict(g_dtype=9), -2), (dict(w_dtype=0), -2), (dict(out_dtype=4), -2), (dict(d_y=P + 2), -1), (dict(d_out=P + 1), -1),
    (dict(d_w_pre=P + 1), -1), (dict(h_token=1 << 40), -2), (dict(out_token=4095), -1), (dict(h_out_token=0), -1),
])
def test_block_norm_refusals(L, kw, status):
    assert L.enc_block_norm(ctypes.byref(norm(**kw)), None) == status
    assert enc.enc_last_error()


def test_block_norm_nothing_to_do(L):
    assert L.enc_block_norm(ctypes.byref(norm(tokens=0, d_h=0)), None) == 0
    assert enc.enc_last_error() == ""
    assert L.enc_block_norm(None, None) == -1
