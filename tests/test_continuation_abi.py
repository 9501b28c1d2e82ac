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


def test_sample_layout():
    assert ctypes.sizeof(enc.EncSampleArgs) == 104


def sample(**kw):
    a = enc.EncSampleArgs()
    for n in ("d_logits", "d_u", "d_temperature", "d_top_p", "d_min_p", "d_top_k", "d_token", "d_probs"):
        setattr(a, n, P)
    a.logits_row = a.probs_row = 1000
    a.rows, a.vocab, a.rows_per_setting, a.dtype, a.probs_dtype = 4, 1000, 1, 3, 1
    for n, v in kw.items():
        setattr(a, n, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(vocab=0), -1), (dict(vocab=2 ** 22 + 1), -2), (dict(rows=2 ** 20 + 1), -2), (dict(dtype=0), -2), (dict(dtype=4), -2),
    (dict(probs_dtype=0), -2), (dict(reserved=1), -1), (dict(d_logits=0), -1), (dict(d_token=0, d_probs=0), -1),
    (dict(d_u=0), -1), (dict(rows_per_setting=0), -1), (dict(d_logits=P + 2), -1), (dict(d_probs=P + 1), -1),
    (dict(d_u=P + 2), -1), (dict(d_top_k=P + 1), -1), (dict(d_temperature=P + 2), -1), (dict(d_token=P + 2), -1),
    (dict(logits_row=1 << 40), -2), (dict(probs_row=999), -1),
])
def test_sample_refusals(L, kw, status):
    assert L.enc_sample(ctypes.byref(sample(**kw)), P, 1 << 40, None) == status
    assert enc.enc_last_error()


def test_sample_workspace(L):
    need = L.enc_sample_workspace_bytes(4, 1000)
    assert need > 0
    a = sample()
    assert L.enc_sample(ctypes.byref(a), P, need - 1, None) == -3
    assert L.enc_sample(ctypes.byref(a), None, need, None) == -1
    assert L.enc_sample(ctypes.byref(a), P + 4, need, None) == -1
    assert L.enc_sample(ctypes.byref(sample(rows=0, d_logits=0)), None, 0, None) == 0
    assert L.enc_sample(None, None, 0, None) == -1
    for rows, vocab in ((0, 10), (10, 0), (2 ** 20 + 1, 10), (10, 2 ** 22 + 1)):
        assert L.enc_sample_workspace_bytes(rows, vocab) == 0
    assert L.enc_sample_workspace_bytes(2 ** 20, 1000) == L.enc_sample_workspace_bytes(1024, 1000)


def test_prefix_layout():
    assert ctypes.sizeof(enc.EncPrefixAttentionArgs) == 288


def prefix(groups=1, d_starts=P, d_shared=P, reserved=0, **kw):
    a = enc.EncPrefixAttentionArgs()
    a.d_starts, a.d_shared, a.groups, a.reserved = d_starts, d_shared, groups, reserved
    t = a.t
    for n in ("d_q", "d_k_new", "d_v_new", "d_k_cache", "d_v_cache", "d_out", "d_lse", "d_table", "d_lens", "d_seqs",
              "d_nodes", "d_mask"):
        setattr(t, n, P)
    for n in ("q", "k_new", "v_new", "out"):
        setattr(t, n + "_batch", 8192)
        setattr(t, n + "_node", 1024)
        setattr(t, n + "_head", 128)
    t.cache_page, t.cache_token, t.cache_head = 16 * 256, 256, 128
    t.batch, t.nodes, t.q_heads, t.kv_heads, t.head_dim, t.dtype = 2, 8, 8, 2, 128, 1
    t.n_pages, t.page_size, t.max_pages, t.max_seqs, t.scale = 100, 16, 50, 2, 0.1
    for n, v in kw.items():
        setattr(t, n, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(reserved=1), -1), (dict(groups=2 ** 20 + 1), -2), (dict(d_starts=0), -1), (dict(d_shared=0), -1),
    (dict(d_starts=P + 2), -1), (dict(d_shared=P + 1), -1), (dict(nodes=0), -1), (dict(nodes=257), -2), (dict(q_heads=9), -5),
    (dict(head_dim=100), -2), (dict(dtype=3), -2), (dict(page_size=0), -1), (dict(scale=NAN), -1), (dict(d_q=0), -1),
    (dict(d_out=P + 8), -1), (dict(d_k_new=0), -1), (dict(d_k_cache=0), -1), (dict(cache_token=260), -1), (dict(d_table=0), -1),
    (dict(d_lens=P + 2), -1), (dict(d_mask=P + 4), -1), (dict(d_seqs=0, batch=3), -1), (dict(cache_page=2 ** 34), -2),
    (dict(batch=2 ** 24), -2),
])
def test_prefix_refusals(L, kw, status):
    assert L.enc_prefix_attention(ctypes.byref(prefix(**kw)), P, 1 << 50, None) == status
    assert enc.enc_last_error()


def test_prefix_workspace(L):
    a = prefix()
    need = L.enc_prefix_attention_workspace_bytes(ctypes.byref(a))
    assert need > 0
    assert L.enc_prefix_attention(ctypes.byref(a), P, need - 1, None) == -3
    assert L.enc_prefix_attention(ctypes.byref(a), None, need, None) == -1
    assert L.enc_prefix_attention(ctypes.byref(a), P + 4, need, None) == -1
    assert L.enc_prefix_attention_workspace_bytes(ctypes.byref(prefix(nodes=0))) == 0
    assert L.enc_prefix_attention_workspace_bytes(None) == 0
    assert L.enc_prefix_attention(None, None, 0, None) == -1
    assert L.enc_prefix_attention(ctypes.byref(prefix(batch=0)), None, 0, None) == 0


def shared_call(L, groups=1, batch=2, seqs=P, starts=P, shared=P, **kw):
    c = enc.EncCache()
    c.d_data = c.d_table = c.d_lens = c.d_refs = P
    c.plane_stride, c.n_planes, c.n_pages, c.page_size, c.row_bytes, c.max_seqs, c.max_pages = 1 << 20, 2, 16, 16, 64, 4, 8
    for n, v in kw.items():
        setattr(c, n, v)
    return L.enc_cache_shared(ctypes.byref(c), seqs, batch, starts, groups, shared, None)


@pytest.mark.parametrize("kw,status", [
    (dict(d_table=0), -1), (dict(page_size=0), -1), (dict(seqs=0), -1), (dict(starts=0), -1), (dict(shared=0), -1),
    (dict(starts=P + 2), -1), (dict(groups=2 ** 20 + 1), -2), (dict(batch=2 ** 31), -2), (dict(max_pages=2 ** 30), -2),
])
def test_cache_shared_refusals(L, kw, status):
    assert shared_call(L, **kw) == status
    assert enc.enc_last_error()


def test_cache_shared_nothing_to_do(L):
    assert shared_call(L, groups=0, starts=0, shared=0) == 0
