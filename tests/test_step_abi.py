"""Host-side checks of the decoding-step entry points, without a GPU: struct
layouts, workspace sizes, and refusals before any launch (each with its
status). Pointers here are never followed: every call is refused, or has
nothing to do, before a HIP call."""
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


def test_struct_layouts():
    assert ctypes.sizeof(enc.EncQkArgs) == 224
    assert ctypes.sizeof(enc.EncTreeAttentionArgs) == 264
    assert ctypes.sizeof(enc.EncVerifyArgs) == 120
    assert ctypes.sizeof(enc.EncCache) == 64


def qk(**kw):
    a = enc.EncQkArgs()
    for n in ("d_q", "d_k", "d_v", "d_q_out", "d_k_out", "d_v_out", "d_q_weight", "d_k_weight", "d_positions", "d_table"):
        setattr(a, n, P)
    for n in ("q", "k", "v", "q_out", "k_out", "v_out"):
        setattr(a, n + "_token", 512)
        setattr(a, n + "_head", 128)
    a.tokens, a.q_heads, a.kv_heads, a.head_dim, a.rot_dim, a.max_pos = 4, 4, 4, 128, 128, 100
    a.in_dtype, a.out_dtype, a.w_dtype, a.eps = 3, 1, 1, 1e-6
    for n, v in kw.items():
        setattr(a, n, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(q_heads=0), -1), (dict(kv_heads=0), -1), (dict(head_dim=0), -1), (dict(head_dim=12), -2),
    (dict(head_dim=520), -2), (dict(rot_dim=7), -1), (dict(rot_dim=130), -1), (dict(in_dtype=0), -2),
    (dict(out_dtype=4), -2), (dict(w_dtype=9), -2), (dict(flags=4), -1), (dict(reserved=1), -1), (dict(eps=-1.0), -1),
    (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1), (dict(d_q=0), -1), (dict(d_k_out=0), -1),
    (dict(d_v_out=0), -1), (dict(d_q=P + 8), -1), (dict(q_token=514), -1), (dict(k_out_head=132), -1),
    (dict(d_q_weight=P + 4), -1), (dict(d_positions=0), -1), (dict(d_table=0), -1), (dict(max_pos=0), -1),
    (dict(tokens=2 ** 31), -2), (dict(q_heads=70000), -2),
])
def test_qk_refusals(L, kw, status):
    assert L.enc_qk_norm_rope(ctypes.byref(qk(**kw)), None) == status
    assert enc.enc_last_error()


def test_qk_nothing_to_do(L):
    assert L.enc_qk_norm_rope(ctypes.byref(qk(tokens=0, d_q=0)), None) == 0
    assert enc.enc_last_error() == ""
    assert L.enc_qk_norm_rope(None, None) == -1


def attention(**kw):
    a = enc.EncTreeAttentionArgs()
    for n in ("d_q", "d_k_new", "d_v_new", "d_k_cache", "d_v_cache", "d_out", "d_lse", "d_table", "d_lens", "d_seqs",
              "d_nodes", "d_mask"):
        setattr(a, n, P)
    for n in ("q", "k_new", "v_new", "out"):
        setattr(a, n + "_batch", 8192)
        setattr(a, n + "_node", 1024)
        setattr(a, n + "_head", 128)
    a.cache_page, a.cache_token, a.cache_head = 16 * 256, 256, 128
    a.batch, a.nodes, a.q_heads, a.kv_heads, a.head_dim, a.dtype = 2, 8, 8, 2, 128, 1
    a.n_pages, a.page_size, a.max_pages, a.max_seqs, a.scale = 100, 16, 50, 2, 0.1
    for n, v in kw.items():
        setattr(a, n, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(nodes=0), -1), (dict(nodes=257), -2), (dict(q_heads=0), -1), (dict(q_heads=9), -5), (dict(kv_heads=0), -1),
    (dict(head_dim=0), -1), (dict(head_dim=100), -2), (dict(head_dim=264), -2), (dict(dtype=3), -2), (dict(dtype=0), -2),
    (dict(page_size=0), -1), (dict(page_size=65537), -2), (dict(n_pages=0), -1), (dict(max_pages=0), -1),
    (dict(max_pages=2 ** 31 // 16), -2), (dict(n_pages=2 ** 31 // 16), -2), (dict(max_seqs=0), -1), (dict(reserved=2), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(d_q=0), -1), (dict(d_out=P + 8), -1),
    (dict(d_k_new=0), -1), (dict(d_v_new=P + 2), -1), (dict(d_k_cache=0), -1), (dict(d_v_cache=0), -1),
    (dict(cache_token=260), -1), (dict(q_head=4), -1), (dict(d_table=0), -1), (dict(d_lens=0), -1),
    (dict(d_lens=P + 2), -1), (dict(d_mask=P + 4), -1), (dict(d_seqs=0, batch=3), -1), (dict(cache_page=2 ** 34), -2),
    (dict(k_new_node=2 ** 36), -2), (dict(batch=2 ** 24), -2), (dict(q_heads=1024, kv_heads=1, nodes=256), -2),
])
def test_attention_refusals(L, kw, status):
    assert L.enc_tree_attention(ctypes.byref(attention(**kw)), P, 1 << 40, None) == status
    assert enc.enc_last_error()


def test_attention_workspace(L):
    a = attention()
    need = L.enc_tree_attention_workspace_bytes(ctypes.byref(a))
    assert need > 0
    assert L.enc_tree_attention(ctypes.byref(a), P, need - 1, None) == -3
    assert L.enc_tree_attention(ctypes.byref(a), None, need, None) == -1
    assert L.enc_tree_attention(ctypes.byref(a), P + 4, need, None) == -1
    assert L.enc_tree_attention_workspace_bytes(ctypes.byref(attention(nodes=0))) == 0
    assert L.enc_tree_attention_workspace_bytes(None) == 0
    assert L.enc_tree_attention(None, None, 0, None) == -1
    assert L.enc_tree_attention(ctypes.byref(attention(batch=0)), None, 0, None) == 0


def verify(**kw):
    a = enc.EncVerifyArgs()
    for n in ("d_parents", "d_tokens", "d_target", "d_draft", "d_u", "d_nodes", "d_path", "d_count", "d_token"):
        setattr(a, n, P)
    a.target_batch = a.draft_batch = 8000
    a.target_node = a.draft_node = 1000
    a.batch, a.nodes, a.vocab, a.dtype = 2, 8, 1000, 3
    for n, v in kw.items():
        setattr(a, n, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(nodes=0), -1), (dict(nodes=257), -2), (dict(vocab=0), -1), (dict(vocab=2 ** 22 + 1), -2), (dict(dtype=4), -2),
    (dict(batch=2 ** 20 + 1), -2), (dict(d_parents=0), -1), (dict(d_tokens=0), -1), (dict(d_target=0), -1),
    (dict(d_u=0), -1), (dict(d_path=0), -1), (dict(d_count=0), -1), (dict(d_token=0), -1), (dict(d_target=P + 2), -1),
    (dict(d_draft=P + 1), -1), (dict(d_u=P + 2), -1),
])
def test_verify_refusals(L, kw, status):
    assert L.enc_verify_tree(ctypes.byref(verify(**kw)), P, 1 << 40, None) == status
    assert enc.enc_last_error()


def test_verify_workspace(L):
    need = L.enc_verify_tree_workspace_bytes(2, 8, 100000)
    a = verify(vocab=100000)
    assert L.enc_verify_tree(ctypes.byref(a), P, need - 1, None) == -3
    assert L.enc_verify_tree(ctypes.byref(a), None, need, None) == -1
    assert L.enc_verify_tree(None, P, need, None) == -1
    assert L.enc_verify_tree(ctypes.byref(verify(batch=0)), None, 0, None) == 0
    for args in ((0, 8, 10), (1, 0, 10), (1, 257, 10), (1, 8, 0), (1, 8, 2 ** 22 + 1)):
        assert L.enc_verify_tree_workspace_bytes(*args) == 0


def cache(**kw):
    c = enc.EncCache()
    c.d_data = c.d_table = c.d_lens = c.d_refs = P
    c.plane_stride, c.n_planes, c.n_pages, c.page_size, c.row_bytes = 100 * 16 * 256, 2, 100, 16, 256
    c.max_seqs, c.max_pages = 4, 10
    for n, v in kw.items():
        setattr(c, n, v)
    return c


BAD_CACHES = [
    (dict(d_data=0), -1), (dict(d_data=P + 8), -1), (dict(d_table=0), -1), (dict(d_lens=P + 1), -1), (dict(d_refs=0), -1),
    (dict(n_planes=0), -1), (dict(n_planes=65536), -2), (dict(n_pages=0), -1), (dict(page_size=0), -1),
    (dict(page_size=65537), -2), (dict(row_bytes=0), -1), (dict(row_bytes=24), -1), (dict(plane_stride=100 * 16 * 256 - 16), -1),
    (dict(plane_stride=100 * 16 * 256 + 8), -1), (dict(max_seqs=0), -1), (dict(max_pages=0), -1),
    (dict(max_pages=2 ** 31 // 16), -2), (dict(n_pages=2 ** 31 - 1, page_size=65536), -2),
]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_cache_refusals(L, kw, status):
    c = ctypes.byref(cache(**kw))
    assert L.enc_cache_commit(c, P, 1, P, 4096, 4096, P, P, 8, P, P, 1 << 40, None) == status
    assert L.enc_cache_fork(c, P, P, 1, None) == status
    assert L.enc_cache_truncate(c, P, P, 1, None) == status
    assert L.enc_cache_workspace_bytes(c, 1, 8) == 0


def test_call_refusals(L):
    c = ctypes.byref(cache())
    need = L.enc_cache_workspace_bytes(c, 3, 8)
    assert need > 0

    def commit(seqs=P, batch=3, draft=P, plane=4096, seq=2048, path=P, count=P, nodes=8, status=P, ws=P, size=need):
        return L.enc_cache_commit(c, seqs, batch, draft, plane, seq, path, count, nodes, status, ws, size, None)

    for kw, status in ((dict(seqs=None), -1), (dict(batch=0), -1), (dict(batch=2 ** 20 + 1), -2), (dict(draft=None), -1),
                       (dict(draft=P + 4), -1), (dict(plane=4100), -1), (dict(seq=8), -1), (dict(path=None), -1),
                       (dict(count=None), -1), (dict(count=P + 2), -1), (dict(nodes=0), -1), (dict(nodes=257), -2),
                       (dict(status=None), -1), (dict(ws=None), -1), (dict(ws=P + 8), -1), (dict(size=need - 1), -3)):
        assert commit(**kw) == status, kw
    for f in (L.enc_cache_fork, L.enc_cache_truncate):
        assert f(c, None, P, 1, None) == -1
        assert f(c, P, None, 1, None) == -1
        assert f(c, P, P + 2, 1, None) == -1
        assert f(c, P, P, 65536, None) == -2
        assert f(c, None, None, 0, None) == 0
        assert f(None, P, P, 1, None) == -1


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(1, 1, 8)
    with pytest.raises(ValueError):
        enc.enc_qk_norm_rope(x, x, x, torch.zeros(1, dtype=torch.int32), None)
    with pytest.raises(ValueError):
        enc.enc_verify_tree(torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32),
                            torch.zeros(1, 1, 4), None, torch.zeros(1, 1))


@pytest.mark.parametrize("kw", [dict(batch=2 ** 23, nodes=1, q_heads=8, kv_heads=2), dict(batch=2 ** 24, nodes=1, q_heads=1, kv_heads=1)])
def test_attention_grids_above_32_bits_of_threads(L, kw):
    a = attention(max_pages=1, **kw)
    assert L.enc_tree_attention(ctypes.byref(a), P, 1 << 40, None) == -2
    assert L.enc_tree_attention_workspace_bytes(ctypes.byref(a)) == 0


def test_verify_grids_above_32_bits_of_threads(L):
    a = verify(batch=2 ** 18, vocab=2 ** 20, target_batch=0, target_node=0)
    assert L.enc_verify_tree(ctypes.byref(a), P, 1 << 40, None) == -2
    assert enc.enc_last_error()
