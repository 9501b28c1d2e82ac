"""Sizes of the workspaces of decoding several continuations, without a GPU."""
import ctypes
import random
import re

import pytest

from lossless_weight_compression_amd import enc
from test_continuation_abi import L, prefix, sample  # noqa: F401


def attention_bytes(L, batch=64, groups=8, nodes=1, room=9600, q_heads=32, kv_heads=8, dim=128):  # noqa: F811
    a = prefix(groups=groups, batch=batch, nodes=nodes, q_heads=q_heads, kv_heads=kv_heads, head_dim=dim, page_size=16,
               max_pages=room // 16)
    return int(L.enc_prefix_attention_workspace_bytes(ctypes.byref(a)))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("batch,nodes", [(1, 1), (2, 1), (9, 1), (64, 1), (2, 33), (1, 256), (64, 40)])
def test_no_groups_need_no_room_for_shared_tokens(L, batch, nodes, dim):  # noqa: F811
    """Without groups there are sequences' own pieces alone: 768 of them, one more for every 16 or 32 rows of a sequence
    and KV head, each with its sums, a maximum and a sum of weights a row in fp32, and the plan of those pieces."""
    without = attention_bytes(L, batch=batch, groups=0, nodes=nodes, dim=dim)
    rows = 4 * nodes
    most = max((768 // 8 + batch * -(-rows // t)) * 8 * t for t in (16, 32))
    plan = 64 * (768 + 8 * batch * -(-rows // 16)) + 4096 + 32 * (batch + 64)
    assert 0 < without <= most * (4 * dim + 8) + plan


def needed(status):
    """What a refused call says that it needs."""
    assert status == -3
    return int(re.search(r"(\d+) needed", enc.enc_last_error()).group(1))


def attention_need(L, **kw):  # noqa: F811
    groups = kw.pop("groups")
    a = prefix(groups=groups, page_size=16, max_seqs=2 ** 20, **kw)
    return needed(L.enc_prefix_attention(ctypes.byref(a), 4096, 0, None))


def sample_need(L, rows, vocab):  # noqa: F811
    a = sample(rows=rows, vocab=vocab, logits_row=vocab, probs_row=vocab)
    return needed(L.enc_sample(ctypes.byref(a), 4096, 0, None))


@pytest.mark.parametrize("vocab", [1, 1000, 16377, 16378, 32003, 50000, 128256, 151936, 262144, 2 ** 20, 2 ** 22 - 8, 2 ** 22])
def test_sample_workspace_serves_fewer_rows(L, vocab):  # noqa: F811
    """Across the change of segments (some 256 segments of 16384 values), the most rows at a time, and 1024 rows."""
    rows = [*range(1, 300), 511, 512, 513, 1000, 1023, 1024, 1025, 5000, 2 ** 20]
    sizes = [int(L.enc_sample_workspace_bytes(n, vocab)) for n in rows]
    needs = [sample_need(L, n, vocab) for n in rows]
    most = 0
    for n, size, need in zip(rows, sizes, needs):
        most = max(most, need)
        assert size >= most, (n, size, most)
    assert sizes[-1] == sizes[rows.index(1024)] <= 330 << 20


HEADS = [(32, 8, 128), (16, 4, 64), (8, 1, 256), (28, 4, 96), (6, 6, 64), (8, 8, 200)]


@pytest.mark.parametrize("q_heads,kv_heads,dim", HEADS)
def test_attention_workspace_serves_smaller_calls(L, q_heads, kv_heads, dim):  # noqa: F811
    """No more sequences, nodes, groups or pages: what the call needs is there, and sizes do not fall."""
    rng = random.Random(q_heads)
    axes = dict(batch=[1, 2, 5, 8, 9, 16, 17, 33, 64, 65, 200, 1025, 4000], nodes=[1, 2, 4, 5, 8, 9, 17, 33, 64, 256],
                groups=[0, 1, 2, 3, 4, 7, 8, 16, 31, 64, 200, 1024, 5000],
                max_pages=[1, 50, 1000, 1024, 1025, 2048, 2049, 8192])
    heads = dict(q_heads=q_heads, kv_heads=kv_heads, head_dim=dim)

    def size_of(groups, **kw):
        a = prefix(groups=groups, page_size=16, **heads, **kw)
        return int(L.enc_prefix_attention_workspace_bytes(ctypes.byref(a)))

    for _ in range(4000):
        big = {n: rng.randrange(len(v)) for n, v in axes.items()}
        small = {n: rng.randint(0, i) if rng.random() < 0.6 else i for n, i in big.items()}
        big, small = ({n: axes[n][i] for n, i in at.items()} for at in (big, small))
        size = size_of(**big)
        if size == 0:                                          # refused: too many pieces, rows or groups
            continue
        assert size >= size_of(**small) >= attention_need(L, **heads, **small), (big, small)


def test_workspace_sizes_are_not_far_from_what_calls_need(L):  # noqa: F811
    """With one group, where tiles are largest, a call needs what it is told but for alignment of the plan's parts."""
    for batch, nodes in ((4, 1), (16, 1), (64, 1), (16, 8), (256, 1), (2, 64)):
        a = prefix(groups=1, batch=batch, nodes=nodes, q_heads=32, kv_heads=8)
        size = int(L.enc_prefix_attention_workspace_bytes(ctypes.byref(a)))
        assert size <= 1.25 * attention_need(L, groups=1, batch=batch, nodes=nodes, q_heads=32, kv_heads=8), (batch, nodes)
