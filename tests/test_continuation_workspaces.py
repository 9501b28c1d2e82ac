"""Sizes of the workspaces of decoding several continuations, without a GPU."""
import ctypes

import pytest

from test_continuation_abi import L, prefix  # noqa: F401


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
