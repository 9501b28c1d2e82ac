"""The plain implementations that the decoding-step kernels are checked with,
checked themselves: against hand-worked values, closed forms and the property
each operator exists for. No GPU."""
import numpy as np
import pytest

import step_ref as ref


def test_rotation_keeps_lengths_and_norm_is_one():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 2, 16))
    ang = rng.standard_normal((8, 6))
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    for adjacent in (False, True):
        y, _ = ref.norm_rope(x, None, table, [0, 5, 7], 0.0, adjacent)
        assert np.allclose((y * y).mean(-1), 1.0)
        assert np.allclose(y[..., 12:], (x / np.sqrt((x * x).mean(-1, keepdims=True)))[..., 12:])
    one = np.zeros((1, 1, 4))
    one[0, 0, 0] = 1.0
    quarter = np.array([[0.0, 0.0, 1.0, 1.0]])     # cos 0, sin 1: a quarter turn
    assert np.array_equal(ref.norm_rope(one, None, quarter, [0], 0.0, False, norm=False)[0].ravel(), [0, 0, 1, 0])
    assert np.array_equal(ref.norm_rope(one, None, quarter, [0], 0.0, True, norm=False)[0].ravel(), [0, 1, 0, 0])


def test_mask_words_and_ancestors():
    parents = np.array([[-1, 0, 0, 1, 3]])
    seen = ref.ancestors(parents)
    assert [list(np.nonzero(seen[0, i])[0]) for i in range(5)] == [[0], [0, 1], [0, 2], [0, 1, 3], [0, 1, 3, 4]]
    assert ref.mask_words(seen)[0, :, 0].tolist() == [1, 3, 5, 11, 27]
    wide = np.zeros((1, 70, 70), bool)
    wide[0, 69, [0, 63, 64, 69]] = True
    assert ref.mask_words(wide).view(np.uint64)[0, 69].tolist() == [1 | 1 << 63, 1 | 1 << 5]


def test_attention_by_hand():
    q = np.zeros((1, 2, 1, 2)); q[0, :, 0, 0] = 1
    kn = np.zeros((1, 2, 1, 2)); vn = np.arange(4.0).reshape(1, 2, 1, 2)
    kc = np.zeros((2, 2, 1, 2)); vc = 10 + np.arange(8.0).reshape(2, 2, 1, 2)
    out, lse, _ = ref.tree_attention(q, kn, vn, kc, vc, np.array([[1, 0]]), [3], np.eye(2, dtype=bool)[None], 1.0)
    # equal scores: the mean of rows (1,0), (1,1), (0,0) and the node itself
    assert np.allclose(out[0, 0, 0], (vc[1, 0, 0] + vc[1, 1, 0] + vc[0, 0, 0] + vn[0, 0, 0]) / 4)
    assert np.allclose(lse[0, :, 0], np.log(4))


@pytest.mark.parametrize("point", [False, True])
@pytest.mark.parametrize("shape", ["chain", "fan", "tree"])
def test_verified_tokens_follow_the_target(point, shape):
    """The first token after the pending one (a drafted child accepted, or the
    one drawn) is distributed as target row 0, whatever the draft."""
    rng = np.random.default_rng([7, point, len(shape)])
    V, n = 5, 40000
    parents = {"chain": [-1, 0, 1], "fan": [-1, 0, 0, 0], "tree": [-1, 0, 0, 1, 1]}[shape]
    T = len(parents)
    p = rng.dirichlet(np.ones(V), T).astype(np.float32)
    q = rng.dirichlet(np.ones(V), T).astype(np.float32)
    tokens = np.zeros((n, T), np.int32)
    for i in range(1, T):
        if point:                                   # named without chance: distinct among siblings
            tokens[:, i] = sum(parents[j] == parents[i] for j in range(1, i))
        else:
            tokens[:, i] = rng.choice(V, n, p=q[parents[i]].astype(np.float64) / q[parents[i]].sum(dtype=np.float64))
    u = rng.random((n, T), dtype=np.float32)
    path, count, token = ref.verify(np.tile(np.array(parents, np.int32), (n, 1)), tokens,
                                    np.broadcast_to(p, (n, T, V)), None if point else np.broadcast_to(q, (n, T, V)), u)
    first = np.where(count > 1, np.take_along_axis(tokens, np.maximum(path[:, 1:2], 0), 1)[:, 0], token)
    got = np.bincount(first, minlength=V) / n
    sigma = np.sqrt(p[0] * (1 - p[0]) / n)
    assert (np.abs(got - p[0]) <= 5 * sigma + 1e-6).all(), (got, p[0])


def test_verify_by_hand():
    f = np.float32
    p = np.array([[[0.5, 0.5, 0, 0], [0, 0, 1, 0]]], f)
    q = np.array([[[1.0, 0, 0, 0], [0.25] * 4]], f)
    par, tok = np.array([[-1, 0]], np.int32), np.array([[9, 0]], np.int32)
    # u q < p: 0.4 < 0.5 accepted, then row 1 gives token 2
    assert [a.tolist() for a in ref.verify(par, tok, p, q, np.array([[0.0, 0.4]], f))] == [[[0, 1]], [2], [2]]
    # 0.5 < 0.5 fails: the rest is token 1 alone
    assert [a.tolist() for a in ref.verify(par, tok, p, q, np.array([[0.99, 0.5]], f))] == [[[0, -1]], [1], [1]]
    # an empty row draws nothing
    assert ref.verify(par, tok, p * 0, q, np.array([[0.5, 0.5]], f))[2].tolist() == [-1]


def test_pages_by_hand():
    c = ref.Pages(np.zeros((1, 4, 2, 1)), np.full((3, 3), -1), np.zeros(3, int), np.zeros(4, int))
    draft = np.arange(1.0, 7.0).reshape(1, 1, 6, 1)
    assert c.commit([0], draft, np.array([[0, 2, 5, 1, 1, 1]]), [3]) == 0
    assert c.table[0].tolist() == [0, 1, -1] and c.data[0, :2, :, 0].tolist() == [[1, 3], [6, 0]]
    c.fork([0], [2])
    assert c.refs.tolist() == [2, 2, 0, 0] and c.lens.tolist() == [3, 0, 3]
    assert c.commit([2], draft, np.array([[4] + [0] * 5]), [1]) == 0      # copies the shared half page
    assert c.table[2].tolist() == [0, 2, -1] and c.data[0, 2, :, 0].tolist() == [6, 5]
    assert c.refs.tolist() == [2, 1, 1, 0]
    assert c.commit([0, 2], np.zeros((1, 2, 6, 1)), np.zeros((2, 6), int), [3, 3]) == -3
    c.truncate([2], [1])
    assert c.refs.tolist() == [2, 1, 0, 0] and c.lens[2] == 1
