"""The plain implementations against closed forms and hand-worked rows."""
import numpy as np

import continuation_ref as ref


def test_norms_by_hand():
    y, h = np.array([[3.0, 4.0]]), np.array([[1.0, -1.0]])
    out, x, _, _ = ref.block_norm(y, h, np.array([[2.0, 1.0]]), np.array([1.0, 0.5]), None, True, 2.0, 0.5, 0.0, False)
    r = 12.5 ** -0.5                                          # 1 / sqrt(mean(9, 16))
    want = np.array([[2 + 0.5 * 2 * 3 * r, -2 + 0.5 * 4 * r * 0.5]])
    assert np.allclose(out, want, rtol=1e-14)
    assert np.allclose(x, want / np.sqrt((want ** 2).mean()), rtol=1e-14)
    _, x, _, _ = ref.block_norm(None, h, None, None, np.array([0.0, 1.0]), False, 1.0, 1.0, 0.0, True)
    assert np.allclose(x, [[1.0, -2.0]], rtol=1e-14)


def test_filters_by_hand():
    l = np.log(np.array([0.1, 0.4, 0.2, 0.25, 0.05]))
    kept = lambda *a: list(np.nonzero(ref.kept_weights(l, *a))[0])  # noqa: E731
    assert kept(1.0, 0, 1.0, 0.0) == [0, 1, 2, 3, 4]
    assert kept(1.0, 2, 1.0, 0.0) == [1, 3]
    assert kept(1.0, 0, 0.6, 0.0) == [1, 3]                   # 0.4, then 0.65 reaches it
    assert kept(1.0, 3, 0.8, 0.0) == [1, 2, 3]                # of 0.85: 0.65 does not reach 0.68
    assert kept(1.0, 0, 1.0, 0.45) == [1, 2, 3]
    assert kept(0.0, 0, 1.0, 0.0) == [1]
    assert kept(1.0, 0, 0.0, 0.0) == [1] and kept(1.0, 0, 1.0, 2.0) == [1]
    e = ref.kept_weights(l, 1.0, 2, 1.0, 0.0)
    assert [ref.draw(e, u) for u in (0.0, 0.6, 0.63, 0.99, 1.0)] == [1, 1, 3, 3, 3]


def test_ties_and_special_values():
    l = np.array([2.0, 5.0, 5.0, np.nan, 5.0, -np.inf])
    assert list(np.nonzero(ref.kept_weights(l, 1.0, 2, 1.0, 0.0))[0]) == [1, 2]
    assert list(np.nonzero(ref.kept_weights(l, 1.0, 0, 0.5, 0.0))[0]) == [1, 2]
    assert list(np.nonzero(ref.kept_weights(l, 0.0, 0, 1.0, 0.0))[0]) == [1]
    inf = np.array([1.0, np.inf, 2.0, np.inf])
    assert list(ref.kept_weights(inf, 0.7, 0, 1.0, 0.0)) == [0, 1, 0, 1]
    assert not ref.kept_weights(np.array([np.nan, -np.inf]), 1.0, 0, 1.0, 0.0).any()
    assert ref.draw(np.zeros(3), 0.5) == -1
