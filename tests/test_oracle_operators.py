"""The oracle's operators against hand-worked cases and closed forms."""
import numpy as np

from oracle import operators as ops


def test_rms_norm_hand():
    # row (3, 4): mean square 12.5; with the residual (1, 1): (4, 5), 20.5
    s, y = ops.rms_norm([[3.0, 4.0]], [2.0, 1.0], 0.0)
    assert np.allclose(y, [[6 / np.sqrt(12.5), 4 / np.sqrt(12.5)]], rtol=1e-15)
    s, y = ops.rms_norm([[3.0, 4.0]], [1.0, 1.0], 0.5, [[1.0, 1.0]])
    assert np.array_equal(s, [[4.0, 5.0]])
    assert np.allclose(y, [[4 / np.sqrt(21.0), 5 / np.sqrt(21.0)]], rtol=1e-15)


def test_quant_hand():
    u, s = ops.quant_i8([[-254.0, 127.0, 1.0], [0.0, 0.0, 0.0]])
    assert np.array_equal(s, [2.0, 0.0])
    assert np.array_equal(u, [[-127.0, 63.5, 0.5], [0.0, 0.0, 0.0]])


def test_linear_hand():
    acc, out = ops.linear_i8([[1, -2]], [0.5], [[3, 4], [-5, 6]], [2.0, 1.0], [1.0, 0.0])
    assert np.array_equal(acc, [[-5, -17]])
    assert np.array_equal(out, [[-4.0, -8.5]])


def test_logprobs_closed_forms():
    V = 8
    r = ops.logprobs(np.zeros((1, V)), [3], 3)          # uniform
    assert np.isclose(r["entropy"][0], np.log(V)) and np.isclose(r["logprob"][0], -np.log(V))
    assert r["rank"][0] == 3 and list(r["top_ids"][0]) == [0, 1, 2]
    x = np.log(np.array([[0.5, 0.25, 0.25, 1e-300]]))
    x[0, 3] = -np.inf                                   # masked: adds nothing
    r = ops.logprobs(x, [2], 2)
    assert np.isclose(r["entropy"][0], 1.5 * np.log(2)) and r["rank"][0] == 2
    assert list(r["top_ids"][0]) == [0, 1] and np.allclose(r["top_logprobs"][0], np.log([0.5, 0.25]))
    r = ops.logprobs(np.full((2, 3), -np.inf), [1, -1], 2)   # nothing left
    assert r["entropy"][0] == 0 and r["logprob"][0] == -np.inf and r["rank"][0] == 1
    assert r["logprob"][1] == 0 and r["rank"][1] == -1 and list(r["top_ids"][0]) == [0, 1]
