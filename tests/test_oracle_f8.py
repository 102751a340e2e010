"""The fp64 restatement of the 8-bit expert layer, by hand and against torch's own
conversion to e4m3."""
import numpy as np
import torch

from oracle import f8


def test_e4m3_as_torch_rounds():
    rng = np.random.default_rng(1)
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    every = np.sort(every[np.isfinite(every)])
    halves = (every[1:] + every[:-1]) / 2
    v = np.concatenate([every, halves, rng.normal(0, 100, 5000).clip(-448, 448), rng.normal(0, 1e-3, 5000)])
    v = v.astype(np.float32)
    assert np.array_equal(f8.e4m3(v), torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy())


def test_quotients_by_hand():
    x = np.zeros((2, 130))
    x[0, 0], x[0, 5], x[0, 129], x[1, 3] = 2.0, -1.0, 0.5, 4.0
    v, s = f8.quotients(x)
    assert v[0, 0] == 448 and v[0, 5] == -224 and v[0, 129] == 448 and v[1, 129] == 0
    assert np.allclose(s, [[2 / 448, 0.5 / 448], [4 / 448, 0]])
    v, s = f8.quotients(x, 128)
    assert v[0, 0] == 224 and v[1, 3] == 448 and s.shape == (1, 2)


def test_linear_by_hand():
    x, w = np.ones((1, 129)), np.ones((129, 129))
    xs, ws = np.array([[2.0, 3.0]]), np.array([[1.0, 10.0], [5.0, 7.0]])
    out, size = f8.linear(x, xs, w, ws)
    assert out[0, 0] == 2 * 128 + 30 and out[0, 128] == 2 * 5 * 128 + 21 and (size == out).all()


def test_route_by_hand():
    x = np.array([[0.0, np.log(3.0), 0.0], [5.0, 5.0, -np.inf], [-np.inf] * 3])
    r = f8.route(x, 2, False)
    assert r["idx"].tolist() == [[1, 0], [0, 1], [0, 1]]
    assert np.allclose(r["weight"], [[0.6, 0.2], [0.5, 0.5], [0, 0]])
    assert r["offsets"].tolist() == [0, 3, 6, 6] and r["perm"].tolist() == [1, 2, 4, 0, 3, 5]
    assert np.allclose(f8.route(x, 2, True)["weight"][0], [0.75, 0.25])


def test_combine_by_hand():
    y = np.array([[1.0], [10.0], [np.nan]])
    out, _ = f8.combine(y, [[2.0, 0.5, 0.0]], [1, 0, 2], [[100.0]])
    assert out[0, 0] == 120.5
    assert f8.combine(y, [[2.0, 0.5]], [-1, 3])[0][0, 0] == 0
