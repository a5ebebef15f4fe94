"""The 64-bit references of the e4m3 rows and products themselves (CPU)."""
import numpy as np
import torch

from tests import f8ref


def test_values_are_torch_s():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).float().double().numpy()
    np.testing.assert_array_equal(f8ref.VALUES, want)


def test_encode_rounds_to_the_nearest_even():
    held = f8ref.HELD
    for i in range(126):
        mid = (held[i] + held[i + 1]) / 2
        assert f8ref.encode(mid) == (i if i % 2 == 0 else i + 1)
        assert f8ref.encode(np.nextafter(mid, 0)) == i and f8ref.encode(np.nextafter(mid, 500)) == i + 1
        assert f8ref.encode(held[i]) == i and f8ref.encode(-held[i + 1]) == i + 1 + 128
    assert f8ref.encode(460.0) == 126 and f8ref.encode(1e9) == 126
    x = np.random.default_rng(0).standard_normal(5000).astype(np.float32) * 30
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(f8ref.encode(x), want)


def test_a_worked_product():
    # two blocks: 1 * 2 * 3 values of 0.5 * 2, then 4 values of -1 * 448 at scales 0.25 and 2
    xc, wc = np.zeros((1, 132), np.uint8), np.zeros((1, 132), np.uint8)
    xc[0, :3], wc[0, :3] = f8ref.encode(0.5), f8ref.encode(2.0)
    xc[0, 128:], wc[0, 128:] = f8ref.encode(-1.0), f8ref.encode(448.0)
    y, _, _ = f8ref.product(xc, np.float32([[2.0, 0.25]]), wc, np.float32([[1.0, 2.0]]), np.float32([7.0]))
    assert y[0, 0] == 3 * 2 - 4 * 448 * 0.5 + 7


def test_a_worked_selection():
    inf = np.inf
    z = np.array([[0.0, 2.0, 2.0, -inf], [-inf, -inf, np.nan, -inf], [inf, 0.0, -1.0, 5.0]])
    e, w, p, r, o = f8ref.select(z, 3, True)
    assert e.tolist() == [[1, 2, 0], [-1, -1, -1], [0, 3, 1]]
    assert o.tolist() == [0, 2, 4, 5, 6] and r.tolist() == [0, 2, 0, 2, 0, 2, -1, -1, -1]
    assert p.tolist() == [[2, 4, 0], [-1, -1, -1], [1, 5, 3]]
    assert np.allclose(w[0], np.exp([0, 0, -2.0]) / (2 + np.exp(-2))) and w[2].tolist() == [1.0, 0.0, 0.0]
