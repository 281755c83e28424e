"""The reference of the token, int8 and dropout operators against values worked
out by hand, published test vectors, and differences."""
import numpy as np

from oracle import tokens as ot


def test_sort_by_hand():
    rows, choices, counts = ot.sort([[2, 0], [-1, 2], [0, 3]], 3)
    # choices 0..5 hold experts 2 0 . 2 0 . ; expert 0: 1, 4; expert 2: 0, 3; dropped: 2, 5
    assert choices.tolist() == [1, 4, 0, 3, 2, 5]
    assert rows.tolist() == [[2, 0], [~4, 3], [1, ~5]]
    assert counts.tolist() == [2, 0, 2]


def test_there_and_back():
    rng = np.random.default_rng(0)
    rows, _, counts = ot.sort(rng.integers(-1, 4, (7, 3)), 4)
    x = rng.standard_normal((7, 5))
    y = ot.dispatch(x, rows, 21)
    kept = (rows >= 0).sum(1)
    assert np.allclose(ot.combine(y, rows)[0], x * kept[:, None])
    assert (y[counts.sum():] == 0).all()
    assert ot.dispatch(x, rows, int(counts.sum())).shape == (counts.sum(), 5)


def test_combine_gradient_against_differences():
    rng = np.random.default_rng(1)
    rows, _, _ = ot.sort(rng.integers(-1, 3, (4, 2)), 3)
    y, w, d = rng.standard_normal((8, 3)), rng.random((4, 2)), rng.standard_normal((4, 3))
    dy, dw, _ = ot.combine_bwd(d, y, rows, w)

    def f(y, w):
        return (ot.combine(y, rows, w)[0] * d).sum()
    for i in np.ndindex(y.shape):
        e = np.zeros(y.shape)
        e[i] = 1e-3
        assert np.isclose((f(y + e, w) - f(y - e, w)) / 2e-3, dy[i], atol=1e-9)
    for i in np.ndindex(w.shape):
        e = np.zeros(w.shape)
        e[i] = 1e-3
        assert np.isclose((f(y, w + e) - f(y, w - e)) / 2e-3, dw[i], atol=1e-9)


def test_int8_by_hand():
    q, s = ot.quantize_int8([[1.0, -2.0, 0.5, 0.0], [0, 0, 0, 0], [1, np.inf, 0, 0], [np.nan, 1, 2, 3]])
    # 127 / 2 = 63.5 and 127 / 4 = 31.75; a tie goes to the even code
    assert q.tolist() == [[64, -127, 32, 0], [0] * 4, [0] * 4, [0] * 4]
    assert s[0] == np.float32(2) / np.float32(127) and s[1] == 0 and np.isinf(s[2]) and np.isnan(s[3])
    out = ot.grouped_int8(np.array([[1, -2], [3, 4]], np.int8), np.array([2.0, 0.5]),
                          np.array([[[1, 1]], [[-128, 127]]], np.int8), np.array([[0.25], [1.0]]), [1, 1])
    assert out.tolist() == [[-0.5], [0.5 * (3 * -128 + 4 * 127)]]


def test_philox_published_vectors():
    # the known answers that the generator's authors publish with it
    for counter, key, want in (
            ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
             (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        assert tuple(int(v) for v in ot.philox4x32(np.array(counter, np.uint64), key)) == want


def test_dropout_mask():
    n = ot.dropout_numbers(100, 1000, seed=5, step=7, call=1)
    # 1e5 draws of 16 bits: the mean of n uniforms is within 5 standard deviations
    assert abs(n.mean() - 32767.5) < 5 * 65536 / np.sqrt(12 * n.size) and n.min() >= 0 and n.max() < 65536
    for other in (dict(seed=6, step=7, call=1), dict(seed=5, step=8, call=1), dict(seed=5, step=7, call=2)):
        assert (ot.dropout_numbers(100, 1000, **other) == n).mean() < 1e-3
    out, kept = ot.dropout(np.ones((100, 1000)), 0.25, 5, 7, 1)
    assert set(np.unique(out)) == {0.0, 4 / 3} and (kept == (out > 0)).all()
    assert not ot.dropout(np.ones((2, 8)), 1.0, 5, 7, 1)[0].any()
    assert (ot.dropout(np.ones((2, 8)), 0.0, 5, 7, 1)[0] == 1).all()
