"""The experts' and dropout oracle against hand cases, published vectors and differences."""
import numpy as np

from oracle import expert_oracle as eo


def test_sort_by_hand():
    row_of, slot_of, bounds = eo.sort(np.array([[2, 0], [-1, 2], [0, 7], [2, 2]]), 3)
    assert bounds.tolist() == [0, 2, 2, 6]
    assert slot_of.tolist() == [1, 4, 0, 3, 6, 7, 2, 5]
    assert row_of.tolist() == [[2, 0], [6, 3], [1, 7], [4, 5]]


def test_philox_vectors():
    """Philox4x32-10: the vectors published with the generator."""
    assert eo.philox4x32((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    ones = 0xFFFFFFFF
    assert eo.philox4x32((ones,) * 4, (ones,) * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert eo.philox4x32((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_dropout_by_hand():
    x = np.arange(1.0, 12.0)
    bits = eo.drop_bits(11, 5, 9)
    words = eo.philox4x32((0, 0, 9, 0), (5, 0)) + eo.philox4x32((1, 0, 9, 0), (5, 0))
    assert bits.tolist() == [v for w in words for v in (w & 0xFFFF, w >> 16)][:11]
    y = eo.dropout(x, 0.25, 5, 9)
    assert np.array_equal(y, np.where(bits >= 16384, x / 0.75, 0.0))
    assert not eo.dropout(x, 1.0, 5, 9).any() and np.array_equal(eo.dropout(x, 0.0, 5, 9, residual=x), 2 * x)


def test_round_trip_and_gradients():
    """The gradients are those of a sum over the formulas, by central differences."""
    rng = np.random.default_rng(0)
    T, k, D, E = 5, 3, 4, 4
    experts = rng.integers(-1, E, (T, k))
    row_of, slot_of, bounds = eo.sort(experts, E)
    live = bounds[-1]
    x, w, res = rng.normal(size=(T, D)), rng.normal(size=(T, k)), rng.normal(size=(T, D))
    dy = rng.normal(size=(T, D))
    scale = 1.0 + np.arange(T * k)[:, None]         # what the experts do to their rows

    def f(x, w):
        return float((dy * eo.combine(eo.dispatch(x, row_of, live) * scale, row_of, live, w, res)).sum())

    ys = eo.dispatch(x, row_of, live) * scale
    dys, dw = eo.combine_backward(dy, ys, row_of, live, w)
    dx = eo.combine(dys * scale, row_of, live)      # the gradient of dispatch
    h = 1e-6
    for arr, grad, pos in ((x, dx, 0), (w, dw, 1)):
        for i in np.ndindex(arr.shape):
            up, dn = arr.copy(), arr.copy()
            up[i] += h
            dn[i] -= h
            num = (f(up, w) - f(dn, w) if pos == 0 else f(x, up) - f(x, dn)) / (2 * h)
            assert abs(num - grad[i]) < 1e-6 * (1 + abs(num))
    assert (experts.reshape(-1)[slot_of[live:]] == -1).all()


def test_product_gradients():
    """The experts' block and layer: gradients by central differences of a sum over the forward formulas."""
    rng = np.random.default_rng(1)
    R, E, D, F = 7, 3, 4, 5
    bounds = [0, 2, 2, 6]
    x, dh, dy = rng.normal(size=(R, D)), rng.normal(size=(R, F)), rng.normal(size=(R, D))
    wg, wu, wd = rng.normal(size=(E, F, D)), rng.normal(size=(E, F, D)), rng.normal(size=(E, D, F))
    h, gate, up = eo.glu_forward(x, wg, wu, bounds, "silu")
    assert not h[6].any() and h[:2].any()
    grads = eo.glu_backward(x, wg, wu, gate, up, dh, bounds, "silu")
    lin = eo.linear_backward(dh, wd, dy, bounds)
    assert not grads[1][1].any() and not lin[1][1].any()

    def differences(f, args, k):
        out = np.zeros(args[k].shape)
        for i in np.ndindex(out.shape):
            up_, dn = [a.copy() for a in args], [a.copy() for a in args]
            up_[k][i] += 1e-6
            dn[k][i] -= 1e-6
            out[i] = (f(*up_) - f(*dn)) / 2e-6
        return out

    def block(x, wg, wu):
        return float((dh * eo.glu_forward(x, wg, wu, bounds, "silu")[0]).sum())

    def layer(v, w):
        return float((dy * eo.linear_forward(v, w, bounds)).sum())
    for k, g in enumerate(grads):
        assert np.allclose(differences(block, [x, wg, wu], k), g, rtol=1e-5, atol=1e-6)
    for k, g in enumerate(lin):
        assert np.allclose(differences(layer, [dh, wd], k), g, rtol=1e-5, atol=1e-6)


def test_segments():
    assert eo.segments([7, 3, 1, 9, -2], 6) == [(0, 3), (3, 3), (1, 6), (6, 6)]
