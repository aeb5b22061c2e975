"""The float64 definitions of layer norm with dropout, grouped routing and 8-bit
products, pinned to published vectors, hand-worked cases and differences (CPU)."""
import numpy as np
import pytest

import oracle


def test_philox_published_vectors():
    # the known answers that the generator's authors publish for philox4x32-10
    full = 0xFFFFFFFF
    for ctr, key, want in [
            ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((full,) * 4, (full,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
             (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))]:
        assert tuple(int(v) for v in oracle.philox(np.array([ctr], np.uint64), key)[0]) == want


def test_dropout_factor_layout_and_share():
    f = oracle.dropout_factor(4, 64, 0.25, 5, 9)
    words = oracle.philox(np.array([[3, 0, 9, 0]], np.uint64), (5, 0))[0]  # elements 24 .. 31
    keep = 49152
    for j in range(8):
        bits = int(words[j // 2]) >> (16 * (j % 2)) & 0xFFFF
        assert f[0, 24 + j] == (65536 / keep if bits < keep else 0.0)
    f = oracle.dropout_factor(512, 1024, 0.1, 123, 1 << 33)
    n, q = f.size, 58982 / 65536
    assert abs((f > 0).sum() - n * q) < 6 * np.sqrt(n * q * (1 - q))
    assert np.array_equal(f[256:], oracle.dropout_factor(256, 1024, 0.1, 123, 1 << 33, first_row=256))


def _difference(f, x, h=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + h
        hi = f()
        x[i] = keep - h
        lo = f()
        x[i] = keep
        g[i] = (hi - lo) / (2 * h)
    return g


def test_layer_norm_gradients_against_differences():
    r = np.random.default_rng(0)
    T, H, eps = 3, 16, 1e-3
    x, y, w, b = r.standard_normal((T, H)), r.standard_normal((T, H)), r.standard_normal(H), r.standard_normal(H)
    a, c = r.standard_normal((T, H)), r.standard_normal((T, H))
    f = oracle.dropout_factor(T, H, 0.3, 7, 1)

    def loss():
        x1, u = oracle.layer_norm(x, y, f, w, b, eps)[:2]
        return (a * x1).sum() + (c * u).sum()

    x1, _, m, rs = oracle.layer_norm(x, y, f, w, b, eps)[:4]
    got = oracle.layer_norm_bwd(x1, m, rs, w, a, c, f)
    for name, arr in (("dx", x), ("dy", y), ("dw", w), ("db", b)):
        np.testing.assert_allclose(got[name][0], _difference(loss, arr), rtol=1e-6, atol=1e-7)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_group_gate_gradients_against_differences(score, renorm):
    r = np.random.default_rng(1)
    z, bias = r.standard_normal((4, 12)), r.standard_normal(12)
    ids, _ = oracle.group_gate(z, bias, 3, score, 4, 2, 2, renorm, 2.5)
    dw = r.standard_normal((4, 3))

    def loss():
        s = oracle.gate_scores(z, score)
        w = np.take_along_axis(s, ids.astype(np.int64), 1)
        if renorm:
            w = w / w.sum(1, keepdims=True)
        return 2.5 * (w * dw).sum()

    got, mag = oracle.group_gate_bwd(z, ids, dw, score, renorm, 2.5)
    np.testing.assert_allclose(got, _difference(loss, z), rtol=1e-6, atol=1e-9)
    assert (np.abs(got) <= mag + 1e-15).all()


def test_group_gate_hand_case():
    # groups of two: ranks 1.5, 1.6 (sum of both); the best expert of all is in the group left out
    s = np.array([[0.9, 0.6, 0.85, 0.75]])
    z = np.log(s / (1 - s))
    ids, w = oracle.group_gate(z, np.zeros(4), 2, "sigmoid", 2, 1, 2, True, 1.0)
    assert ids.tolist() == [[2, 3]]
    np.testing.assert_allclose(w, [[0.85 / 1.6, 0.75 / 1.6]])
    ids, w = oracle.group_gate(z, np.zeros(4), 2, "sigmoid", 2, 1, 1, False, 2.0)
    assert ids.tolist() == [[0, 1]]
    np.testing.assert_allclose(w, [[1.8, 1.2]])
    # the bias moves the choice and not the weights; equal values by index
    ids, w = oracle.group_gate(np.zeros((1, 4)), np.array([0.0, 0.1, 0.1, 0.0]), 3, "softmax", 1, 1, 1, True, 1.0)
    assert ids.tolist() == [[1, 2, 0]]
    np.testing.assert_allclose(w, [[1 / 3] * 3])


def test_q8_hand_case():
    x = np.array([[127.0, -63.5, 0.5, 1.5], [0, 0, 0, 0], [np.inf, 1, 2, 3]])
    q, s = oracle.q8_quantize(x)
    assert q[0].tolist() == [127, -64, 0, 2] and s[0] == 1.0  # halves to even
    assert q[1].tolist() == [0, 0, 0, 0] and s[1] == 0.0
    assert q[2].tolist() == [0, 0, 0, 0] and np.isinf(s[2])
    out, mag, reach = oracle.q8_gemm(q[:1], s[:1], np.array([[1, 2, 3, 4]], np.int8), np.array([0.5], np.float32), None)
    assert out.tolist() == [[0.5 * (127 - 128 + 8)]] and reach == 127 + 128 + 8
