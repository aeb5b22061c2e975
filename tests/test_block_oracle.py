"""Pins of the block oracle: gradients against central differences, closed
forms, hand-placed nibbles (CPU only)."""
import math

import numpy as np
import pytest

import oracle


def _diff(f, x, at, h=1e-5):
    p, m = x.copy(), x.copy()
    p[at] += h
    m[at] -= h
    return (f(p) - f(m)) / (2 * h)


@pytest.mark.parametrize("post_norm", [True, False])
@pytest.mark.parametrize("gate", [None, (1, 12), (3, 12), (6, 1), (2, 1)])
def test_norm_gradients_are_differences(post_norm, gate):
    r = np.random.default_rng(1)
    T, H, eps, rho = 6, 12, 1e-3, 0.7
    v = {"x": r.standard_normal((T, H)), "y": r.standard_normal((T, H)), "w_pre": r.standard_normal(H),
         "rho": np.array([rho])}
    v["w_post"] = r.standard_normal(H) if post_norm else None
    v["gate"] = None if gate is None else r.standard_normal(gate)
    dx1, du = r.standard_normal((T, H)), r.standard_normal((T, H))

    def loss(**kw):
        a = {**v, **kw}
        x1, u, _, _ = oracle.block_norm(a["x"], a["y"], a["w_post"], a["gate"], a["rho"][0], a["w_pre"], eps, post_norm)
        return (x1 * dx1).sum() + (u * du).sum()

    got = oracle.block_norm_bwd(v["x"], v["y"], v["w_post"], v["gate"], rho, v["w_pre"], eps, dx1, du, post_norm)
    names = {"x": "dx", "y": "dy", "w_pre": "dw_pre", "rho": "dres", "w_post": "dw_post", "gate": "dgate"}
    for name, grad in names.items():
        if v[name] is None:
            assert grad not in got
            continue
        for at in [tuple(r.integers(0, s) for s in v[name].shape) for _ in range(6)]:
            want = _diff(lambda a: loss(**{name: a}), v[name], at)
            assert abs(got[grad][0][at] - want) < 1e-6 * (1 + abs(want)), (name, at)


def test_norm_of_constant_rows():
    x = np.full((2, 8), 3.0)
    x1, u, r_y, r_x = oracle.block_norm(x, None, None, None, 1.0, None, 0.0)
    assert np.array_equal(x1, x) and r_y is None
    assert np.allclose(r_x, 1 / 3) and np.allclose(u, 1.0)


def _router_case(T=12, E=5, k=2, S=3, seed=0, mask=True):
    r = np.random.default_rng(seed)
    logits = r.standard_normal((T, E))
    ids, w = oracle.moe_topk_gate(logits.astype(np.float32), k)
    m = (r.random(T) < 0.7).astype(np.uint8) if mask else None
    return logits, ids, w.astype(np.float64), S, m


def test_router_gradient_is_differences():
    logits, ids, _, S, mask = _router_case()
    T, E = logits.shape
    k, a, b = ids.shape[1], 0.3, 0.2
    dw = np.random.default_rng(5).standard_normal((T, k))

    def gate(z):
        s = np.take_along_axis(z, ids.astype(np.int64), 1)
        e = np.exp(s - s.max(1, keepdims=True))
        return e / e.sum(1, keepdims=True)

    def total(z):  # the choice of experts held fixed
        loss, *_ = oracle.balance_loss(z, ids, S, a, b, mask)
        return 0.6 * loss[0] + 1.7 * loss[1] + (gate(z) * dw).sum()

    _, counts, _, tokens, _ = oracle.balance_loss(logits, ids, S, a, b, mask)
    got, _ = oracle.router_bwd(logits, ids, gate(logits), S, a, b, counts, tokens, (0.6, 1.7), dw, mask)
    for t in range(T):
        for e in range(E):
            assert abs(got[t, e] - _diff(total, logits, (t, e))) < 1e-7


def test_balance_loss_of_a_perfect_balance_is_its_coefficient():
    # every expert gets its share of slots and of probability: f P sums to 1 / E x E
    E, k, S = 4, 2, 2
    ids = np.array([[0, 1], [2, 3]] * 4, np.int32)
    loss, counts, probs, tokens, lse = oracle.balance_loss(np.zeros((8, E)), ids, S, 0.01, 1.0)
    assert abs(loss[0] - 0.01) < 1e-15 and abs(loss[1] - math.log(E) ** 2) < 1e-12
    assert (counts == 2).all() and np.allclose(probs, 0.25) and tokens.tolist() == [4, 4, 8]


def test_router_odd_rows():
    p, lse = oracle.router_softmax([math.nan, 0.0, math.nan])
    assert p == [0.0, 1.0, 0.0] and lse == 0.0
    p, lse = oracle.router_softmax([math.inf, 0.0, math.inf])
    assert p == [0.5, 0.0, 0.5] and lse == math.inf
    p, lse = oracle.router_softmax([-math.inf] * 4)
    assert p == [0.25] * 4 and lse == -math.inf


def test_w4_format_by_hand():
    # input 0: first nibble; 1: fifth; 2: second; 8: byte 16; 32: byte 4; 128: byte 64
    for k, (byte, shift) in {0: (0, 0), 1: (2, 0), 2: (0, 4), 7: (3, 4), 8: (16, 0), 32: (4, 0), 128: (64, 0)}.items():
        codes = np.zeros((1, 129), np.int64)
        codes[0, k] = 15
        q = oracle.w4_pack(codes)
        assert q.shape == (1, 128)
        want = np.zeros(128, np.uint8)
        want[byte] = 15 << shift
        assert (q[0, :64] == want[:64]).all() and q[0, byte] & (15 << shift) == 15 << shift
    r = np.random.default_rng(2).integers(0, 16, (3, 2, 200))
    assert np.array_equal(oracle.w4_codes(oracle.w4_pack(r), 200), r)


def test_w4_quantize_error_is_half_a_step():
    w = np.random.default_rng(3).standard_normal((2, 96, 8))
    codes, scales = oracle.w4_quantize(w, 32, lambda s: oracle.round_to(s, "bf16"))
    back = oracle.w4_weights(oracle.w4_pack(codes), scales, 96, 32)
    step = np.repeat(scales, 32, axis=1)
    # a scale rounded down by 2^-9 puts the largest magnitude 7 (1 + 2^-9) steps out
    assert (np.abs(back - w) <= step * (0.5 + 7 * 2.0 ** -8)).all()


def test_w4_layers_are_the_products_of_their_experts():
    r = np.random.default_rng(4)
    T, k, E, K, N = 5, 2, 3, 16, 8
    W = r.standard_normal((E, K, N))
    ids = np.array([[0, 1], [2, 0], [1, 2], [1, 9], [-1, 0]], np.int32)
    x, w = r.standard_normal((T, K)), r.random((T, k))
    h, _ = oracle.w4_layer0(x, W, ids)
    assert np.allclose(h[3], x[1] @ W[0]) and not h[7].any() and not h[8].any()
    h = r.standard_normal((T * k, K))
    y, _ = oracle.w4_layer1(h, W, ids, w)
    assert np.allclose(y[2], w[2, 0] * h[4] @ W[1] + w[2, 1] * h[5] @ W[2])
    assert np.allclose(y[3], w[3, 0] * h[6] @ W[1])
