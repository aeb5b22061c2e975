"""Float64 definitions of the operators around an MoE block (numpy, CPU).

TEST INFRASTRUCTURE ONLY, as the rest of this package.  Inputs are float64
arrays holding the exact values of the stored inputs.  Where a GPU result is
a sum, the function also returns the sum of the terms' magnitudes, from which
a test derives how far fp32 arithmetic may be off.

  block_norm / block_norm_bwd   norms, gate and residual between two blocks
  balance_loss / router_bwd     balance and z losses, gradient of the scores
  w4_codes / w4_quantize        the 4-bit weight format
  w4_gemv / w4_layer0 / w4_layer1
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["block_norm", "block_norm_bwd", "router_softmax", "balance_loss", "router_bwd", "w4_codes",
           "w4_pack", "w4_place", "w4_quantize", "w4_weights", "w4_gemv", "w4_layer0", "w4_layer1"]


def _gate_rows(gate, T, H):
    """The gate of every token, [T, H]."""
    if gate is None:
        return np.ones((T, H))
    g = np.asarray(gate, np.float64)
    return np.broadcast_to(np.repeat(g, T // g.shape[0], axis=0), (T, H))


def block_norm(x, y, w_post, gate, rho, w_pre, eps, post_norm=True):
    """(x', u, r_y, r_x); y None: x' = x.  w_* None: ones."""
    T, H = x.shape
    r_y = None
    if y is None:
        x1 = x
    else:
        z = y
        if post_norm:
            r_y = 1.0 / np.sqrt((y * y).mean(axis=1) + eps)
            z = y * r_y[:, None] * (1.0 if w_post is None else w_post)
        x1 = rho * x + _gate_rows(gate, T, H) * z
    r_x = 1.0 / np.sqrt((x1 * x1).mean(axis=1) + eps)
    u = x1 * r_x[:, None] * (1.0 if w_pre is None else w_pre)
    return x1, u, r_y, r_x


def block_norm_bwd(x, y, w_post, gate, rho, w_pre, eps, dx1, du, post_norm=True):
    """Gradients by the chain rule, each a (value, magnitude) pair, by name.

    dx1 None: zeros; du None: the forward call had no u.
    """
    T, H = x.shape
    x1, _, r_y, r_x = block_norm(x, y, w_post, gate, rho, w_pre, eps, post_norm)
    out = {}
    d = np.zeros((T, H)) if dx1 is None else dx1.copy()
    dmag = np.abs(d)
    if du is not None:
        wp = np.ones(H) if w_pre is None else w_pre
        xn = x1 * r_x[:, None]
        # the magnitude of x' is that of its two terms: the GPU computes it again
        x1mag = np.abs(x1) if y is None else np.abs(rho * x) + np.abs(x1 - rho * x)
        xnmag = x1mag * r_x[:, None]
        out["dw_pre"] = ((du * xn).sum(0), (np.abs(du) * xnmag).sum(0))
        g = du * wp
        d = d + r_x[:, None] * (g - xn * (g * xn).mean(axis=1, keepdims=True))
        dmag = dmag + r_x[:, None] * (np.abs(g) + xnmag * (np.abs(g) * xnmag).mean(axis=1, keepdims=True))
    out["dx"] = (rho * d if y is not None else d, np.abs(rho) * dmag if y is not None else dmag)
    if y is not None:
        G = _gate_rows(gate, T, H)
        yn = y * r_y[:, None] if post_norm else y
        wq = np.ones(H) if w_post is None or not post_norm else w_post
        z = yn * wq
        out["dres"] = (np.array([(d * x).sum()]), np.array([(dmag * np.abs(x)).sum()]))
        if gate is not None:
            rows, cols = np.asarray(gate).shape
            for k, v in (("v", d * z), ("m", dmag * np.abs(z))):
                if cols == 1:
                    v = v.sum(axis=1, keepdims=True)
                out[k] = v.reshape(rows, T // rows, cols).sum(axis=1)
            out["dgate"] = (out.pop("v"), out.pop("m"))
        dz, dzmag = d * G, dmag * np.abs(G)
        if post_norm:
            out["dw_post"] = ((dz * yn).sum(0), (dzmag * np.abs(yn)).sum(0))
            c, cmag = dz * wq, dzmag * np.abs(wq)
            dy = r_y[:, None] * (c - yn * (c * yn).mean(axis=1, keepdims=True))
            dymag = r_y[:, None] * (cmag + np.abs(yn) * (cmag * np.abs(yn)).mean(axis=1, keepdims=True))
            out["dy"] = (dy, dymag)
        else:
            out["dy"] = (dz, dzmag)
    return out


def router_softmax(row):
    """(p, lse) of one token's scores with the gate's rules for odd rows."""
    row = [-math.inf if math.isnan(v) else float(v) for v in row]
    top = max(row)
    if math.isinf(top):
        hit = [1.0 if v == top else 0.0 for v in row]
        return [h / sum(hit) for h in hit], top
    e = [math.exp(v - top) for v in row]
    s = math.fsum(e)
    return [v / s for v in e], top + math.log(s)


def balance_loss(logits, ids, S, balance_coef, z_coef, mask=None):
    """loss [2], counts [S, E], probs [S, E], tokens [S + 1], lse [T], token by token."""
    T, E = logits.shape
    k = ids.shape[1]
    counts, probs = np.zeros((S, E), np.int64), np.zeros((S, E))
    tokens, lse, z = np.zeros(S + 1, np.int64), np.zeros(T), 0.0
    for t in range(T):
        s = t // (T // S)
        p, lse[t] = router_softmax(logits[t])
        if mask is not None and mask[t] == 0:
            continue
        tokens[s] += 1
        probs[s] += p
        z += lse[t] ** 2 if math.isfinite(lse[t]) else 0.0
        for e in ids[t]:
            if 0 <= e < E:
                counts[s, e] += 1
    tokens[S] = tokens[:S].sum()
    bal = 0.0
    for s in range(S):
        if tokens[s]:
            probs[s] /= tokens[s]
            bal += float((counts[s] / tokens[s] * probs[s]).sum())
    loss = np.array([balance_coef * E / (k * S) * bal, z_coef * z / max(tokens[S], 1)])
    return loss, counts, probs, tokens, lse


def router_bwd(logits, ids, weights, S, balance_coef, z_coef, counts, tokens, dloss, dweights, mask=None):
    """(dlogits, magnitude)."""
    T, E = logits.shape
    k = ids.shape[1]
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        s = t // (T // S)
        p, lse = router_softmax(logits[t])
        if math.isinf(lse):
            continue
        p = np.array(p)
        if mask is None or mask[t] != 0:
            a = dloss[0] * balance_coef * E * counts[s] / (k * S * float(tokens[s]) ** 2)
            zt = dloss[1] * 2 * z_coef * lse / tokens[S]
            out[t] = p * (a - (p * a).sum() + zt)
            mag[t] = p * (np.abs(a) + (p * np.abs(a)).sum() + abs(zt))
        if dweights is not None:
            dot = sum(weights[t, j] * dweights[t, j] for j in range(k))
            dmag = sum(abs(weights[t, j] * dweights[t, j]) for j in range(k))
            for j in range(k):
                if 0 <= ids[t, j] < E:
                    out[t, ids[t, j]] += weights[t, j] * (dweights[t, j] - dot)
                    mag[t, ids[t, j]] += weights[t, j] * (abs(dweights[t, j]) + dmag)
    return out, mag


def w4_place(k):
    """(byte in the column, shift) of input k."""
    run, r = divmod(k, 128)
    j, r = divmod(r, 32)
    c, r = divmod(r, 8)
    nibble = r // 2 + (4 if r % 2 else 0)
    return run * 64 + c * 16 + j * 4 + nibble // 2, 4 * (nibble % 2)


def w4_pack(codes):
    """uint8 [.., N, 64 ceil(K / 128)] from codes [.., N, K] (unused codes 8)."""
    K = codes.shape[-1]
    runs = -(-K // 128)
    out = np.zeros(codes.shape[:-1] + (runs * 64,), np.uint8)
    for k in range(runs * 128):
        byte, shift = w4_place(k)
        out[..., byte] |= (codes[..., k].astype(np.uint8) if k < K else np.uint8(8)) << np.uint8(shift)
    return out


def w4_codes(q, K):
    """Codes [.., N, K] from packed bytes."""
    out = np.zeros(q.shape[:-1] + (K,), np.int64)
    for k in range(K):
        byte, shift = w4_place(k)
        out[..., k] = (q[..., byte] >> shift) & 15
    return out


def w4_weights(q, scales, K, group):
    """W [E, K, N] in float64 from bytes [E, N, ..] and scales [E, groups, N]."""
    codes = w4_codes(q, K).astype(np.float64)
    out = np.zeros((q.shape[0], K, q.shape[1]))
    for k in range(K):
        out[:, k] = (codes[:, :, k] - 8) * scales[:, k // group]
    return out


def w4_quantize(w, group, round16):
    """(codes [E, N, K], scales [E, groups, N]) of weights [E, K, N]; round16 rounds a scale."""
    E, K, N = w.shape
    groups = -(-K // group)
    codes, scales = np.full((E, N, K), 8, np.int64), np.zeros((E, groups, N))
    for g in range(groups):
        part = w[:, g * group:(g + 1) * group]
        # the device divides in fp32
        top = np.float32(np.abs(part).max(axis=1)) / np.float32(7)
        scales[:, g] = round16(top.astype(np.float64))
        for e in range(E):
            for n in range(N):
                if scales[e, g, n] > 0:
                    q = np.rint(np.float32(part[e, :, n]) / np.float32(scales[e, g, n]))
                    codes[e, n, g * group:g * group + part.shape[1]] = np.clip(q + 8, 0, 15)
    return codes, scales


def w4_gemv(x, W):
    """(x . W, sum of magnitudes)."""
    return x @ W, np.abs(x) @ np.abs(W)


def w4_layer0(x, W, ids):
    """Rows in slot order: x[t] . W[ids[t, j]], zeros for an id out of range."""
    T, k = ids.shape
    out, mag = np.zeros((T * k, W.shape[2])), np.zeros((T * k, W.shape[2]))
    for t in range(T):
        for j in range(k):
            if 0 <= ids[t, j] < W.shape[0]:
                out[t * k + j], mag[t * k + j] = w4_gemv(x[t], W[ids[t, j]])
    return out, mag


def w4_layer1(h, W, ids, weights):
    T, k = ids.shape
    rows, mags = w4_layer0(h, W, ids.reshape(-1, 1)) if k else (None, None)
    w = weights[:, :, None]
    return (rows.reshape(T, k, -1) * w).sum(1), (mags.reshape(T, k, -1) * np.abs(w)).sum(1)
