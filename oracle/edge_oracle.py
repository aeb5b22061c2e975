"""Float64 definitions of layer norm with dropout, grouped routing and 8-bit products (numpy, CPU).

TEST INFRASTRUCTURE ONLY, as the rest of this package.  Inputs are float64
arrays holding the exact values of the stored inputs.  Where a GPU result is
a sum, the function also returns the sum of the terms' magnitudes.

  philox / dropout_factor        the counter generator and what it keeps
  layer_norm / layer_norm_bwd    dropout, residual and norm between two blocks
  group_gate / group_gate_bwd    routing with expert groups
  q8_quantize / q8_gemm          rows in 8 bits and their products
"""
from __future__ import annotations

import numpy as np

__all__ = ["philox", "dropout_factor", "layer_norm", "layer_norm_bwd", "gate_scores", "group_gate", "group_gate_bwd",
           "q8_quantize", "q8_gemm"]


def philox(counter, key):
    """Philox4x32-10: counter [n, 4] and key [2] of 32-bit numbers -> [n, 4]."""
    c = [np.asarray(counter, np.uint64)[:, i] for i in range(4)]
    k = [int(key[0]), int(key[1])]
    low = np.uint64(0xFFFFFFFF)
    s = np.uint64(32)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> s) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> s) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, axis=1).astype(np.uint32)


def dropout_factor(T, H, p, seed, offset, first_row=0):
    """What every element is multiplied by, [T, H]: 0 or 65536 / keep."""
    keep = int(np.rint((1.0 - float(np.float32(p))) * 65536))
    block = (np.arange(T * H // 8, dtype=np.uint64) + np.uint64(first_row * H // 8))
    ctr = np.empty((block.size, 4), np.uint64)
    ctr[:, 0], ctr[:, 1] = block & np.uint64(0xFFFFFFFF), block >> np.uint64(32)
    ctr[:, 2], ctr[:, 3] = offset & 0xFFFFFFFF, offset >> 32
    words = philox(ctr, (seed & 0xFFFFFFFF, seed >> 32))
    bits = np.stack([words & 0xFFFF, words >> 16], axis=2).reshape(T, H)
    return np.where(bits < keep, 65536.0 / keep, 0.0)


def layer_norm(x, y, factor, weight, bias, eps):
    """(x', u, m, r, magnitude of x', of u); x None: zeros, y None: x' = x, factor None: nothing dropped."""
    z = 0.0 if y is None else y if factor is None else np.where(factor > 0, y * factor, 0.0)
    x1 = z + 0.0 if x is None else x + z
    mag = (0.0 if x is None else np.abs(x)) + np.abs(z)
    m = x1.mean(axis=1, keepdims=True)
    r = 1.0 / np.sqrt(((x1 - m) ** 2).mean(axis=1, keepdims=True) + eps)
    w = 1.0 if weight is None else weight
    b = 0.0 if bias is None else bias
    n = (x1 - m) * r
    # fp32 errors of the row (of size `top`) shift every distance from the mean and scale r
    top = mag.max(axis=1, keepdims=True)
    umag = np.abs(w) * (np.abs(n) * (1.0 + 2.0 * top * r) + 2.0 * top * r) + np.abs(b)
    return x1, n * w + b, m[:, 0], r[:, 0], mag, umag


def layer_norm_bwd(x1, m, r, weight, dx1, du, factor):
    """Gradients (value, magnitude) by name from the stored x' and its statistics."""
    out = {}
    d = np.zeros_like(du if dx1 is None else dx1) if dx1 is None else dx1.copy()
    dmag = np.abs(d)
    if du is not None:
        m, r = m[:, None], r[:, None]
        w = 1.0 if weight is None else weight
        n, nmag = (x1 - m) * r, (np.abs(x1) + np.abs(m)) * r
        g = du * w
        out["dw"] = ((du * n).sum(0), (np.abs(du) * nmag).sum(0))
        out["db"] = (du.sum(0), np.abs(du).sum(0))
        mean = lambda v: v.mean(axis=1, keepdims=True)  # noqa: E731
        d = d + r * (g - mean(g) - n * mean(g * n))
        dmag = dmag + r * (np.abs(g) + mean(np.abs(g)) + nmag * mean(np.abs(g) * nmag))
    out["dx"] = (d, dmag)
    out["dy"] = (d, dmag) if factor is None else (d * factor, dmag * factor)
    return out


def gate_scores(logits, score):
    """Scores [T, E] with the rules for odd rows."""
    z = np.where(np.isnan(logits), -np.inf, logits).astype(np.float64)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-z))
    top = z.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.where(np.isinf(top), (z == top).astype(np.float64), np.exp(z - top))
    return e / e.sum(axis=1, keepdims=True)


def group_gate(logits, bias, topk, score, groups, kept, top, renorm, scale):
    """ids [T, topk] and weights of the routing with groups, token by token."""
    T, E = logits.shape
    n = E // groups
    z = np.where(np.isnan(logits), -np.inf, logits).astype(np.float64)
    s = gate_scores(logits, score)
    c = z if bias is None else s + np.where(np.isnan(bias), -np.inf, bias)[None, :]
    ids = np.empty((T, topk), np.int32)
    weights = np.empty((T, topk))
    for t in range(T):
        if kept < groups:
            rank = []
            for g in range(groups):
                mine = slice(g * n, (g + 1) * n)
                if top == 1:
                    rank.append(c[t, mine].max())
                else:
                    v = s[t, mine] if bias is None else c[t, mine]
                    rank.append(np.sort(v)[::-1][:2].sum())
            rank = np.array(rank)
            rank[np.isnan(rank)] = -np.inf  # a bias of +inf beside one of -inf
            best = np.argsort(-rank, kind="stable")[:kept]
            pool = np.concatenate([np.arange(g * n, (g + 1) * n) for g in sorted(best)])
        else:
            pool = np.arange(E)
        pick = pool[np.argsort(-c[t, pool], kind="stable")[:topk]]
        ids[t] = pick
        if not renorm:
            w = s[t, pick]
        else:
            x = z[t, pick]
            peak = x.max()
            if (score == "softmax" and np.isinf(peak)) or peak == -np.inf:
                w = (x == peak).astype(np.float64)
            elif score == "softmax":
                w = np.exp(x - peak)
            else:  # sigmoid times e^-min(peak, 0), which the shares do not see
                w = np.exp(np.minimum(x, 0.0) - min(peak, 0.0)) / (1.0 + np.exp(-np.abs(x)))
            w = w / w.sum()
        weights[t] = scale * w
    return ids, weights


def group_gate_bwd(logits, ids, dweights, score, renorm, scale):
    """(d logits, magnitude) [T, E]; ids outside [0, E) add nothing."""
    T, E = logits.shape
    z = np.where(np.isnan(logits), -np.inf, logits).astype(np.float64)
    s = gate_scores(logits, score)
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        ok = (ids[t] >= 0) & (ids[t] < E)
        e, g = ids[t][ok], scale * dweights[t][ok]
        if e.size == 0:
            continue
        x = z[t, e]
        if renorm:
            peak = x.max()
            if (score == "softmax" and np.isinf(peak)) or peak == -np.inf:
                continue
            v = np.exp(x - peak) if score == "softmax" else \
                np.exp(np.minimum(x, 0.0) - min(peak, 0.0)) / (1.0 + np.exp(-np.abs(x)))
            v = v / v.sum()
            left = 1.0 if score == "softmax" else 1.0 / (1.0 + np.exp(np.minimum(x, 700.0)))
            d[t, e] = v * left * (g - (v * g).sum())
            mag[t, e] = v * left * (np.abs(g) + (v * np.abs(g)).sum())
        elif score == "sigmoid":
            d[t, e] = s[t, e] * (1.0 / (1.0 + np.exp(np.minimum(x, 700.0)))) * g
            mag[t, e] = np.abs(d[t, e])
        else:
            if np.isinf(z[t].max()):
                continue
            up, upmag = np.zeros(E), np.zeros(E)
            up[e], upmag[e] = g, np.abs(g)
            d[t] = s[t] * (up - (s[t] * up).sum())
            mag[t] = s[t] * (upmag + (s[t] * upmag).sum())
    return d, mag


def q8_quantize(x):
    """int8 codes and float32 scales of rows (float64 values of 16-bit numbers)."""
    rows, K = x.shape
    q, scales = np.zeros((rows, K), np.int8), np.zeros(rows, np.float32)
    for i in range(rows):
        top = np.abs(x[i]).max() if K else 0.0
        scales[i] = np.float32(top) / np.float32(127.0)
        if np.isfinite(scales[i]) and scales[i] > 0:
            q[i] = np.rint(x[i] / np.float64(scales[i])).astype(np.int8)
    return q, scales


def q8_gemm(x, x_scales, w, w_scales, bias):
    """(out, magnitude of the scaled sum and the bias, largest sum of magnitudes)."""
    total = x.astype(np.int64) @ w.astype(np.int64).T
    reach = np.abs(x.astype(np.int64)) @ np.abs(w.astype(np.int64)).T
    out = total * x_scales[:, None].astype(np.float64) * w_scales[None, :].astype(np.float64)
    mag = np.abs(out)
    if bias is not None:
        out, mag = out + bias, mag + np.abs(bias)
    return out, mag, int(reach.max()) if reach.size else 0
