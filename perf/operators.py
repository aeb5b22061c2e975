"""The operators around and inside an MoE block, as cases that can be timed and compared.

Three families, each with the calls that a user makes of the package (``own``
true) and a plain form of elementary torch operations in 32 bits (``own``
false):

* the norms around a block (``flux_block_norm`` / ``flux_block_norm_bwd``): the
  block's output is normalised, gated and added to the scaled residual stream,
  and the sum is normalised for the next block, all of it in one pass;
* the router's training side (``flux_moe_balance_loss`` / ``flux_moe_router_bwd``):
  balance and z losses with the per-expert counts, and the gradient of the
  router scores from both losses and from the gate weights;
* products of few rows with 4-bit weights (``flux_w4_gemv``,
  ``flux_moe_w4_layer0``, ``flux_moe_w4_layer1``): one decode step of an MLP or
  of an MoE layer.

``listed`` holds the cases, ``draw`` makes more of the same ranges.
"""
import math

import torch

own = False

#: One zeroed workspace, as a program keeps it for all of these calls.
WORKSPACE_BYTES = 64 << 20

F16, BF16, F32, F64 = torch.float16, torch.bfloat16, torch.float32, torch.float64
EPS = 1e-6


def _dtype(case):
    return {"f16": F16, "bf16": BF16}[case["dtype"]]


def _code(case):
    return {"f16": 0, "bf16": 1}[case["dtype"]]


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decoded token between two blocks: post-norm, residual and pre-norm of H 4096
        dict(name="norm_token", op="norm", bwd=False, form="both", R=1, T=1, H=4096, dtype="bf16", post=True,
             gate="none", G=1, res=False),
        # the residual stream of a training step, sharded over 8 ranks by rows, a gate per channel
        dict(name="norm_train", op="norm", bwd=False, form="both", R=8, T=32768, H=4096, dtype="bf16", post=True,
             gate="channel", G=1, res=True),
        # its backward pass, with the gradients of every weight
        dict(name="norm_train_bwd", op="norm", bwd=True, form="both", R=8, T=32768, H=4096, dtype="bf16", post=True,
             gate="channel", G=1, res=True),
        # a wide model in fp16 with a gate row for each of 31 sequences and an odd row count
        dict(name="norm_gated_bwd", op="norm", bwd=True, form="both", R=1, T=4061, H=12288, dtype="f16", post=True,
             gate="channel", G=31, res=False),
        # the router of the 8-expert layer on its 4096 tokens
        dict(name="balance_4096", op="balance", bwd=False, T=4096, E=8, k=2, S=1, mask=False),
        # many experts on a long batch, a balance loss for each of 64 padded sequences
        dict(name="balance_long", op="balance", bwd=False, T=131072, E=256, k=8, S=64, mask=True),
        # the router's gradient on a micro-batch
        dict(name="router_bwd_4096", op="balance", bwd=True, T=4096, E=8, k=2, S=1, mask=False),
        # and on the long batch
        dict(name="router_bwd_long", op="balance", bwd=True, T=131072, E=256, k=8, S=64, mask=True),
        # one token through an attention-sized projection: the launch and the tail count
        dict(name="w4_token", op="w4", M=1, N=4096, K=4096, group=128, dtype="bf16"),
        # 13 decoding requests through the 70B-class down-projection
        dict(name="w4_down_13", op="w4", M=13, N=8192, K=28672, group=64, dtype="f16"),
        # up-projections of the 8-expert layer for 4 tokens
        dict(name="moe_w4_up_4", op="moe0", T=4, N=14336, K=4096, E=8, k=2, group=128, dtype="bf16"),
        # down-projections and the weighted combine of 64 small experts for 24 tokens
        dict(name="moe_w4_down_24", op="moe1", T=24, N=4096, K=1792, E=64, k=6, group=32, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["f16", "bf16"])
    op = rng.choice(["norm", "norm_bwd", "balance", "balance_bwd", "w4", "moe0", "moe1"])
    if op.startswith("norm"):
        H = 8 * _log(rng, 8, 2048)
        R = rng.choice([1, 1, 2, 4, 8])
        rows = max(1, _log(rng, 1, max(1, min(32768, (1 << 27) // H))) // R)
        T = R * rows
        gate = rng.choice(["none", "channel", "channel", "token"])
        G = T if gate == "token" else 1
        if gate == "channel" and rng.random() < 0.5:
            G = rng.choice([g for g in (1, 2, 3, 5, 8, 31, 64, T) if T % g == 0 and (g <= 64 or T <= 64)])
        return dict(op="norm", bwd=op == "norm_bwd", form=rng.choice(["both", "both", "pre", "post"]), R=R, T=T, H=H,
                    dtype=dtype, post=rng.random() < 0.7, gate=gate, G=G, res=rng.random() < 0.5)
    if op.startswith("balance"):
        E = rng.choice([rng.randint(1, 64), _log(rng, 2, 1024), 8, 64, 256])
        k = min(E, rng.choice([1, 2, 2, 4, 6, 8]))
        T = _log(rng, 1, min(131072, (1 << 25) // E))
        S = rng.choice([1, 1, 2, 7, 16, 64])
        T = max(S, T // S * S)
        return dict(op="balance", bwd=op == "balance_bwd", T=T, E=E, k=k, S=S, mask=rng.random() < 0.5)
    group = rng.choice([32, 64, 128])
    if op == "w4":
        K = 8 * _log(rng, 32, 3584)
        N = 8 * _log(rng, 8, max(8, min(3584, 8192 * 28672 // K // 8)))
        return dict(op="w4", M=rng.choice([1, 1, 2, 4, 8, rng.randint(1, 16), rng.randint(9, 16)]), N=N, K=K,
                    group=group, dtype=dtype)
    E = rng.choice([4, 8, 16, 40, 64])
    k = min(E, rng.choice([1, 2, 2, 4, 6]))
    K = 8 * _log(rng, 32, 1792)
    N = 8 * _log(rng, 8, max(8, min(1792, (1 << 28) // (K * E) // 8)))
    return dict(op=op, T=_log(rng, 1, 32), N=N, K=K, E=E, k=k, group=group, dtype=dtype)


# ------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op == "norm":
        T, H = case["T"], case["H"]
        both, pre = case["form"] == "both", case["form"] == "pre"
        gate = {"none": 0, "channel": case["G"] * H, "token": T}[case["gate"]] if not pre else 0
        if case["bwd"]:
            # x, y, both gradients in, dx and dy out (a form without y or without u lacks its share)
            big = {"both": 6, "pre": 4, "post": 5}[case["form"]]
            small = 2 * gate + 4 * gate + (6 + 6) * H
            return {"bytes": big * T * H * 2 + small + 8 * T, "flops": (24 if both else 12) * T * H}
        big = {"both": 4, "pre": 2, "post": 3}[case["form"]]
        return {"bytes": big * T * H * 2 + 2 * gate + 4 * H + 8 * T, "flops": (12 if both else 6) * T * H}
    if op == "balance":
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        mask = T if case["mask"] else 0
        if case["bwd"]:
            return {"bytes": 8 * T * E + T * k * 12 + 4 * T + mask + 4 * S * E, "flops": 7 * T * E}
        return {"bytes": 4 * T * E + 4 * T * k + 4 * T + mask + 8 * S * E, "flops": 5 * T * E}
    N, K, group = case["N"], case["K"], case["group"]
    weights = N * K // 2 + 2 * N * -(-K // group)
    if op == "w4":
        return {"bytes": weights + 2 * case["M"] * (N + K), "flops": 2 * case["M"] * N * K}
    E, T, k = case["E"], case["T"], case["k"]
    # each expert that some token chose is read once (k of E uniformly for each token)
    active = E * (1 - (1 - k / E) ** T)
    rows = 2 * T * K + 2 * T * k * N if op == "moe0" else 2 * T * k * K + 2 * T * N + 4 * T * k
    return {"bytes": int(active * weights) + rows + 4 * T * k, "flops": 2 * T * k * N * K}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std, dtype, mean=0.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=F32) * std + mean).to(dtype)


def _empty(shape, dtype=F32):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _shards(g, R, T, H, std, dtype):
    return [_normal(g, (T // R, H), std, dtype) for _ in range(R)]


def _pack(codes):
    """uint8 codes [.., N, 128 B] in the library's order: in every run of 128 inputs, 16 bytes for
    each c of 0..3, in them a 32-bit word for each j of 0..3, whose nibbles i and i + 4 are the
    inputs 32 j + 8 c + 2 i and the next one."""
    lead = codes.shape[:-1]
    d = codes.reshape(-1, 4, 4, 2, 2, 2)  # [block, j, c, half, pair, odd]: input 32 j + 8 c + 4 half + 2 pair + odd
    d = d.permute(0, 2, 1, 5, 3, 4)       # [block, c, j, odd, half, pair]
    return (d[..., 0] | (d[..., 1] << 4)).contiguous().reshape(*lead, -1)


def _unpack(q):
    lead = q.shape[:-1]
    d = torch.stack([q & 15, q >> 4], dim=-1).reshape(-1, 4, 4, 2, 2, 2)  # [block, c, j, odd, half, pair]
    return d.permute(0, 2, 1, 4, 5, 3).reshape(*lead, -1)


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = {"case": case, "ws": torch.zeros(WORKSPACE_BYTES // 4, dtype=torch.int32, device="cuda")}
    if op == "norm":
        dt, R, T, H = _dtype(case), case["R"], case["T"], case["H"]
        n = case["form"]
        s["x"] = _shards(g, R, T, H, 2.0, dt)
        s["w_pre"] = None if n == "post" else _normal(g, (H,), 0.2, dt, 1.0)
        s["y"] = s["w_post"] = s["gate"] = s["res"] = None
        if n != "pre":
            s["y"] = _shards(g, R, T, H, 0.7, dt)
            s["w_post"] = _normal(g, (H,), 0.2, dt, 1.0) if case["post"] else None
            if case["gate"] != "none":
                cols = H if case["gate"] == "channel" else 1
                s["gate"] = _normal(g, (case["G"], cols), 0.2, dt, 0.6)
            if case["res"]:
                s["res"] = _normal(g, (1,), 0.05, F32, 0.9)
        if not case["bwd"]:
            s["x_out"] = None if n == "pre" else [_empty((T // R, H), dt) for _ in range(R)]
            s["u_out"] = None if n == "post" else [_empty((T // R, H), dt) for _ in range(R)]
            s["rstd_y"] = _empty(T) if n != "pre" and case["post"] else None
            s["rstd_x"] = _empty(T) if n != "post" else None
            return s
        s["dx_out"] = _shards(g, R, T, H, 0.01, dt)
        s["du"] = None if n == "post" else _shards(g, R, T, H, 0.01, dt)
        # the statistics that the forward pass kept
        _, x1, ry, rx = _norm_forward(s, F64)
        s["rstd_y"] = None if ry is None else ry.to(F32).reshape(-1)
        s["rstd_x"] = None if rx is None else rx.to(F32).reshape(-1)
        del x1
        s["dx"] = [_empty((T // R, H), dt) for _ in range(R)]
        s["dy"] = None if n == "pre" else [_empty((T // R, H), dt) for _ in range(R)]
        s["dw_post"] = None if s["w_post"] is None else _empty(H)
        s["dgate"] = None if s["gate"] is None else _empty(s["gate"].shape)
        s["dres"] = None if s["res"] is None else _empty(1)
        s["dw_pre"] = None if n == "post" else _empty(H)
        return s
    if op == "balance":
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        p = torch.arange(1, E + 1, device="cuda", dtype=F32) ** -1.2
        s["logits"] = torch.randn((T, E), generator=g, device="cuda") + (p / p.sum()).log()
        top, ids = torch.topk(s["logits"], k, dim=1)
        s["ids"] = ids.to(torch.int32).contiguous()
        s["weights"] = (top - top[:, :1]).exp()
        s["weights"] = (s["weights"] / s["weights"].sum(1, keepdim=True)).contiguous()
        s["mask"] = None
        if case["mask"]:  # padding at the end of every sequence, up to a quarter of it
            length = T // S - (torch.rand(S, generator=g, device="cuda") * (T // S) * 0.25).long()
            s["mask"] = (torch.arange(T // S, device="cuda")[None, :] < length[:, None]).to(torch.uint8).reshape(-1).contiguous()
        s["loss"], s["counts"], s["probs"] = _empty(2), _empty((S, E), torch.int32), _empty((S, E))
        s["tokens"], s["lse"] = _empty(S + 1, torch.int32), _empty(T)
        if case["bwd"]:
            _, counts, _, tokens, lse = _balance_forward(s, F64)
            s["counts"], s["tokens"], s["lse"] = counts, tokens, lse.to(F32)
            s["dloss"] = torch.tensor([1.0, 0.5], device="cuda")
            s["dweights"] = _normal(g, (T, k), 0.1 / T, F32)
            s["dlogits"] = _empty((T, E))
        return s
    N, K, group, dt, E = case["N"], case["K"], case["group"], _dtype(case), case.get("E", 1)
    pad, lead = -(-K // 128) * 128, (E,) if op != "w4" else ()
    codes = _empty((*lead, N, pad)).normal_(generator=g).mul_(2.6).round_().add_(8).clamp_(0, 15).to(torch.uint8)
    s["q"] = _pack(codes)
    del codes
    std = 2.7 / 7 / math.sqrt(K)
    s["scales"] = (torch.rand((*lead, -(-K // group), N), generator=g, device="cuda") * 0.6 * std + 0.7 * std).to(dt)
    if op == "w4":
        s["x"], s["out"] = _normal(g, (case["M"], K), 1.0, dt), _empty((case["M"], N), dt)
        return s
    T, k = case["T"], case["k"]
    s["ids"] = torch.rand((T, E), generator=g, device="cuda").argsort(dim=1)[:, :k].to(torch.int32).contiguous()
    s["weights"] = torch.rand((T, k), generator=g, device="cuda") + 0.1
    s["weights"] = (s["weights"] / s["weights"].sum(1, keepdim=True)).contiguous()
    rows_in, rows_out = (T, T * k) if op == "moe0" else (T * k, T)
    s["x"], s["out"] = _normal(g, (rows_in, K), 1.0, dt), _empty((rows_out, N), dt)
    return s


# ------------------------------------------------------------------ one pass
BALANCE, ZLOSS = 0.01, 0.001


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import reducescatter_tcgen05_tmem_gb300 as fx
    c = s["case"]
    if c["op"] == "norm":
        cols = 0 if s["gate"] is None else s["gate"].shape[1]
        if c["bwd"]:
            fx.flux_block_norm_bwd(c["R"], c["T"], c["H"], _code(c), c["post"], c["G"], cols, s["x"], s["y"], s["w_post"],
                                   s["gate"], s["res"], s["w_pre"], s["rstd_y"], s["rstd_x"], s["dx_out"], s["du"],
                                   s["dx"], s["dy"], s["dw_post"], s["dgate"], s["dres"], s["dw_pre"], s["ws"])
            return {n: s[n] for n in ("dx", "dy", "dw_post", "dgate", "dres", "dw_pre")}
        fx.flux_block_norm(c["R"], c["T"], c["H"], _code(c), c["post"], c["G"], cols, EPS, s["x"], s["y"], s["w_post"],
                           s["gate"], s["res"], s["w_pre"], s["x_out"], s["u_out"], s["rstd_y"], s["rstd_x"])
        return {n: s[n] for n in ("x_out", "u_out", "rstd_y", "rstd_x")}
    if c["op"] == "balance":
        if c["bwd"]:
            fx.flux_moe_router_bwd(c["T"], c["E"], c["k"], c["S"], BALANCE, ZLOSS, s["logits"], s["ids"], s["weights"],
                                   s["mask"], s["lse"], s["counts"], s["tokens"], s["dloss"], s["dweights"], s["dlogits"])
            return s["dlogits"]
        fx.flux_moe_balance_loss(c["T"], c["E"], c["k"], c["S"], BALANCE, ZLOSS, s["logits"], s["ids"], s["mask"],
                                 s["loss"], s["counts"], s["probs"], s["tokens"], s["lse"], s["ws"])
        return {n: s[n] for n in ("loss", "counts", "probs", "tokens", "lse")}
    if c["op"] == "w4":
        fx.flux_w4_gemv(c["M"], c["N"], c["K"], c["group"], _code(c), s["x"], s["q"], s["scales"], s["out"], s["ws"])
    elif c["op"] == "moe0":
        fx.flux_moe_w4_layer0(c["T"], c["K"], c["N"], c["E"], c["k"], c["group"], _code(c), s["x"], s["q"], s["scales"],
                              s["ids"], s["out"], s["ws"])
    else:
        fx.flux_moe_w4_layer1(c["T"], c["N"], c["K"], c["E"], c["k"], c["group"], _code(c), s["x"], s["q"], s["scales"],
                              s["ids"], s["weights"], s["out"], s["ws"])
    return s["out"]


def _norm_forward(s, f):
    """(u, x', 1 / rms of y, 1 / rms of x') in the type f; None for what the form lacks."""
    c = s["case"]
    x1, ry, rx, u = torch.cat(s["x"]).to(f), None, None, None
    if s["y"] is not None:
        z = torch.cat(s["y"]).to(f)
        if c["post"]:
            ry = (z.square().mean(1, keepdim=True) + EPS).rsqrt()
            z = z * ry * s["w_post"].to(f)
        if s["gate"] is not None:
            z = z * s["gate"].to(f).repeat_interleave(c["T"] // c["G"], dim=0)
        x1 = (x1 if s["res"] is None else x1 * s["res"].to(f)) + z
    if s["w_pre"] is not None:
        rx = (x1.square().mean(1, keepdim=True) + EPS).rsqrt()
        u = x1 * rx * s["w_pre"].to(f)
    return u, x1, ry, rx


def _plain_norm(s):
    c = s["case"]
    dt, R, T, G = _dtype(c), c["R"], c["T"], c["G"]
    if not c["bwd"]:
        u, x1, ry, rx = _norm_forward(s, F32)
        return {"x_out": None if s["y"] is None else list(x1.to(dt).chunk(R)), "u_out": None if u is None else list(u.to(dt).chunk(R)),
                "rstd_y": None if ry is None else ry.reshape(-1), "rstd_x": None if rx is None else rx.reshape(-1)}
    x, d = torch.cat(s["x"]).float(), torch.cat(s["dx_out"]).float()
    out = dict.fromkeys(("dx", "dy", "dw_post", "dgate", "dres", "dw_pre"))
    z = yn = gate = None
    x1 = x
    if s["y"] is not None:
        z = torch.cat(s["y"]).float()
        if c["post"]:
            yn = z * s["rstd_y"][:, None]
            z = yn * s["w_post"].float()
        gate = None if s["gate"] is None else s["gate"].float().repeat_interleave(T // G, dim=0)
        x1 = (x if s["res"] is None else x * s["res"]) + (z if gate is None else z * gate)
    if s["du"] is not None:
        du, xn = torch.cat(s["du"]).float(), x1 * s["rstd_x"][:, None]
        out["dw_pre"] = (du * xn).sum(0)
        du = du * s["w_pre"].float()
        d = d + s["rstd_x"][:, None] * (du - xn * (du * xn).mean(1, keepdim=True))
    if s["y"] is not None:
        if s["res"] is not None:
            out["dres"] = (d * x).sum().reshape(1)
        if gate is not None:
            dg = (d * z).sum(1, keepdim=True) if s["gate"].shape[1] == 1 else d * z
            out["dgate"] = dg.reshape(G, T // G, -1).sum(1)
        dz = d if gate is None else d * gate
        if c["post"]:
            out["dw_post"] = (dz * yn).sum(0)
            dz = dz * s["w_post"].float()
            dz = s["rstd_y"][:, None] * (dz - yn * (dz * yn).mean(1, keepdim=True))
        out["dy"] = list(dz.to(dt).chunk(R))
        d = d if s["res"] is None else d * s["res"]
    out["dx"] = list(d.to(dt).chunk(R))
    return out


def _balance_forward(s, f):
    c = s["case"]
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    z = s["logits"].to(f)
    top = z.max(1, keepdim=True).values
    e = (z - top).exp()
    total = e.sum(1, keepdim=True)
    lse, p = (top + total.log()).reshape(-1), e / total
    m = torch.ones(T, dtype=torch.int32, device=z.device) if s["mask"] is None else (s["mask"] != 0).to(torch.int32)
    tokens = m.reshape(S, T // S).sum(1)
    at = torch.arange(T, device=z.device)[:, None] // (T // S) * E + s["ids"]
    counts = torch.zeros(S * E, dtype=torch.int32, device=z.device)
    counts = counts.index_add_(0, at.reshape(-1), m.repeat_interleave(k)).reshape(S, E)
    n = tokens.to(f)[:, None].clamp(min=1)
    probs = (p * m[:, None].to(f)).reshape(S, T // S, E).sum(1) / n
    balance = BALANCE * (E / (k * S)) * (counts.to(f) / n * probs).sum()
    zloss = ZLOSS * (lse.square() * m.to(f)).sum() / tokens.sum().clamp(min=1).to(f)
    tokens = torch.cat([tokens, tokens.sum().reshape(1)]).to(torch.int32)
    return torch.stack([balance, zloss]), counts, probs, tokens, lse


def _plain_balance(s):
    c = s["case"]
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    if not c["bwd"]:
        loss, counts, probs, tokens, lse = _balance_forward(s, F32)
        return {"loss": loss, "counts": counts, "probs": probs, "tokens": tokens, "lse": lse}
    p = (s["logits"] - s["lse"][:, None]).exp()
    n = s["tokens"][:S].float().clamp(min=1)[:, None]
    a = s["dloss"][0] * (BALANCE * E / (S * k)) * s["counts"].float() / (n * n)
    a = a.repeat_interleave(T // S, dim=0)
    z = s["dloss"][1] * (2 * ZLOSS) * s["lse"] / s["tokens"][S].clamp(min=1)
    d = p * (a - (p * a).sum(1, keepdim=True) + z[:, None])
    if s["mask"] is not None:
        d = d * (s["mask"] != 0).float()[:, None]
    w, dw = s["weights"], s["dweights"]
    return d.scatter_add(1, s["ids"].long(), w * (dw - (w * dw).sum(1, keepdim=True)))


def _weights(s, f):
    """The weights [.., N, K] that the codes and scales stand for."""
    c = s["case"]
    scale = s["scales"].to(f).transpose(-1, -2).repeat_interleave(c["group"], dim=-1)[..., :c["K"]]
    return (_unpack(s["q"])[..., :c["K"]].to(f) - 8) * scale


def _plain_w4(s):
    c = s["case"]
    x, w = s["x"].float(), _weights(s, F32)
    if c["op"] == "w4":
        return torch.matmul(x, w.T).to(_dtype(c))
    every = torch.matmul(x, w.transpose(1, 2))  # [E, rows, N]
    ids, T, k = s["ids"].long(), c["T"], c["k"]
    rows = torch.arange(T * k, device=x.device).reshape(T, k)
    if c["op"] == "moe0":
        return every[ids, rows // k].reshape(T * k, -1).to(_dtype(c))
    return (every[ids, rows] * s["weights"][:, :, None]).sum(1).to(_dtype(c))


def _run_plain(s):
    return {"norm": _plain_norm, "balance": _plain_balance}.get(s["case"]["op"], _plain_w4)(s)


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op, D = case["op"], F64
    if op == "norm":
        return _exact_norm(case, s)
    if op == "balance":
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        z = s["logits"].to(D)
        lse = torch.logsumexp(z, 1)
        p = torch.softmax(z, 1)
        keep = torch.ones(T, dtype=D, device="cuda") if s["mask"] is None else (s["mask"] > 0).to(D)
        hot = torch.zeros((T, E), dtype=D, device="cuda").scatter_(1, s["ids"].long(), 1.0) * keep[:, None]
        n = keep.view(S, -1).sum(1).clamp(min=1)
        f = hot.view(S, -1, E).sum(1) * (E / k) / n[:, None]
        if not case["bwd"]:
            P = (p * keep[:, None]).view(S, -1, E).sum(1) / n[:, None]
            loss = torch.stack([BALANCE * (f * P).sum() / S, ZLOSS * (lse * lse * keep).sum() / keep.sum().clamp(min=1)])
            return {"loss": loss, "counts": None, "probs": P, "tokens": None, "lse": lse}
        # d(sum_e f_e P_e)/dz and d(lse^2)/dz, the statistics as the call gets them
        g0, g1 = (float(v) for v in s["dloss"])
        f = (f * (g0 * BALANCE / S) / n[:, None]).repeat_interleave(T // S, 0)
        d = p * f - p * (p * f).sum(1, keepdim=True) + p * (2 * ZLOSS * g1 * lse / keep.sum().clamp(min=1))[:, None]
        d *= keep[:, None]
        w, dw = s["weights"].to(D), s["dweights"].to(D)
        gate = w * dw - w * (w * dw).sum(1, keepdim=True)
        return d.scatter_add_(1, s["ids"].long(), gate)
    N, K, group = case["N"], case["K"], case["group"]
    # input by input: which nibble of which byte holds it
    i = torch.arange(K, device="cuda")
    r = i % 128
    nibble = (r % 8) // 2 + 4 * (r % 2)
    byte = i // 128 * 64 + (r % 32) // 8 * 16 + r // 32 * 4 + nibble // 2
    shift = (nibble % 2 * 4).to(torch.uint8)

    def of(e):
        q, sc = (s["q"], s["scales"]) if e is None else (s["q"][e], s["scales"][e])
        code = (q.index_select(1, byte) >> shift) & 15
        return (code.to(D) - 8.0).T * sc.to(D).index_select(0, i // group)  # [K, N]

    x = s["x"].to(D)
    if op == "w4":
        return x @ of(None)
    T, k = case["T"], case["k"]
    slots = torch.zeros((T * k, N), dtype=D, device="cuda")
    flat = s["ids"].reshape(-1).long()
    for e in range(case["E"]):
        at = (flat == e).nonzero().reshape(-1)
        if at.numel():
            slots[at] = x[at // k if op == "moe0" else at] @ of(e)
    if op == "moe0":
        return slots
    return torch.einsum("tk,tkn->tn", s["weights"].to(D), slots.view(T, k, N))


def _exact_norm(case, s):
    D, R, T, H, G = F64, case["R"], case["T"], case["H"], case["G"]
    x = torch.cat([v.to(D) for v in s["x"]])
    has_y, has_u = s["y"] is not None, s["w_pre"] is not None
    per = T // G
    rho = 1.0 if s["res"] is None else float(s["res"])
    gate = 1.0 if s["gate"] is None else s["gate"].to(D)[:, None, :].expand(G, per, -1).reshape(T, -1)
    z, ry = 0.0, None
    if has_y:
        y = torch.cat([v.to(D) for v in s["y"]])
        z = y
        if case["post"]:
            ry = 1 / torch.sqrt((y * y).sum(1) / H + EPS) if not case["bwd"] else s["rstd_y"].to(D)
            z = y * ry[:, None] * s["w_post"].to(D)[None]
    xo = rho * x + gate * z if has_y else x
    rx = None
    if has_u:
        rx = 1 / torch.sqrt((xo * xo).sum(1) / H + EPS) if not case["bwd"] else s["rstd_x"].to(D)
    if not case["bwd"]:
        return {"x_out": list(torch.split(xo, T // R)) if has_y else None,
                "u_out": list(torch.split(xo * rx[:, None] * s["w_pre"].to(D), T // R)) if has_u else None,
                "rstd_y": ry, "rstd_x": rx}
    got = {"dx": None, "dy": None, "dw_post": None, "dgate": None, "dres": None, "dw_pre": None}
    dxo = torch.cat([v.to(D) for v in s["dx_out"]])
    if has_u:
        du = torch.cat([v.to(D) for v in s["du"]])
        got["dw_pre"] = (du * xo * rx[:, None]).sum(0)
        g = du * s["w_pre"].to(D)
        # u = w x' r(x'):  d r / d x' = -r^3 x' / H
        dxo = dxo + g * rx[:, None] - xo * (rx ** 3 * (g * xo).sum(1) / H)[:, None]
    if has_y:
        if s["res"] is not None:
            got["dres"] = (dxo * x).sum(1).sum().view(1)
        if s["gate"] is not None:
            t = dxo * z
            got["dgate"] = (t.sum(1, keepdim=True) if s["gate"].shape[1] == 1 else t).view(G, per, -1).sum(1)
        dz = dxo * gate
        if case["post"]:
            got["dw_post"] = (dz * y * ry[:, None]).sum(0)
            g = dz * s["w_post"].to(D)
            dz = g * ry[:, None] - y * (ry ** 3 * (g * y).sum(1) / H)[:, None]
        got["dy"] = list(torch.split(dz, T // R))
    got["dx"] = list(torch.split(rho * dxo, T // R))
    return got
