"""Three more families of operators beside those around an MoE block, as cases that can be timed and compared.

Each has the calls that a user makes of the package (``own`` true) and a plain
form of elementary torch operations (``own`` false):

* the edge of a block with layer norm and dropout (``flux_layer_norm`` /
  ``flux_layer_norm_bwd``): the block's output is dropped out and added to the
  residual stream, and the sum is normalised for the next block.  The random
  bits come from a counter (Philox4x32-10 of the element's index), so the
  backward pass makes them again and no mask is stored;
* routing with groups (``flux_moe_group_gate`` / ``flux_moe_group_gate_bwd``):
  softmax or sigmoid scores, a bias that steers the choice alone, groups of
  experts, top-k, renormalised and scaled weights, and the scores' gradient;
* products in 8-bit integers (``flux_q8_quantize``, ``flux_q8_gemm``): tokens
  quantised row by row as they come, weights with a scale for each channel.

``listed`` holds the cases, ``draw`` makes more of the same ranges.
"""
import math

import torch

own = False

#: One zeroed workspace, as a program keeps it for all of these calls.
WORKSPACE_BYTES = 512 << 20

F16, BF16, F32, F64, I64 = torch.float16, torch.bfloat16, torch.float32, torch.float64, torch.int64
EPS = 1e-5
LOW32 = 0xFFFFFFFF


def _dtype(case):
    return {"f16": F16, "bf16": BF16}[case["dtype"]]


def _code(case):
    return {"f16": 0, "bf16": 1}[case["dtype"]]


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step of four requests between two blocks: residual and layer norm of H 4096
        dict(name="ln_step", op="ln", bwd=False, form="both", R=1, T=4, H=4096, dtype="bf16", p=0.0, affine=True),
        # the residual stream of a training step, sharded over 8 ranks by rows, a tenth dropped
        dict(name="ln_train", op="ln", bwd=False, form="both", R=8, T=32768, H=4096, dtype="bf16", p=0.1, affine=True),
        # its backward pass with the gradients of weight and bias
        dict(name="ln_train_bwd", op="ln", bwd=True, form="both", R=8, T=32768, H=4096, dtype="bf16", p=0.1, affine=True),
        # the first norm of a wide model in fp16, no block before it, an odd row count
        dict(name="ln_wide_bwd", op="ln", bwd=True, form="pre", R=1, T=4061, H=12288, dtype="f16", p=0.0, affine=True),
        # 13 decoding requests choose 8 of 256 experts in 4 of 8 groups
        dict(name="gate_decode", op="gate", bwd=False, T=13, E=256, k=8, score="sigmoid", bias=True, groups=8, kept=4,
             top=2, renorm=True, scale=2.5),
        # the same router on a long training batch
        dict(name="gate_long", op="gate", bwd=False, T=131072, E=256, k=8, score="sigmoid", bias=True, groups=8, kept=4,
             top=2, renorm=True, scale=2.5),
        # softmax scores that are not renormalised, on a micro-batch: every score gets a gradient
        dict(name="gate_softmax_bwd", op="gate", bwd=True, T=4096, E=64, k=6, score="softmax", bias=False, groups=8, kept=3,
             top=1, renorm=False, scale=1.0),
        # the long batch's gradient: zeros but for the chosen experts
        dict(name="gate_long_bwd", op="gate", bwd=True, T=131072, E=256, k=8, score="sigmoid", bias=True, groups=8, kept=4,
             top=2, renorm=True, scale=2.5),
        # one token through an attention-sized projection: the launches and the tail count
        dict(name="q8_token", op="q8", M=1, N=4096, K=4096, dtype="bf16", bias=False),
        # 13 decoding requests through the 70B-class down-projection
        dict(name="q8_down_13", op="q8", M=13, N=8192, K=28672, dtype="f16", bias=False),
        # an odd chunk of a prompt through a down-projection with a bias
        dict(name="q8_chunk", op="q8", M=333, N=4096, K=14336, dtype="f16", bias=True),
        # a prompt of 4096 tokens through an up-projection
        dict(name="q8_prompt", op="q8", M=4096, N=14336, K=4096, dtype="bf16", bias=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["f16", "bf16"])
    op = rng.choice(["ln", "ln_bwd", "gate", "gate_bwd", "q8", "q8"])
    if op.startswith("ln"):
        H = 8 * _log(rng, 8, 2048)
        R = rng.choice([1, 1, 2, 4, 8])
        T = R * max(1, _log(rng, 1, max(1, min(32768, (1 << 27) // H))) // R)
        form = rng.choice(["both", "both", "pre", "sum"])
        p = 0.0 if form == "pre" else rng.choice([0.0, 0.1, 0.1, round(rng.uniform(0.01, 0.6), 3)])
        return dict(op="ln", bwd=op == "ln_bwd", form=form, R=R, T=T, H=H, dtype=dtype, p=p, affine=rng.random() < 0.8)
    if op.startswith("gate"):
        groups = rng.choice([1, 1, 2, 4, 8, 8, 16])
        E = groups * _log(rng, 2, 1024 // groups)
        kept = groups if groups == 1 else rng.randint(1, groups)
        k = min(kept * (E // groups), rng.choice([1, 2, 4, 6, 8, 8, rng.randint(1, 16)]))
        return dict(op="gate", bwd=op == "gate_bwd", T=_log(rng, 1, min(131072, (1 << 25) // E)), E=E, k=k,
                    score=rng.choice(["sigmoid", "softmax"]), bias=rng.random() < 0.6, groups=groups, kept=kept,
                    top=rng.choice([1, 2]), renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]))
    K = 16 * _log(rng, 16, 1792)
    N = 8 * _log(rng, 8, 3584)
    M = _log(rng, 1, max(1, min(8192, 4096 * 14336 * 4096 // (N * K))))
    if rng.random() < 0.4:
        M = min(M, rng.randint(1, 48))
    return dict(op="q8", M=M, N=N, K=K, dtype=dtype, bias=rng.random() < 0.3)


# ------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op == "ln":
        T, H = case["T"], case["H"]
        w = 4 * H if case["affine"] and case["form"] != "sum" else 0
        if case["bwd"]:
            # x', du and the gradient of x' in, dx and dy out (a form lacks its share; dy is dx without dropout)
            big = {"both": 4 + (case["p"] > 0), "pre": 4, "sum": 1 + (case["p"] > 0)}[case["form"]]
            stats = 0 if case["form"] == "sum" else 8 * T
            return {"bytes": big * T * H * 2 + w + 2 * w + stats, "flops": 14 * T * H}
        big = {"both": 4, "pre": 2, "sum": 3}[case["form"]]
        return {"bytes": big * T * H * 2 + w + (0 if case["form"] == "sum" else 8 * T), "flops": 9 * T * H}
    if op == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        if case["bwd"]:
            every = case["score"] == "softmax" and not case["renorm"]  # the whole row takes part in the softmax
            return {"bytes": 4 * T * E + T * k * 8 + (4 * T * E if every else 4 * T * k), "flops": (8 * E if every else 10 * k) * T}
        return {"bytes": 4 * T * E + 8 * T * k + (4 * E if case["bias"] else 0), "flops": 6 * T * E}
    M, N, K = case["M"], case["N"], case["K"]
    return {"bytes": 2 * M * K + N * K + 4 * N + 2 * M * N + (2 * N if case["bias"] else 0), "flops": 2 * M * N * K}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std, dtype, mean=0.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=F32) * std + mean).to(dtype)


def _empty(shape, dtype=F32):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _shards(g, R, T, H, std, dtype, mean=0.0):
    return [_normal(g, (T // R, H), std, dtype, mean) for _ in range(R)]


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = {"case": case, "ws": torch.zeros(WORKSPACE_BYTES // 4, dtype=torch.int32, device="cuda")}
    if op == "ln":
        dt, R, T, H, form = _dtype(case), case["R"], case["T"], case["H"], case["form"]
        rows = lambda: [_empty((T // R, H), dt) for _ in range(R)]  # noqa: E731
        s["rng"] = torch.randint(0, 1 << 40, (2,), generator=g, device="cuda") if case["p"] > 0 else None
        s["w"] = _normal(g, (H,), 0.2, dt, 1.0) if case["affine"] and form != "sum" else None
        s["b"] = _normal(g, (H,), 0.1, dt) if case["affine"] and form != "sum" else None
        if not case["bwd"]:
            s["x"] = _shards(g, R, T, H, 2.0, dt, 0.1)
            s["y"] = None if form == "pre" else _shards(g, R, T, H, 0.7, dt)
            s["x_out"] = None if form == "pre" else rows()
            s["u_out"] = None if form == "sum" else rows()
            s["mean"], s["rstd"] = (None, None) if form == "sum" else (_empty(T), _empty(T))
            return s
        s["dx_out"] = _shards(g, R, T, H, 0.01, dt)
        s["dx"] = rows()
        s["dy"] = rows() if case["p"] > 0 else None
        s["x"] = s["du"] = s["mean"] = s["rstd"] = s["dw"] = s["db"] = None
        if form != "sum":  # x' as the forward pass wrote it, its statistics as it kept them
            s["x"] = _shards(g, R, T, H, 2.1, dt, 0.1)
            s["du"] = _shards(g, R, T, H, 0.01, dt)
            stats = [torch.var_mean(v.double(), dim=1, correction=0) for v in s["x"]]
            s["mean"] = torch.cat([m for _, m in stats]).float()
            s["rstd"] = torch.cat([(v + EPS).rsqrt() for v, _ in stats]).float()
            if case["affine"]:
                s["dw"], s["db"] = _empty(H), _empty(H)
        return s
    if op == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        tilt = torch.randn(E, generator=g, device="cuda") * 0.5  # some experts are liked better
        s["logits"] = torch.randn((T, E), generator=g, device="cuda") + tilt
        s["bias"] = -0.05 * tilt + 0.02 * torch.randn(E, generator=g, device="cuda") if case["bias"] else None
        s["ids"], s["weights"] = _empty((T, k), torch.int32), _empty((T, k))
        if case["bwd"]:
            s["ids"] = _plain_gate(s)["ids"]
            s["dweights"] = _normal(g, (T, k), 0.1, F32)
            s["dlogits"] = _empty((T, E))
        return s
    M, N, K, dt = case["M"], case["N"], case["K"], _dtype(case)
    s["x"] = _normal(g, (M, K), 1.0, F32)
    s["x"][:, torch.randint(0, K, (max(1, K // 512),), generator=g, device="cuda")] *= 8  # channels that stand out
    s["x"] = s["x"].to(dt)
    s["wq"] = _empty((N, K)).normal_(generator=g).mul_(34.0).round_().clamp_(-127, 127).to(torch.int8)
    s["wscale"] = (torch.rand(N, generator=g, device="cuda") * 0.6 + 0.7) * (1 / 34.0 / math.sqrt(K))
    s["b"] = _normal(g, (N,), 0.1, dt) if case["bias"] else None
    s["xq"], s["xscale"], s["out"] = _empty((M, K), torch.int8), _empty(M), _empty((M, N), dt)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _run_own(s) if own else {"ln": _plain_ln, "gate": _plain_gate_pass, "q8": _plain_q8}[s["case"]["op"]](s)


def _run_own(s):
    import reducescatter_tcgen05_tmem_gb300 as fx
    c = s["case"]
    if c["op"] == "ln":
        if c["bwd"]:
            fx.flux_layer_norm_bwd(c["R"], c["T"], c["H"], _code(c), c["p"], s["x"], s["rng"], s["w"], s["mean"], s["rstd"],
                                   s["dx_out"], s["du"], s["dx"], s["dy"], s["dw"], s["db"], s["ws"])
            return {n: s[n] for n in ("dx", "dy", "dw", "db")}
        fx.flux_layer_norm(c["R"], c["T"], c["H"], _code(c), c["p"], EPS, s["x"], s["y"], s["rng"], s["w"], s["b"],
                           s["x_out"], s["u_out"], s["mean"], s["rstd"])
        return {n: s[n] for n in ("x_out", "u_out", "mean", "rstd")}
    if c["op"] == "gate":
        score = {"softmax": fx.FLUX_SCORE_SOFTMAX, "sigmoid": fx.FLUX_SCORE_SIGMOID}[c["score"]]
        if c["bwd"]:
            fx.flux_moe_group_gate_bwd(c["T"], c["E"], c["k"], score, c["renorm"], c["scale"], s["logits"], s["ids"],
                                       s["dweights"], 0, s["dlogits"])
            return s["dlogits"]
        fx.flux_moe_group_gate(c["T"], c["E"], c["k"], score, c["groups"], c["kept"], c["top"], c["renorm"], c["scale"],
                               s["logits"], s["bias"], s["ids"], s["weights"])
        return {"ids": s["ids"], "weights": s["weights"]}
    fx.flux_q8_quantize(c["M"], c["K"], _code(c), s["x"], s["xq"], s["xscale"])
    fx.flux_q8_gemm(c["M"], c["N"], c["K"], _code(c), s["xq"], s["xscale"], s["wq"], s["wscale"], s["b"], s["out"], s["ws"])
    return s["out"]


def _keep_of(p):
    """Of 65536 draws, how many keep an element."""
    return int(round((1.0 - p) * 65536))


def _plain_mask(s):
    """Which elements stay, [T, H]: 16 of a counter's 128 bits for each of eight neighbours."""
    c = s["case"]
    seed, offset = s["rng"][0], s["rng"][1]
    block = torch.arange(c["T"] * c["H"] // 8, device="cuda", dtype=I64)
    a, b = block & LOW32, block >> 32
    d, e = (offset & LOW32).expand_as(a), ((offset >> 32) & LOW32).expand_as(a)
    k0, k1 = seed & LOW32, (seed >> 32) & LOW32
    for i in range(10):
        m0, m1 = a * 0xD2511F53, d * 0xCD9E8D57  # the low 64 bits: the sign does not matter to the masks
        a, b, d, e = ((m1 >> 32) & LOW32) ^ b ^ k0, m1 & LOW32, ((m0 >> 32) & LOW32) ^ e ^ k1, m0 & LOW32
        k0, k1 = (k0 + 0x9E3779B9) & LOW32, (k1 + 0xBB67AE85) & LOW32
    keep = _keep_of(c["p"])
    return torch.stack([v < keep for w in (a, b, d, e) for v in (w & 0xFFFF, w >> 16)], dim=1).reshape(c["T"], c["H"])


def _plain_ln(s):
    c = s["case"]
    dt, R = _dtype(c), c["R"]
    drop = c["p"] > 0
    if not c["bwd"]:
        x1 = torch.cat(s["x"]).float()
        out = dict.fromkeys(("x_out", "u_out", "mean", "rstd"))
        if s["y"] is not None:
            y = torch.cat(s["y"]).float()
            x1 = x1 + (torch.where(_plain_mask(s), y * (65536.0 / _keep_of(c["p"])), 0.0) if drop else y)
            out["x_out"] = list(x1.to(dt).chunk(R))
        if c["form"] != "sum":
            mean = x1.mean(1, keepdim=True)
            d = x1 - mean
            rstd = (d.square().mean(1, keepdim=True) + EPS).rsqrt()
            u = d * rstd
            if s["w"] is not None:
                u = u * s["w"].float() + s["b"].float()
            out["u_out"], out["mean"], out["rstd"] = list(u.to(dt).chunk(R)), mean.reshape(-1), rstd.reshape(-1)
        return out
    d = torch.cat(s["dx_out"]).float()
    out = dict.fromkeys(("dx", "dy", "dw", "db"))
    if c["form"] != "sum":
        xn = (torch.cat(s["x"]).float() - s["mean"][:, None]) * s["rstd"][:, None]
        du = torch.cat(s["du"]).float()
        if s["w"] is not None:
            out["dw"], out["db"] = (du * xn).sum(0), du.sum(0)
            du = du * s["w"].float()
        d = d + s["rstd"][:, None] * (du - du.mean(1, keepdim=True) - xn * (du * xn).mean(1, keepdim=True))
    out["dx"] = list(d.to(dt).chunk(R))
    if drop:
        out["dy"] = list(torch.where(_plain_mask(s), d * (65536.0 / _keep_of(c["p"])), 0.0).to(dt).chunk(R))
    return out


def _plain_gate(s):
    """The choice is made on 64-bit values: neighbours in rank are often closer than 32 bits tell apart."""
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    z = s["logits"].double()
    if c["score"] == "sigmoid":
        score = 1 / (1 + (-z).exp())
    else:
        e = (z - z.max(1, keepdim=True).values).exp()
        score = e / e.sum(1, keepdim=True)
    value = score if s["bias"] is None else score + s["bias"].double()
    order = z if s["bias"] is None else value  # the scores keep the logits' order
    if c["kept"] < G:
        if c["top"] == 1:
            rank = order.reshape(T, G, E // G).max(2).values
        else:
            rank = torch.sort(value.reshape(T, G, E // G), dim=2, descending=True).values[:, :, :2].sum(2)
        best = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :c["kept"]]
        allowed = torch.zeros((T, G), dtype=torch.bool, device=z.device).scatter_(1, best, True)
        order = order.masked_fill(~allowed.repeat_interleave(E // G, dim=1), -math.inf)
    ids = torch.sort(order, dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32).contiguous(), "weights": (w * c["scale"]).float()}


def _plain_gate_pass(s):
    c = s["case"]
    if not c["bwd"]:
        return _plain_gate(s)
    z, ids, g = s["logits"], s["ids"].long(), s["dweights"] * c["scale"]
    if c["score"] == "sigmoid":
        p = 1 / (1 + (-z.gather(1, ids)).exp())
        if c["renorm"]:
            w = p / p.sum(1, keepdim=True)
            d = w * (1 - p) * (g - (w * g).sum(1, keepdim=True))
        else:
            d = p * (1 - p) * g
        return torch.zeros_like(z).scatter_(1, ids, d)
    e = (z - z.max(1, keepdim=True).values).exp()
    if c["renorm"]:
        w = e.gather(1, ids)
        w = w / w.sum(1, keepdim=True)
        return torch.zeros_like(z).scatter_(1, ids, w * (g - (w * g).sum(1, keepdim=True)))
    p = e / e.sum(1, keepdim=True)
    full = torch.zeros_like(z).scatter_(1, ids, g)
    return p * (full - (p * full).sum(1, keepdim=True))


def _plain_q8(s):
    # scale and codes as they are defined: the scale in 32 bits, the quotient rounded from its
    # 64-bit value (in 32 bits some quotients fall on the border between two codes)
    x = s["x"].float()
    scale = x.abs().amax(1) / 127
    code = (x.double() / scale.double()[:, None]).round().float().nan_to_num()
    out = torch.matmul(code, s["wq"].float().T) * scale[:, None] * s["wscale"]
    if s["b"] is not None:
        out = out + s["b"].float()
    return out.to(_dtype(s["case"]))


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"ln": _exact_ln, "gate": _exact_gate, "q8": _exact_q8}[case["op"]](case, s)


def _mulhi(a, m):
    """High 32 bits of the product of 32-bit numbers, by halves of 16 bits."""
    a0, a1, m0, m1 = a & 0xFFFF, a >> 16, m & 0xFFFF, m >> 16
    mid = a1 * m0 + (a0 * m0 >> 16)
    return a1 * m1 + (mid >> 16) + ((mid & 0xFFFF) + a0 * m1 >> 16)


def _mullo(a, m):
    return ((a & 0xFFFF) * m + (((a >> 16) * (m & 0xFFFF) & 0xFFFF) << 16)) & LOW32


def _exact_factor(case, s):
    """0 or 1 / (share kept) for each element, from the generator's definition."""
    T, H = case["T"], case["H"]
    seed, offset = (int(v) for v in s["rng"].tolist())
    n = torch.arange(T * H // 8, device="cuda", dtype=I64)
    ctr = [n % (1 << 32), n // (1 << 32), torch.full_like(n, offset % (1 << 32)), torch.full_like(n, offset // (1 << 32))]
    key = [seed % (1 << 32), seed // (1 << 32)]
    for _ in range(10):
        ctr = [_mulhi(ctr[2], 0xCD9E8D57) ^ ctr[1] ^ key[0], _mullo(ctr[2], 0xCD9E8D57),
               _mulhi(ctr[0], 0xD2511F53) ^ ctr[3] ^ key[1], _mullo(ctr[0], 0xD2511F53)]
        key = [(key[0] + 0x9E3779B9) % (1 << 32), (key[1] + 0xBB67AE85) % (1 << 32)]
    keep = round((1.0 - case["p"]) * 65536)
    f = torch.empty((T * H // 8, 8), dtype=F64, device="cuda")
    for j in range(8):
        f[:, j] = ((ctr[j // 2] // (1 << 16 * (j % 2))) % 65536 < keep).to(F64) * (65536 / keep)
    return f.view(T, H)


def _exact_ln(case, s):
    D, T, H, R = F64, case["T"], case["H"], case["R"]
    split = lambda v: None if v is None else list(torch.split(v, T // R))  # noqa: E731
    factor = _exact_factor(case, s) if case["p"] > 0 else 1.0
    w = 1.0 if s["w"] is None else s["w"].to(D)
    if not case["bwd"]:
        x = torch.cat([v.to(D) for v in s["x"]])
        if s["y"] is not None:
            x = x + factor * torch.cat([v.to(D) for v in s["y"]])
        out = {"x_out": None if s["y"] is None else split(x), "u_out": None, "mean": None, "rstd": None}
        if case["form"] != "sum":
            m = x.sum(1) / H
            r = 1 / torch.sqrt(((x - m[:, None]) ** 2).sum(1) / H + EPS)
            u = (x - m[:, None]) * r[:, None] * w + (0.0 if s["b"] is None else s["b"].to(D))
            out.update(u_out=split(u), mean=m, rstd=r)
        return out
    d = torch.cat([v.to(D) for v in s["dx_out"]])
    out = {"dx": None, "dy": None, "dw": None, "db": None}
    if case["form"] != "sum":
        r, c = s["rstd"].to(D)[:, None], torch.cat([v.to(D) for v in s["x"]]) - s["mean"].to(D)[:, None]
        du = torch.cat([v.to(D) for v in s["du"]])
        if s["w"] is not None:
            out["dw"], out["db"] = torch.einsum("th,th,tk->h", du, c, r), du.sum(0)
        g = du * w
        # u = w c r + b with c = x - mean(x), r = (mean(c^2) + eps)^-1/2: dr = -r^3 mean(c dc)
        d = d + r * (g - g.sum(1, keepdim=True) / H) - r ** 3 * c * ((g * c).sum(1, keepdim=True) / H)
    out["dx"] = split(d)
    if case["p"] > 0:
        out["dy"] = split(d * factor)
    return out


def _exact_gate(case, s):
    D, T, E, k, G = F64, case["T"], case["E"], case["k"], case["groups"]
    z = s["logits"].to(D)
    soft = case["score"] == "softmax"
    score = torch.softmax(z, 1) if soft else torch.sigmoid(z)
    if case["bwd"]:
        ids, g = s["ids"].long(), s["dweights"].to(D) * case["scale"]
        hot = torch.zeros((T, E), dtype=D, device="cuda").scatter_(1, ids, 1.0)
        up = torch.zeros((T, E), dtype=D, device="cuda").scatter_(1, ids, g)
        if case["renorm"]:  # w = score / sum of the chosen scores
            total = (score * hot).sum(1, keepdim=True)
            up = (up / total - (up * score).sum(1, keepdim=True) / total ** 2) * hot
        if soft:
            return score * up - score * (score * up).sum(1, keepdim=True)
        return up * score * (1 - score)
    value = score + s["bias"].to(D) if case["bias"] else score
    order = (value if case["bias"] else z).clone()
    if case["kept"] < G:
        per = (order if case["top"] == 1 else value).view(T, G, E // G)
        rank = per.amax(2)
        if case["top"] == 2 and E // G > 1:
            rank = torch.topk(per, 2, dim=2).values.sum(2)
        allowed = torch.zeros((T, G), dtype=torch.bool, device="cuda")
        at = torch.arange(T, device="cuda")
        for _ in range(case["kept"]):
            left = rank.masked_fill(allowed, -math.inf)
            first = (left == left.amax(1, keepdim=True)).to(torch.int8).argmax(1)
            allowed[at, first] = True
        order[~allowed.repeat_interleave(E // G, 1)] = -math.inf
    ids = torch.empty((T, k), dtype=I64, device="cuda")
    number = torch.arange(E, device="cuda")
    for j in range(k):  # the largest left, the lowest number among equals
        best = order.amax(1, keepdim=True)
        ids[:, j] = torch.where(order == best, number, E).amin(1)
        order.scatter_(1, ids[:, j:j + 1], -math.inf)
    w = score.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": w * case["scale"]}


def _exact_q8(case, s):
    D = F64
    x = s["x"].to(D)
    scale = (x.abs().max(1).values.to(F32) / torch.tensor(127.0, device="cuda")).to(D)  # held in 32 bits
    q = torch.round(x / scale.view(-1, 1)).nan_to_num()
    out = torch.einsum("mk,nk->mn", q, s["wq"].to(D)) * torch.outer(scale, s["wscale"].to(D))
    return out if s["b"] is None else out + s["b"].to(D)
