"""The block-norm, router and 4-bit kernels at lengths where a team of warps comes
round several times: buffers and places are used again, sums run over many rows of
one thread, and shards, sequences and gate rows end inside a team's stretch.
Compared with plain implementations in float64 on the same GPU."""
import pytest

from tests.rounding import U16, U32

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import reducescatter_tcgen05_tmem_gb300 as fx  # noqa: E402

F64 = torch.float64
DT = {"f16": (fx.FLUX_F16, torch.float16), "bf16": (fx.FLUX_BF16, torch.bfloat16)}
EPS = 1e-5


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ws(nbytes):
    return torch.zeros(max(nbytes, 256) // 4, dtype=torch.int32, device="cuda")


def _close(got, ref, mag, unit, depth, what, floor=0.0):
    """As tests/rounding.py: the output's rounding, and depth fp32 roundings of the terms' magnitudes."""
    before = depth * U32 * mag
    bound = unit * (ref.abs() + before) + before + floor
    off = (got.to(F64) - ref).abs() - bound
    assert not bool(off.isnan().any()), f"{what}: NaN"
    assert bool((off <= 0).all()), f"{what}: {int((off > 0).sum())} of {off.numel()} off, worst by {float(off.max()):.3e}"


def _near16(got, ref, mag, dtype, what, depth=128):
    _close(got, ref, mag, U16[dtype], depth, what, 2.0 ** -25 if dtype == "f16" else 0.0)


def _near32(got, ref, mag, what, depth):
    _close(got, ref, mag, U32, depth, what, 1e-45)


# ------------------------------------------------------------------ block norms
# rows of a team (2 DEPTH + 1 at least in the backward pass), by 152 SMs: T / (CTAs an
# SM x 152 x teams of a CTA); R and the gate's rows cut the stretches anywhere
NORMS = [
    # R, T, H, dtype, form, post, gate rows x columns, res
    (7, 49987, 64, "bf16", "both", True, None, True),          # one warp
    (3, 30003, 256, "f16", "both", True, (73, 256), True),
    (1, 20011, 512, "bf16", "both", True, (1, 512), True),     # two warps of one vector
    (2, 20014, 520, "f16", "both", True, (20014, 1), False),
    (5, 11005, 1024, "bf16", "both", True, (31, 1024), True),
    (1, 8191, 1280, "bf16", "both", True, (1, 1), True),       # three warps
    (4, 8004, 1536, "f16", "pre", True, None, False),
    (3, 8001, 2048, "bf16", "both", False, (9, 1), True),      # four
    (1, 7001, 2056, "bf16", "post", True, (7001, 2056), True),  # six; a gate for every row
    (2, 6998, 3064, "f16", "both", True, (2, 3064), True),
    (1, 4061, 4096, "bf16", "both", True, (31, 4096), False),  # eight
    (1, 2999, 4104, "f16", "both", True, (1, 4104), True),     # twelve
    (2, 3002, 6144, "bf16", "pre", True, None, False),
    (1, 2503, 6152, "bf16", "both", True, (1, 6152), True),    # sixteen
    (4, 2500, 8192, "f16", "both", True, (25, 8192), True),
    (3, 1503, 8200, "bf16", "both", True, (3, 8200), True),    # three vectors
    (1, 1500, 12288, "f16", "both", True, (60, 12288), True),
    (5, 1500, 12296, "bf16", "both", True, (500, 1), True),    # four vectors
    (1, 1201, 16384, "bf16", "both", True, (1, 16384), True),
    (2, 1202, 16376, "f16", "post", False, (2, 16376), True),
]


@pytest.mark.parametrize("case", NORMS, ids=lambda c: "-".join(str(v) for v in c).replace(" ", ""))
def test_block_norm_of_many_rows(case):
    R, T, H, dtype, form, post, gate, res = case
    code, dt = DT[dtype]
    g = _gen(T + H)
    draw = lambda shape, std, mean=0.0: (torch.randn(shape, device="cuda", generator=g) * std + mean).to(dt)  # noqa: E731
    has_y, has_u = form != "pre", form != "post"
    post = post and has_y
    x, dx1 = draw((T, H), 2.0), draw((T, H), 0.05)
    y = draw((T, H), 0.7) if has_y else None
    du, w_pre = (draw((T, H), 0.05), draw((H,), 1.0)) if has_u else (None, None)
    w_post = draw((H,), 1.0) if post else None
    gt = draw(gate, 1.0) if gate else None
    rho = torch.tensor([0.85], device="cuda") if has_y and res else None
    shards = lambda t: None if t is None else list(t.view(R, T // R, H))  # noqa: E731
    sizes = (R, T, H, code, int(post), *(gate or (0, 0)))

    # float64, with the magnitudes of the terms
    X, rho64 = x.to(F64), 1.0 if rho is None else float(rho)
    wp = 1.0 if w_pre is None else w_pre.to(F64)
    G = 1.0 if gt is None else gt.to(F64).repeat_interleave(T // gate[0], 0)
    x1, mag, ry = X, X.abs(), None
    if has_y:
        Y = y.to(F64)
        ry = (Y.square().mean(1, keepdim=True) + EPS).rsqrt() if post else None
        yn = Y * ry if post else Y
        wq = w_post.to(F64) if post else 1.0
        x1 = rho64 * X + G * (yn * wq)
        mag = (rho64 * X).abs() + (G * (yn * wq)).abs()
    rx = (x1.square().mean(1, keepdim=True) + EPS).rsqrt()

    new = lambda: torch.full((T, H), float("nan"), dtype=dt, device="cuda")  # noqa: E731
    xo, uo = new() if has_y else None, new() if has_u else None
    ry32 = torch.empty(T, device="cuda") if post else None
    rx32 = torch.empty(T, device="cuda") if has_u else None
    fx.flux_block_norm(*sizes, EPS, shards(x), shards(y), w_post, gt, rho, w_pre, shards(xo), shards(uo), ry32, rx32)
    if has_y:
        _near16(xo, x1, mag, dtype, "x'")
    if has_u:
        _near16(uo, x1 * rx * wp, (mag * rx * wp).abs(), dtype, "u")
        _near32(rx32, rx[:, 0], rx[:, 0], "rstd_x", 128)
    if post:
        _near32(ry32, ry[:, 0], ry[:, 0], "rstd_y", 128)
    del xo, uo

    e = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731
    dx, dy = new(), new() if has_y else None
    dwq, dg = e(H) if post else None, e(*gate) if gt is not None else None
    dr, dwp = e(1) if rho is not None else None, e(H) if has_u else None
    ws = _ws(fx.flux_block_norm_workspace_size(T, H, *(gate or (0, 0))))
    fx.flux_block_norm_bwd(*sizes, shards(x), shards(y), w_post, gt, rho, w_pre, ry32, rx32, shards(dx1), shards(du), shards(dx),
                           shards(dy), dwq, dg, dr, dwp, ws)
    assert not bool(ws.any()), "the workspace is not zero again"
    # rows of a thread, teams, CTAs (as the other tests of these sums), and the row's own arithmetic
    depth = 128 + 512
    d = dx1.to(F64)
    dmag = d.abs()
    if has_u:
        U = du.to(F64)
        xn, xnm = x1 * rx, mag * rx
        _near32(dwp, (U * xn).sum(0), (U.abs() * xnm).sum(0), "dw_pre", depth)
        U = U * wp
        d = d + rx * (U - xn * (U * xn).mean(1, keepdim=True))
        dmag = dmag + rx * (U.abs() + xnm * (U.abs() * xnm).mean(1, keepdim=True))
        del U, xn, xnm
    _near16(dx, rho64 * d, abs(rho64) * dmag, dtype, "dx")
    if not has_y:
        return
    if dr is not None:
        _near32(dr, (d * X).sum().view(1), (dmag * X.abs()).sum().view(1), "dres", depth)
    if gt is not None:
        rows = lambda t: (t.sum(1, keepdim=True) if gate[1] == 1 else t).view(gate[0], T // gate[0], -1).sum(1)  # noqa: E731
        z = yn * wq
        _near32(dg, rows(d * z), rows(dmag * z.abs()), "dgate", depth)
    dz, dzm = d * G, dmag * (G.abs() if gt is not None else 1.0)
    if post:
        _near32(dwq, (dz * yn).sum(0), (dzm * yn.abs()).sum(0), "dw_post", depth)
        c, cm = dz * wq, dzm * wq.abs()
        dz = ry * (c - yn * (c * yn).mean(1, keepdim=True))
        dzm = ry * (cm + yn.abs() * (cm * yn.abs()).mean(1, keepdim=True))
    _near16(dy, dz, dzm, dtype, "dy")
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ router
ROUTER = [
    # T, E, topk, S, mask: several groups of tokens a warp in both directions
    (250001, 3, 2, 1, True),
    (400000, 8, 2, 64, True),
    (300003, 16, 4, 3, False),
    (120000, 33, 5, 1, True),
    (130000, 64, 6, 26, True),
    (60060, 100, 8, 7, False),
    (50000, 128, 3, 1000, True),     # more sequences than CTAs
    (40002, 256, 8, 2, True),
    (20001, 300, 4, 1, True),
    (20000, 512, 9, 8, False),
    (15000, 1000, 16, 1, True),
    (16384, 1024, 40, 16, True),
]


def _softmax_choice(z, k):
    top, ids = z.topk(k, dim=1)
    w = torch.softmax(top.to(F64), 1).float()
    return ids.to(torch.int32).contiguous(), w.contiguous()


@pytest.mark.parametrize("case", ROUTER, ids=lambda c: "-".join(str(v) for v in c))
def test_router_of_many_tokens(case):
    T, E, k, S, masked = case
    a, b = 0.02, 0.003
    g = _gen(T)
    logits = torch.randn((T, E), device="cuda", generator=g) - 1.2 * torch.arange(1, E + 1, device="cuda").log()
    ids, w = _softmax_choice(logits, k)
    mask = (torch.rand(T, device="cuda", generator=g) < 0.7).to(torch.uint8) if masked else None
    keep = torch.ones(T, dtype=F64, device="cuda") if mask is None else mask.to(F64)
    e = lambda n, dt=torch.float32: torch.full((n,), 77, dtype=dt, device="cuda")  # noqa: E731
    loss, counts, probs, tokens, lse = e(2), e(S * E, torch.int32), e(S * E), e(S + 1, torch.int32), e(T)
    # the workspace of a larger batch, and one that the calls before have left dirty past its header
    size = max(fx.flux_moe_balance_workspace_size(n, E, k, S) for n in (T, T + 8 * S))
    ws = _ws(size)
    ws[64:] = 0x7F7F7F7F
    fx.flux_moe_balance_loss(T, E, k, S, a, b, logits, ids, mask, loss, counts, probs, tokens, lse, ws)
    assert not bool(ws[:64].any())

    z = logits.to(F64)
    L = torch.logsumexp(z, 1)
    p = torch.exp(z - L[:, None])
    n = keep.view(S, -1).sum(1)
    seq = torch.arange(T, device="cuda") // (T // S)
    c = torch.zeros(S * E, dtype=F64, device="cuda")
    c.index_add_(0, (seq[:, None] * E + ids).reshape(-1), keep[:, None].expand(T, k).reshape(-1))
    c = c.view(S, E)
    P = (p * keep[:, None]).view(S, T // S, E).sum(1) / n.clamp(min=1)[:, None]
    assert torch.equal(counts.view(S, E).to(F64), c)
    assert torch.equal(tokens[:S].to(F64), n) and int(tokens[S]) == int(n.sum())
    _near32(lse, L, L.abs() + 1.0, "lse", 128)
    # the exponent's argument, exp and the division, and the sum over the tokens of a thread, a CTA, a sequence
    depth = 160 + 512
    _near32(probs.view(S, E), P, 2 * P, "probs", depth)
    want = torch.stack([a * E / (k * S) * (c / n.clamp(min=1)[:, None] * P).sum(), b * (keep * L * L).sum() / n.sum()])
    _near32(loss, want, 2 * want.abs(), "loss", depth)

    for gate in (True, False):
        dw = torch.randn((T, k), device="cuda", generator=g) if gate else None
        dloss = torch.tensor([0.7, -1.3], device="cuda") if gate else None
        dl = torch.full((T, E), float("nan"), device="cuda")
        fx.flux_moe_router_bwd(T, E, k, S, a, b, logits, ids if gate else None, w if gate else None, mask, lse, counts, tokens,
                               dloss, dw, dl)
        d0, d1 = (0.7, -1.3) if gate else (1.0, 1.0)
        A = (d0 * a * E / (k * S) * c / n.clamp(min=1)[:, None].square())[seq]
        zt = (d1 * 2 * b * L / n.sum())[:, None]
        ref = p * (A - (p * A).sum(1, keepdim=True) + zt) * keep[:, None]
        mag = p * (A.abs() + (p * A.abs()).sum(1, keepdim=True) + zt.abs()) * keep[:, None]
        # |score - lse| and the lse itself are rounded before the exponential
        mag = mag * (1 + (z - L[:, None]).abs() / 64 + L[:, None].abs() / 64)
        if gate:
            w64, dw64 = w.to(F64), dw.to(F64)
            dot, dm = (w64 * dw64).sum(1, keepdim=True), (w64 * dw64).abs().sum(1, keepdim=True)
            ref.scatter_add_(1, ids.long(), w64 * (dw64 - dot))
            mag.scatter_add_(1, ids.long(), w64 * (dw64.abs() + dm))
        _near32(dl, ref, mag, f"dlogits, gate {gate}", 128)
        del A, ref, mag
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ 4-bit products
def _pack(codes):
    """[.., N, 128 B] codes in the order that the header gives."""
    i = torch.arange(128, device="cuda")
    j, c, r = i // 32, i % 32 // 8, i % 8
    nibble = r // 2 + 4 * (r % 2)
    byte = c * 16 + j * 4 + nibble // 2
    d = codes.view(*codes.shape[:-1], -1, 128)
    q = torch.zeros((*d.shape[:-1], 64), dtype=torch.uint8, device="cuda")
    for s in range(128):
        q[..., byte[s]] |= d[..., s] << (4 * (int(nibble[s]) % 2))
    return q.reshape(*codes.shape[:-1], -1)


PRODUCTS = [
    # rows, N, K, group, dtype: more runs of 128 inputs of one tile in a team's stretch than two of its buffers hold
    (1, 4096, 32768, 128, "bf16"),
    (8, 4096, 32768, 64, "f16"),
    (6, 4104, 30024, 32, "bf16"),
    (13, 2304, 32768, 128, "f16"),
    (16, 2312, 30000, 32, "bf16"),
    (32, 2048, 16384, 64, "bf16"),
    (40, 1024, 32768, 128, "f16"),
    (31, 2056, 16392, 32, "f16"),
]


def _weights(E, N, K, group, seed, dt):
    g = _gen(seed)
    codes = torch.randint(0, 16, (E, N, -(-K // 128) * 128), dtype=torch.uint8, device="cuda", generator=g)
    scales = (torch.rand((E, -(-K // group), N), device="cuda", generator=g) * 0.02 + 0.01).to(dt)
    q = _pack(codes)
    W = (codes[..., :K].to(F64) - 8) * scales.to(F64).transpose(1, 2).repeat_interleave(group, 2)[..., :K]
    return q, scales, W.transpose(1, 2)


def _depth(K, group, parts=40):
    # a tensor instruction adds 16 products to its sum with an error of at most 34 units
    # of the largest (17 terms cut, not rounded); then one rounding a group of the
    # tile's sum, the parts of cut tiles, the conversion
    return 34 * (group // 16) + -(-K // group) + parts


@pytest.mark.parametrize("case", PRODUCTS, ids=lambda c: "-".join(str(v) for v in c))
def test_long_product(case):
    M, N, K, group, dtype = case
    code, dt = DT[dtype]
    q, scales, W = _weights(1, N, K, group, K + M, dt)
    x = torch.randn((M, K), device="cuda", generator=_gen(M)).to(dt)
    out = torch.full((M, N), float("nan"), dtype=dt, device="cuda")
    ws = _ws(fx.flux_w4_workspace_size(M, N, K))
    fx.flux_w4_gemv(M, N, K, group, code, x, q, scales, out, ws)
    _near16(out, x.to(F64) @ W[0], x.to(F64).abs() @ W[0].abs(), dtype, "product", _depth(K, group))
    assert not bool(ws.any())


@pytest.mark.parametrize("case", PRODUCTS, ids=lambda c: "-".join(str(v) for v in c))
def test_long_product_of_whole_numbers_is_exact(case):
    # every partial sum is a whole number below 2^24, whatever the order
    M, N, K, group, dtype = case
    code, dt = DT[dtype]
    q, scales, W = _weights(1, N, K, group, K + M, dt)
    W = (W / scales.to(F64).repeat_interleave(group, 1)[:, :K]).round()
    x = torch.randint(-1, 2, (M, K), device="cuda", generator=_gen(M)).to(dt)
    x[:, K // 3:K // 2] = 0
    out = torch.empty((M, N), dtype=dt, device="cuda")
    fx.flux_w4_gemv(M, N, K, group, code, x, q, torch.ones_like(scales), out, _ws(fx.flux_w4_workspace_size(M, N, K)))
    assert torch.equal(out, (x.to(F64) @ W[0]).to(dt))


MOE = [
    # T, N, K, E, topk, group, dtype: experts of 8, 16 and 32 rows a tile, long tiles
    (4, 2048, 16384, 4, 2, 128, "bf16"),
    (16, 2048, 16392, 2, 1, 64, "f16"),
    (40, 1032, 16384, 3, 2, 32, "bf16"),
    (1, 4096, 14336, 16, 8, 128, "f16"),
]


@pytest.mark.parametrize("case", MOE, ids=lambda c: "-".join(str(v) for v in c))
def test_long_expert_products(case):
    T, N, K, E, k, group, dtype = case
    code, dt = DT[dtype]
    q, scales, W = _weights(E, N, K, group, K + T, dt)
    g = _gen(T)
    ids = torch.rand((T, E), device="cuda", generator=g).argsort(1)[:, :k].to(torch.int32).contiguous()
    gw = torch.rand((T, k), device="cuda", generator=g)
    x, h = (torch.randn((n, K), device="cuda", generator=g).to(dt) for n in (T, T * k))
    ws = _ws(fx.flux_w4_workspace_size(T * k, N, K, E))
    rows, out = torch.full((T * k, N), float("nan"), dtype=dt, device="cuda"), torch.full((T, N), float("nan"), dtype=dt, device="cuda")
    fx.flux_moe_w4_layer0(T, K, N, E, k, group, code, x, q, scales, ids, rows, ws)
    fx.flux_moe_w4_layer1(T, N, K, E, k, group, code, h, q, scales, ids, gw, out, ws)
    ref = torch.zeros((2, T * k, N), dtype=F64, device="cuda")
    mag = torch.zeros_like(ref)
    flat = ids.reshape(-1).long()
    xs = x.to(F64).repeat_interleave(k, 0), h.to(F64)
    for e in range(E):
        at = (flat == e).nonzero().reshape(-1)
        for i in range(2):
            ref[i, at], mag[i, at] = xs[i][at] @ W[e], xs[i][at].abs() @ W[e].abs()
    _near16(rows, ref[0], mag[0], dtype, "layer0", _depth(K, group))
    wt = gw.to(F64)[:, :, None]
    _near16(out, (ref[1].view(T, k, N) * wt).sum(1), (mag[1].view(T, k, N) * wt).sum(1), dtype, "layer1", _depth(K, group) + k)
    assert not bool(ws.any())
