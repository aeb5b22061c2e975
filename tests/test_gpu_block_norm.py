"""GPU parity of the norms around a block (flux_block_norm, flux_block_norm_bwd)
with their float64 definitions, through the C ABI."""
import numpy as np
import pytest

import oracle
from tests.rounding import U16, check16, check32
from workloads import gen
from workloads.torch_io import from_device, to_device, torch_dtype

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import reducescatter_tcgen05_tmem_gb300 as fx  # noqa: E402

DT = {"f16": fx.FLUX_F16, "bf16": fx.FLUX_BF16}
EPS = 1e-5
GUARD = 64  # elements either side of every output


def _ws(nbytes):
    n = max(nbytes, 256) // 4
    ws = torch.zeros(n + 64, dtype=torch.int32, device="cuda")
    off = (-ws.data_ptr()) % 256 // 4
    return ws[off:off + n]


class Out:
    """An output between guards that have to keep their value."""

    def __init__(self, shape, dtype):
        n = int(np.prod(shape))
        self.flat = torch.full((n + 2 * GUARD,), 7.0, dtype=dtype, device="cuda")
        self.t = self.flat[GUARD:GUARD + n].view(shape)
        self.t.fill_(float("nan"))

    def read(self):
        g = torch.cat([self.flat[:GUARD], self.flat[GUARD + self.t.numel():]])
        assert bool((g == 7.0).all()), "write outside an output"
        return self.t.double().cpu().numpy()


class Case:
    def __init__(self, R, T, H, dtype, form="both", post=True, gate=None, res=True, seed=1):
        self.R, self.T, self.H, self.dtype, self.form, self.post = R, T, H, dtype, form, post
        self.gate_shape = {None: None, "channel": (1, H), "scalar": (1, 1), "token": (T, 1), "full": (T, H)}.get(gate, gate)
        draw = lambda i, shape, std: gen.normal16((seed, i), shape, std, dtype)  # noqa: E731
        has_y, has_u = form != "pre", form != "post"
        raw = {"x": draw(1, (T, H), 2.0), "dx1": draw(2, (T, H), 0.05),
               "y": draw(3, (T, H), 0.7) if has_y else None,
               "du": draw(4, (T, H), 0.05) if has_u else None,
               "w_post": draw(5, (H,), 1.0) if has_y and post else None,
               "w_pre": draw(6, (H,), 1.0) if has_u else None,
               "gate": draw(7, self.gate_shape, 1.0) if has_y and self.gate_shape else None}
        self.np = {k: None if v is None else oracle.widen(v, dtype) for k, v in raw.items()}
        self.cu = {k: None if v is None else to_device(v, dtype) for k, v in raw.items()}
        self.rho = np.float32(0.85) if has_y and res else None
        self.res = None if self.rho is None else torch.tensor([float(self.rho)], device="cuda")
        g = self.gate_shape if self.cu["gate"] is not None else (3, 5)  # ignored without a gate
        self.sizes = (R, T, H, DT[dtype], int(post), g[0], g[1])

    def shards(self, t):
        return None if t is None else list(t.view(self.R, self.T // self.R, self.H))

    def outs(self):
        return [Out((self.T // self.R, self.H), torch_dtype(self.dtype)) for _ in range(self.R)]

    def forward(self, stream=None):
        c = self.cu
        xo = self.outs() if c["y"] is not None else None
        uo = self.outs() if self.form != "post" else None
        ry = Out((self.T,), torch.float32) if xo and self.post else None
        rx = Out((self.T,), torch.float32) if uo else None
        t = lambda o: None if o is None else [i.t for i in o] if isinstance(o, list) else o.t  # noqa: E731
        fx.flux_block_norm(*self.sizes, EPS, self.shards(c["x"]), self.shards(c["y"]), c["w_post"], c["gate"], self.res,
                           c["w_pre"], t(xo), t(uo), t(ry), t(rx), stream=stream)
        return xo, uo, ry, rx

    def reference(self):
        n = self.np
        rho = 1.0 if self.rho is None else float(self.rho)
        x1, u, ry, rx = oracle.block_norm(n["x"], n["y"], n["w_post"], n["gate"], rho, n["w_pre"], EPS, self.post)
        mag = np.abs(x1) if n["y"] is None else np.abs(rho * n["x"]) + np.abs(x1 - rho * n["x"])
        w = 1.0 if n["w_pre"] is None else np.abs(n["w_pre"])
        return x1, u, ry, rx, mag, mag * rx[:, None] * w


def _join(outs):
    return np.concatenate([o.read() for o in outs])


CASES = [
    # R, T, H, dtype, form, post, gate, res
    (1, 1, 8, "bf16", "both", True, "channel", True),
    (1, 1, 4096, "bf16", "both", True, None, False),
    (1, 3, 64, "f16", "both", True, "token", True),
    (2, 6, 256, "bf16", "both", False, "channel", False),
    (1, 67, 264, "f16", "both", True, "full", True),       # a gate for every token and channel
    (4, 20, 520, "bf16", "both", True, (5, 520), True),    # gate rows that cross shards
    (1, 130, 1016, "f16", "post", True, (2, 1), True),     # a scalar gate for each of two sequences
    (8, 88, 1032, "bf16", "pre", True, None, False),
    (1, 35, 2056, "f16", "both", True, (7, 2056), False),
    (3, 321, 2048, "bf16", "both", True, "channel", True),
    (1, 611, 512, "bf16", "both", True, (13, 512), True),  # gates whose rows several CTAs share
    (1, 17, 4104, "bf16", "both", True, "scalar", True),
    (2, 10, 8192, "f16", "both", True, "channel", True),
    (1, 5, 8200, "bf16", "both", True, (5, 8200), False),
    (1, 9, 12296, "f16", "both", False, "token", True),
    (1, 4, 16384, "bf16", "post", False, None, True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c).replace(" ", ""))
def test_forward(case):
    c = Case(*case)
    xo, uo, ry, rx = c.forward()
    x1, u, wry, wrx, mag, umag = c.reference()
    if xo:
        check16(_join(xo), x1, mag, c.dtype, what="x'")
    if uo:
        check16(_join(uo), u, umag, c.dtype, what="u")
        check32(rx.read(), wrx, wrx, what="rstd_x")
    if ry:
        check32(ry.read(), wry, wry, what="rstd_y")


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c).replace(" ", ""))
def test_backward(case):
    c = Case(*case, seed=2)
    x1, u, wry, wrx, _, _ = c.reference()
    f32 = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()  # noqa: E731
    ry = f32(wry) if wry is not None else None
    rx = f32(wrx) if c.form != "post" else None
    d, n = c.cu, c.np
    out = {"dx": c.outs(), "dy": c.outs() if d["y"] is not None else None,
           "dw_post": Out((c.H,), torch.float32) if d["w_post"] is not None else None,
           "dgate": Out(c.gate_shape, torch.float32) if d["gate"] is not None else None,
           "dres": Out((1,), torch.float32) if c.res is not None else None,
           "dw_pre": Out((c.H,), torch.float32) if d["du"] is not None else None}
    t = lambda o: None if o is None else [i.t for i in o] if isinstance(o, list) else o.t  # noqa: E731
    g = c.gate_shape if d["gate"] is not None else (0, 0)
    ws = _ws(fx.flux_block_norm_workspace_size(c.T, c.H, *g))
    for _ in range(2):  # the second call uses the workspace as the first left it
        fx.flux_block_norm_bwd(*c.sizes, c.shards(d["x"]), c.shards(d["y"]), d["w_post"], d["gate"], c.res, d["w_pre"],
                               ry, rx, c.shards(d["dx1"]), c.shards(d["du"]), t(out["dx"]), t(out["dy"]),
                               t(out["dw_post"]), t(out["dgate"]), t(out["dres"]), t(out["dw_pre"]), ws)
        first = {k: None if v is None else _join(v) if isinstance(v, list) else v.read() for k, v in out.items()}
        assert not bool(ws.any()), "the workspace is not zero again"
        if _ == 0:
            before = first
    for k in first:  # fixed summation order
        assert first[k] is None or np.array_equal(first[k], before[k]), k
    rho = 1.0 if c.rho is None else float(c.rho)
    ref = oracle.block_norm_bwd(n["x"], n["y"], n["w_post"], n["gate"], rho, n["w_pre"], EPS, n["dx1"], n["du"], c.post)
    for k in ("dx", "dy"):
        if first[k] is not None:
            check16(first[k], *ref[k], c.dtype, what=k)
    for k in ("dw_post", "dgate", "dres", "dw_pre"):
        if first[k] is not None:
            # rows summed by one thread, teams, CTAs, and the row's own arithmetic
            check32(first[k], *ref[k], depth=128 + min(c.T, 512), what=k)


def test_no_gradient_of_the_sum():
    # dx_out NULL stands for zeros; gradients that are not wanted are left out
    c = Case(1, 21, 768, "bf16", gate="channel")
    *_, wry, wrx, _, _ = c.reference()
    d, n = c.cu, c.np
    dx, dy = c.outs(), c.outs()
    ws = _ws(fx.flux_block_norm_workspace_size(c.T, c.H, 1, c.H))
    f32 = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()  # noqa: E731
    fx.flux_block_norm_bwd(*c.sizes, c.shards(d["x"]), c.shards(d["y"]), d["w_post"], d["gate"], c.res, d["w_pre"],
                           f32(wry), f32(wrx), None, c.shards(d["du"]), [o.t for o in dx], [o.t for o in dy],
                           None, None, None, None, ws)
    ref = oracle.block_norm_bwd(n["x"], n["y"], n["w_post"], n["gate"], float(c.rho), n["w_pre"], EPS, None, n["du"])
    check16(_join(dx), *ref["dx"], "bf16", what="dx")
    check16(_join(dy), *ref["dy"], "bf16", what="dy")
    assert not bool(ws.any())


def test_backward_in_place_equals_backward():
    c = Case(2, 600, 1024, "f16", gate="channel")
    *_, wry, wrx, _, _ = c.reference()
    d = c.cu
    f32 = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()  # noqa: E731
    ry, rx = f32(wry), f32(wrx)
    ws = _ws(fx.flux_block_norm_workspace_size(c.T, c.H, 1, c.H))

    def run(dx1, du, dx, dy):
        fx.flux_block_norm_bwd(*c.sizes, c.shards(d["x"]), c.shards(d["y"]), d["w_post"], d["gate"], c.res, d["w_pre"],
                               ry, rx, c.shards(dx1), c.shards(du), c.shards(dx), c.shards(dy), None, None, None, None, ws)
        return dx.clone(), dy.clone()

    want = run(d["dx1"], d["du"], torch.empty_like(d["x"]), torch.empty_like(d["x"]))
    a, b = d["dx1"].clone(), d["du"].clone()
    got = run(a, b, a, b)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    a, b = d["dx1"].clone(), d["du"].clone()
    got = run(a, b, b, a)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_forward_in_place_and_on_another_stream():
    c = Case(2, 514, 1280, "bf16", gate="token")
    xo, uo, _, _ = c.forward()
    want = (_join(xo), _join(uo))
    x, y = c.cu["x"].clone(), c.cu["y"].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    fx.flux_block_norm(*c.sizes, EPS, c.shards(x), c.shards(y), c.cu["w_post"], c.cu["gate"], c.res, c.cu["w_pre"],
                       c.shards(x), c.shards(y), stream=s)
    s.synchronize()
    assert np.array_equal(x.double().cpu().numpy(), want[0])
    assert np.array_equal(y.double().cpu().numpy(), want[1])


def test_odd_rows_stay_in_their_rows():
    # zeros, a NaN, an infinity and the largest values in rows of their own
    c = Case(1, 40, 1024, "bf16", gate=None, res=False)
    x, y = c.cu["x"], c.cu["y"]
    clean_x, clean_y = x.clone(), y.clone()
    xo, uo, _, _ = c.forward()
    want_x, want_u = _join(xo), _join(uo)
    x[3], y[3] = 0, 0
    y[7, 5] = float("nan")
    x[11, 1023] = float("inf")
    x[20], y[20] = torch.finfo(torch.bfloat16).max / 4, 0
    xo, uo, ry, rx = c.forward()
    got_x, got_u = _join(xo), _join(uo)
    keep = [i for i in range(40) if i not in (3, 7, 11, 20)]
    assert np.array_equal(got_x[keep], want_x[keep]) and np.array_equal(got_u[keep], want_u[keep])
    assert not got_x[3].any() and not got_u[3].any()
    assert abs(rx.read()[3] - EPS ** -0.5) < 1e-4 * EPS ** -0.5
    assert np.isnan(got_u[7]).all() and np.isinf(got_x[11, 1023])
    # 2^126 squared is past fp32: the mean is infinite and the norm 0
    assert np.isfinite(got_x[20]).all() and not got_u[20].any()
    x.copy_(clean_x), y.copy_(clean_y)


def test_offsets_past_32_bits():
    T, H = 131080, 16384  # 2^31 + 2^17 elements
    tail = 5
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    r = gen.normal16((77, 1), (tail, H), 1.0, "bf16")
    x[-tail:] = to_device(r, "bf16")
    y = x.flip(0)
    fx.flux_block_norm(1, T, H, fx.FLUX_BF16, 1, 0, 0, EPS, [x], [y], None, None, None, None, [x], [y])
    n = oracle.widen(r, "bf16")
    x1, u, _, _ = oracle.block_norm(n, np.zeros_like(n), None, None, 1.0, None, EPS)
    got = oracle.widen(from_device(x[-tail:]), "bf16"), oracle.widen(from_device(y[-tail:]), "bf16")
    check16(got[0], x1, np.abs(x1), "bf16")
    check16(got[1], u, np.abs(u), "bf16")
    assert not bool(x[tail:2048].any())
    torch.cuda.empty_cache()


def test_empty():
    f = lambda n: torch.full((n,), 3.0, device="cuda")  # noqa: E731
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    a = torch.zeros(64, dtype=torch.bfloat16, device="cuda")  # an address for the empty shards
    fx.flux_block_norm(1, 0, 64, fx.FLUX_BF16, 1, 1, 64, EPS, [a], [a], None, a, None, None, [a], [a])
    dw, dg, dr, dp = f(64), f(64), f(4), f(64)
    res = f(4)
    fx.flux_block_norm_bwd(1, 0, 64, fx.FLUX_BF16, 1, 1, 64, [a], [a], a, a, res, a, None, None, None, [a], [a], [a],
                           dw, dg, dr, dp, _ws(256))
    assert not dw.any() and not dg.any() and not dp.any() and float(dr[0]) == 0.0 and float(dr[1]) == 3.0
    assert e.numel() == 0


def test_chain_of_sizes_keeps_unit_rows():
    # every width that changes how a row is held: u of a unit-weight norm has mean square 1
    for H in (8, 16, 248, 256, 264, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 12288, 12296, 16384):
        x = torch.randn((9, H), device="cuda").to(torch.float16)
        u = torch.empty_like(x)
        fx.flux_block_norm(1, 9, H, fx.FLUX_F16, 0, 0, 0, 0.0, [x], None, None, None, None, None, None, [u])
        ms = u.double().square().mean(1)
        assert float((ms - 1).abs().max()) < 4 * U16["f16"], H
