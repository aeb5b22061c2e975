"""GPU parity of layer norm with dropout and residual (flux_layer_norm,
flux_layer_norm_bwd) with their float64 definitions, through the C ABI."""
import numpy as np
import pytest

import oracle
from tests.rounding import check16, check32
from workloads import gen
from workloads.torch_io import to_device, torch_dtype

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import reducescatter_tcgen05_tmem_gb300 as fx  # noqa: E402

DT = {"f16": fx.FLUX_F16, "bf16": fx.FLUX_BF16}
EPS = 1e-5
GUARD = 64
SEED, OFFSET = 0x123456789ABCDEF, (5 << 32) + 77


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


def _join(outs):
    return np.concatenate([o.read() for o in outs])


def _t(o):
    return None if o is None else [i.t for i in o] if isinstance(o, list) else o.t


class Case:
    """form: both (x, y, u), pre (x, u), sum (x, y), first (y, u)."""

    def __init__(self, R, T, H, dtype, form="both", p=0.1, weight=True, bias=True, seed=1, shift=0.0):
        self.R, self.T, self.H, self.dtype, self.form = R, T, H, dtype, form
        self.p = p if form != "pre" else 0.0
        draw = lambda i, shape, std: gen.normal16((seed, i), shape, std, dtype)  # noqa: E731
        has_u = form != "sum"
        raw = {"x": draw(1, (T, H), 2.0) if form != "first" else None, "y": draw(2, (T, H), 0.7) if form != "pre" else None,
               "w": draw(3, (H,), 1.0) if has_u and weight else None, "b": draw(4, (H,), 0.5) if has_u and bias else None,
               "dx1": draw(5, (T, H), 0.05), "du": draw(6, (T, H), 0.05) if has_u else None}
        self.cu = {k: None if v is None else to_device(v, dtype) for k, v in raw.items()}
        if shift:
            self.cu["x"] += shift
        self.np = {k: None if v is None else v.double().cpu().numpy() for k, v in self.cu.items()}
        self.rng = torch.tensor([SEED, OFFSET], dtype=torch.int64, device="cuda") if self.p > 0 else None
        self.factor = oracle.dropout_factor(T, H, self.p, SEED, OFFSET) if self.p > 0 else None
        self.sizes = (R, T, H, DT[dtype], self.p)

    def shards(self, t):
        return None if t is None else list(t.view(self.R, self.T // self.R, self.H))

    def outs(self):
        return [Out((self.T // self.R, self.H), torch_dtype(self.dtype)) for _ in range(self.R)]

    def forward(self, stream=None):
        c = self.cu
        xo = self.outs() if c["y"] is not None else None
        uo, m, r = (self.outs(), Out((self.T,), torch.float32), Out((self.T,), torch.float32)) if self.form != "sum" else (None,) * 3
        fx.flux_layer_norm(*self.sizes, EPS, self.shards(c["x"]), self.shards(c["y"]), self.rng, c["w"], c["b"],
                           _t(xo), _t(uo), _t(m), _t(r), stream=stream)
        return xo, uo, m, r

    def reference(self):
        n = self.np
        return oracle.layer_norm(n["x"], n["y"], self.factor, n["w"], n["b"], EPS)


CASES = [
    # R, T, H, dtype, form, p, weight, bias
    (1, 1, 8, "bf16", "both", 0.1, True, True),
    (1, 1, 4096, "bf16", "both", 0.0, True, True),
    (1, 3, 64, "f16", "both", 0.5, True, False),
    (2, 6, 256, "bf16", "both", 0.1, False, True),
    (1, 67, 264, "f16", "both", 0.25, True, True),
    (4, 20, 520, "bf16", "both", 0.9, True, True),
    (1, 130, 1016, "f16", "sum", 0.1, False, False),
    (8, 88, 1032, "bf16", "pre", 0.0, True, True),
    (1, 35, 2056, "f16", "first", 0.1, True, True),
    (3, 321, 2048, "bf16", "both", 0.1, True, True),
    (1, 1611, 512, "bf16", "both", 0.1, True, True),
    (1, 17, 4104, "bf16", "both", 1e-3, True, True),
    (2, 10, 8192, "f16", "both", 0.1, True, True),
    (1, 5, 8200, "bf16", "pre", 0.0, True, True),
    (1, 9, 12296, "f16", "both", 0.1, True, True),
    (1, 4, 16384, "bf16", "first", 0.3, False, False),
    (1, 700, 5120, "f16", "both", 0.1, True, True),
    (1, 3000, 8, "f16", "both", 0.1, True, True),
]
IDS = lambda c: "-".join(str(v) for v in c)  # noqa: E731


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    c = Case(*case)
    xo, uo, m, r = c.forward()
    x1, u, wm, wr, mag, umag = c.reference()
    if xo:
        check16(_join(xo), x1, mag, c.dtype, what="x'")
        if c.form == "first":
            assert np.array_equal(_join(xo) != 0, (c.factor > 0) & (c.np["y"] != 0))
    if uo:
        check16(_join(uo), u, umag, c.dtype, what="u")
        check32(m.read(), wm, mag.mean(1), what="mean")
        check32(r.read(), wr, wr * (1 + 2 * mag.max(1) * wr), what="rstd")


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case):
    c = Case(*case, seed=2)
    d, n = c.cu, c.np
    x1 = m = r = None
    if c.form != "sum":
        full = c.reference()
        x1 = to_device(gen.normal16((9, 1), (c.T, c.H), 2.0, c.dtype), c.dtype) if c.form == "pre" else \
            torch.from_numpy(full[0]).to(torch_dtype(c.dtype)).cuda()
        h = x1.double()
        m, r = h.mean(1).float(), (h.var(1, unbiased=False) + EPS).rsqrt().float()
    has_y = c.form != "pre"
    out = {"dx": c.outs(), "dy": c.outs() if has_y else None,
           "dw": Out((c.H,), torch.float32) if x1 is not None else None,
           "db": Out((c.H,), torch.float32) if x1 is not None else None}
    ws = _ws(fx.flux_layer_norm_workspace_size(c.T, c.H))
    for i in range(2):  # the second call uses the workspace as the first left it
        fx.flux_layer_norm_bwd(*c.sizes, c.shards(x1), c.rng, d["w"], m, r, c.shards(d["dx1"]), c.shards(d["du"]),
                               _t(out["dx"]), _t(out["dy"]), _t(out["dw"]), _t(out["db"]), ws)
        got = {k: None if v is None else _join(v) if isinstance(v, list) else v.read() for k, v in out.items()}
        if i == 0:
            first = got
    assert not bool(ws.any()), "the workspace is left zero"
    f64 = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    want = oracle.layer_norm_bwd(f64(x1), f64(m), f64(r), n["w"], n["dx1"], n["du"], c.factor)
    for k, v in got.items():
        if v is None:
            continue
        assert np.array_equal(v, first[k]), k
        check = check16 if k in ("dx", "dy") else check32
        args = (c.dtype,) if k in ("dx", "dy") else ()
        check(v, *want[k], *args, what=k)
    if c.factor is not None and has_y:
        assert np.array_equal(got["dy"] != 0, (c.factor > 0) & (got["dy"] != 0)), "a dropped element has no gradient"


def test_rows_far_from_zero():
    # a mean 500 times the deviation: the squares alone would lose the variance
    c = Case(1, 50, 1024, "f16", "pre", shift=1000.0)
    _, uo, m, r = c.forward()
    x1, u, wm, wr, mag, umag = c.reference()
    check16(_join(uo), u, umag, c.dtype, what="u")
    check32(m.read(), wm, mag.mean(1), what="mean")
    check32(r.read(), wr, wr * (1 + 2 * mag.max(1) * wr), what="rstd")


def test_constant_rows_and_what_a_dropped_element_held():
    H = 512
    x = torch.full((2, H), 3.0, dtype=torch.bfloat16, device="cuda")
    u = torch.empty_like(x)
    fx.flux_layer_norm(1, 2, H, fx.FLUX_BF16, 0.0, EPS, [x], None, None, None, None, None, [u])
    assert bool((u == 0).all())
    f = oracle.dropout_factor(2, H, 0.5, SEED, OFFSET)
    rng = torch.tensor([SEED, OFFSET], dtype=torch.int64, device="cuda")
    y = torch.ones(2, H, dtype=torch.bfloat16, device="cuda")
    y[torch.from_numpy(f == 0).cuda()] = float("nan")
    xo = torch.empty_like(x)
    fx.flux_layer_norm(1, 2, H, fx.FLUX_BF16, 0.5, EPS, [x], [y], rng, None, None, [xo], [u])
    assert np.array_equal(xo.double().cpu().numpy(), 3.0 + f)
    assert bool(torch.isfinite(u).all())


def test_a_row_that_is_not_finite_stays_alone():
    c = Case(1, 40, 1040, "bf16")
    clean = [_join(o) if isinstance(o, list) else o.read() for o in c.forward()]
    c.cu["x"][17, 3] = float("inf")
    got = [_join(o) if isinstance(o, list) else o.read() for o in c.forward()]
    rows = np.arange(40) != 17
    for a, b in zip(got, clean):
        assert np.array_equal(a[rows], b[rows])


def test_outputs_over_inputs():
    c = Case(2, 24, 1032, "bf16", seed=4)
    xo, uo, m, r = c.forward()
    x, y = c.cu["x"].clone(), c.cu["y"].clone()
    fx.flux_layer_norm(*c.sizes, EPS, c.shards(x), c.shards(y), c.rng, c.cu["w"], c.cu["b"], c.shards(x), c.shards(y))
    assert torch.equal(x, torch.cat([o.t for o in xo])) and torch.equal(y, torch.cat([o.t for o in uo]))
    ws = _ws(fx.flux_layer_norm_workspace_size(c.T, c.H))
    want = [c.outs(), c.outs()]
    d = c.cu
    fx.flux_layer_norm_bwd(*c.sizes, c.shards(x), c.rng, d["w"], m.t, r.t, c.shards(d["dx1"]), c.shards(d["du"]),
                           _t(want[0]), _t(want[1]), None, None, ws)
    dx1, du = d["dx1"].clone(), d["du"].clone()
    fx.flux_layer_norm_bwd(*c.sizes, c.shards(x), c.rng, d["w"], m.t, r.t, c.shards(dx1), c.shards(du),
                           c.shards(dx1), c.shards(du), None, None, ws)
    assert torch.equal(dx1, torch.cat([o.t for o in want[0]])) and torch.equal(du, torch.cat([o.t for o in want[1]]))


@pytest.mark.parametrize("which", ["dx", "dy", "dx_zero", "dw", "db"])
def test_parts_of_the_backward_pass(which):
    c = Case(1, 77, 2048, "f16", seed=5)
    xo, _, m, r = c.forward()
    x1 = xo[0].t
    d = c.cu
    ws = _ws(fx.flux_layer_norm_workspace_size(c.T, c.H))
    dx, dy, dw, db = c.outs(), c.outs(), Out((c.H,), torch.float32), Out((c.H,), torch.float32)
    dx1 = None if which == "dx_zero" else [d["dx1"]]
    fx.flux_layer_norm_bwd(*c.sizes, [x1], c.rng, d["w"], m.t, r.t, dx1, [d["du"]], None if which == "dy" else _t(dx),
                           None if which == "dx" else _t(dy), None if which == "db" else dw.t,
                           None if which == "dw" else db.t, ws)
    want = oracle.layer_norm_bwd(x1.double().cpu().numpy(), m.read(), r.read(), c.np["w"], None if dx1 is None else c.np["dx1"],
                                 c.np["du"], c.factor)
    for k, o, left in (("dx", dx, which == "dy"), ("dy", dy, which == "dx"), ("dw", dw, which == "db"), ("db", db, which == "dw")):
        v = _join(o) if isinstance(o, list) else o.read()
        if left:
            assert np.isnan(v).all(), f"{k} was not asked for"
        elif k in ("dx", "dy"):
            check16(v, *want[k], c.dtype, what=k)
        else:
            check32(v, *want[k], what=k)


def test_long_batch_sums():
    # 288 rows and more of a team in one register: the order's depth grows with them
    T, H = 140000, 520
    c = Case(1, T, H, "bf16", seed=6)
    xo, _, m, r = c.forward()
    x1 = xo[0].t
    ws = _ws(fx.flux_layer_norm_workspace_size(T, H))
    dx, dy, dw, db = (torch.empty_like(x1) for _ in range(2)), None, torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    dx, dy = dx
    fx.flux_layer_norm_bwd(*c.sizes, [x1], c.rng, c.cu["w"], m.t, r.t, [c.cu["dx1"]], [c.cu["du"]], [dx], [dy], dw, db, ws)
    want = oracle.layer_norm_bwd(x1.double().cpu().numpy(), m.read(), r.read(), c.np["w"], c.np["dx1"], c.np["du"], c.factor)
    check16(dx.double().cpu().numpy(), *want["dx"], "bf16", what="dx")
    check16(dy.double().cpu().numpy(), *want["dy"], "bf16", what="dy")
    check32(dw.double().cpu().numpy(), *want["dw"], depth=512, what="dw")
    check32(db.double().cpu().numpy(), *want["db"], depth=512, what="db")


def test_no_rows():
    ws = _ws(256)
    dw = torch.full((64,), 5.0, device="cuda")
    db = dw.clone()
    one = torch.zeros(64, device="cuda")
    fx.flux_layer_norm_bwd(1, 0, 64, fx.FLUX_F16, 0.0, [None], None, None, one, one, None, [None], [None], None, dw, db, ws)
    assert not bool(dw.any()) and not bool(db.any())


def test_captured_step_draws_the_numbers_it_finds():
    c = Case(1, 64, 1024, "bf16", seed=7)
    side = torch.cuda.Stream()
    xo, uo = torch.empty_like(c.cu["x"]), torch.empty_like(c.cu["x"])
    m, r = torch.empty(64, device="cuda"), torch.empty(64, device="cuda")
    dx, dy, dw = torch.empty_like(xo), torch.empty_like(xo), torch.empty(1024, device="cuda")
    ws = _ws(fx.flux_layer_norm_workspace_size(64, 1024))

    def step():
        d = c.cu
        fx.flux_layer_norm(*c.sizes, EPS, [d["x"]], [d["y"]], c.rng, d["w"], d["b"], [xo], [uo], m, r)
        fx.flux_layer_norm_bwd(*c.sizes, [xo], c.rng, d["w"], m, r, [d["dx1"]], [d["du"]], [dx], [dy], dw, None, ws)
        c.rng[1] += 1

    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    for _ in range(3):
        offset = int(c.rng[1])
        graph.replay()
        torch.cuda.synchronize()
        f = oracle.dropout_factor(64, 1024, c.p, SEED, offset)
        want = oracle.layer_norm(c.np["x"], c.np["y"], f, c.np["w"], c.np["b"], EPS)
        check16(xo.double().cpu().numpy(), want[0], want[4], "bf16", what="x'")
        assert np.array_equal(dy.double().cpu().numpy() != 0, (f > 0) & (dx.double().cpu().numpy() != 0))


def test_repeats_and_own_stream():
    c = Case(1, 999, 4096, "bf16", seed=8)
    first = [_join(o) if isinstance(o, list) else o.read() for o in c.forward()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = c.forward(stream=side)
    side.synchronize()
    for a, b in zip(out, first):
        assert np.array_equal(_join(a) if isinstance(a, list) else a.read(), b)
