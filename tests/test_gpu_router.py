"""GPU parity of the router's losses, counts and score gradient
(flux_moe_balance_loss, flux_moe_router_bwd) with their float64 definitions."""
import numpy as np
import pytest

import oracle
from tests.rounding import U32, check32

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import reducescatter_tcgen05_tmem_gb300 as fx  # noqa: E402

A, B = 0.02, 0.003


def _ws(nbytes):
    n = max(nbytes, 256) // 4
    ws = torch.zeros(n + 64, dtype=torch.int32, device="cuda")
    off = (-ws.data_ptr()) % 256 // 4
    return ws[off:off + n]


def _inputs(T, E, k, S, mask, seed):
    r = np.random.default_rng(seed)
    logits = (r.standard_normal((T, E)) + np.log(np.arange(1, E + 1.0) ** -1.2)).astype(np.float32)
    m = None
    if mask == "some":
        m = (r.random(T) < 0.6).astype(np.uint8) * 3  # any nonzero value keeps a token
    elif mask == "empty":  # the first sequence has no token left
        m = np.ones(T, np.uint8)
        m[:T // S] = 0
    elif mask == "none left":
        m = np.zeros(T, np.uint8)
    ids, w = oracle.moe_topk_gate(logits, k)
    return logits, ids, w.astype(np.float32), m


class Router:
    def __init__(self, T, E, k, S, mask, seed=3, logits=None):
        self.T, self.E, self.k, self.S = T, E, k, S
        self.logits, self.ids, self.w, self.mask = _inputs(T, E, k, S, mask, seed)
        if logits is not None:
            self.logits = logits
            self.ids, w = oracle.moe_topk_gate(logits, k)
            self.w = w.astype(np.float32)
        cu = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.d = [cu(a) for a in (self.logits, self.ids, self.w, self.mask)]
        e = lambda n, dt: torch.full((n + 8,), 77, dtype=dt, device="cuda")  # noqa: E731
        self.out = {"loss": e(2, torch.float32), "counts": e(S * E, torch.int32), "probs": e(S * E, torch.float32),
                    "tokens": e(S + 1, torch.int32), "lse": e(T, torch.float32)}
        self.ws = _ws(fx.flux_moe_balance_workspace_size(T, E, k, S))

    def forward(self):
        o = self.out
        fx.flux_moe_balance_loss(self.T, self.E, self.k, self.S, A, B, self.d[0], self.d[1], self.d[3], o["loss"],
                                 o["counts"], o["probs"], o["tokens"], o["lse"], self.ws)
        got = {}
        for name, n in (("loss", 2), ("counts", self.S * self.E), ("probs", self.S * self.E), ("tokens", self.S + 1),
                        ("lse", self.T)):
            a = o[name].cpu().numpy()
            assert (a[n:] == 77).all(), f"write past {name}"
            got[name] = a[:n]
        got["counts"] = got["counts"].reshape(self.S, self.E)
        got["probs"] = got["probs"].reshape(self.S, self.E).astype(np.float64)
        return got

    def reference(self):
        return oracle.balance_loss(self.logits.astype(np.float64), self.ids, self.S, A, B, self.mask)


CASES = [
    # T, E, topk, S, mask
    (1, 1, 1, 1, None),
    (1, 8, 2, 1, None),
    (5, 2, 1, 5, None),
    (37, 3, 3, 1, "some"),
    (128, 8, 2, 4, "empty"),
    (129, 32, 4, 3, "some"),
    (64, 33, 2, 64, "some"),      # a sequence per token
    (200, 64, 6, 2, None),
    (96, 100, 8, 1, "none left"),
    (77, 256, 8, 7, "some"),
    (63, 300, 5, 1, None),
    (30, 1000, 9, 2, "some"),
    (24, 1024, 40, 1, None),
    (4099, 16, 2, 1, "some"),
    (3000, 7, 2, 600, None),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c).replace(" ", "_"))
def test_losses_and_counts(case):
    r = Router(*case)
    got = r.forward()
    again = r.forward()  # the workspace is left as it was found, the order of the sums is fixed
    loss, counts, probs, tokens, lse = r.reference()
    for k in got:
        assert np.array_equal(got[k], again[k]), k
    assert np.array_equal(got["counts"], counts) and np.array_equal(got["tokens"], tokens)
    check32(got["lse"], lse, np.abs(lse) + 1.0, what="lse")
    # a probability is off by the exponent's argument (|score - lse| 2^-24), exp and
    # the division; then the sum over the tokens
    depth = 160 + min(r.T, 512)
    check32(got["probs"], probs, probs * 2, depth=depth, what="probs")
    check32(got["loss"], loss, np.abs(loss) * 2, depth=depth, what="loss")
    assert not bool(r.ws.any())


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c).replace(" ", "_"))
@pytest.mark.parametrize("gate", [True, False])
def test_score_gradient(case, gate):
    r = Router(*case, seed=4)
    _, counts, _, tokens, lse = r.reference()
    rng = np.random.default_rng(9)
    dw = rng.standard_normal((r.T, r.k)).astype(np.float32) if gate else None
    dloss = np.array([0.7, -1.3], np.float32) if gate else None
    cu = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    out = torch.full((r.T * r.E + 16,), 77.0, device="cuda")
    lse32 = lse.astype(np.float32)
    fx.flux_moe_router_bwd(r.T, r.E, r.k, r.S, A, B, r.d[0], r.d[1] if gate else None, r.d[2] if gate else None, r.d[3],
                           cu(lse32), cu(counts.astype(np.int32)), cu(tokens.astype(np.int32)), cu(dloss), cu(dw), out)
    assert bool((out[r.T * r.E:] == 77.0).all())
    got = out[:r.T * r.E].view(r.T, r.E).double().cpu().numpy()
    ref, mag = oracle.router_bwd(r.logits.astype(np.float64), r.ids, r.w.astype(np.float64), r.S, A, B, counts, tokens,
                                 (1.0, 1.0) if dloss is None else dloss.astype(np.float64),
                                 None if dw is None else dw.astype(np.float64), r.mask)
    check32(got, ref, mag, depth=128, what="dlogits")


def test_score_gradient_is_the_losses_difference():
    # the device's gradient against central differences of the float64 losses
    r = Router(24, 9, 2, 2, "some", seed=6)
    got = r.forward()
    o = r.out
    out = torch.empty((24, 9), device="cuda")
    fx.flux_moe_router_bwd(24, 9, 2, 2, A, B, r.d[0], None, None, r.d[3], o["lse"], o["counts"], o["tokens"], None, None, out)
    g = out.double().cpu().numpy()
    z, h = r.logits.astype(np.float64), 1e-5
    for t, e in [(0, 0), (5, 8), (11, 3), (12, 0), (23, 7)]:
        p, m = z.copy(), z.copy()
        p[t, e] += h
        m[t, e] -= h
        f = lambda a: oracle.balance_loss(a, r.ids, 2, A, B, r.mask)[0].sum()  # noqa: E731
        want = (f(p) - f(m)) / (2 * h)
        assert abs(g[t, e] - want) <= 128 * U32 * (abs(want) + A + B) + 1e-9, (t, e)
    assert got["tokens"][2] == int((r.mask != 0).sum())


def test_odd_scores():
    T, E = 8, 6
    z = np.random.default_rng(1).standard_normal((T, E)).astype(np.float32)
    z[1] = -np.inf
    z[2, 3] = np.inf
    z[3, [0, 5]] = np.inf
    z[4, 2] = np.nan
    z[5] = np.nan
    z[6, 1:] = -np.inf
    z[7] = -3.4028235e38
    r = Router(T, E, 2, 1, None, logits=z)
    got = r.forward()
    loss, counts, probs, tokens, lse = r.reference()
    assert np.array_equal(got["counts"], counts)
    fin = np.isfinite(lse)
    assert np.array_equal(got["lse"][~fin], lse[~fin].astype(np.float32))
    check32(got["lse"][fin], lse[fin], np.abs(lse[fin]) + 1)
    check32(got["probs"], probs, probs * 2)
    # row 7: the square of its lse is past fp32 and takes the z loss to infinity
    assert np.isinf(got["loss"][1]) and abs(got["loss"][0] - loss[0]) < 1e-6
    dw = torch.randn((T, 2), device="cuda")
    out = torch.full((T, E), 77.0, device="cuda")
    o = r.out
    fx.flux_moe_router_bwd(T, E, 2, 1, A, 0.0, r.d[0], r.d[1], r.d[2], None, o["lse"], o["counts"], o["tokens"], None, dw, out)
    g = out.double().cpu().numpy()
    assert not g[[1, 2, 3, 5]].any() and np.isfinite(g[[0, 4, 6]]).all()
    assert g[4, 2] == 0 and not g[6, 1:].any()


def test_id_out_of_range_is_reported():
    r = Router(16, 4, 2, 1, None)
    r.d[1][3, 1] = 4
    r.d[1][5, 0] = -1
    ids = r.ids.copy()
    ids[3, 1], ids[5, 0] = 4, -1
    got = r.forward()
    _, counts, *_ = oracle.balance_loss(r.logits.astype(np.float64), ids, 1, A, B)
    assert np.array_equal(got["counts"], counts)
    st, _ = fx.flux_get_status(r.ws)
    assert st == fx.FLUX_ERR_INVALID_ARG
    st, _ = fx.flux_get_status(r.ws)
    assert st == fx.FLUX_OK


def test_no_tokens():
    o = Router(4, 5, 2, 1, None)
    fx.flux_moe_balance_loss(0, 5, 2, 1, A, B, None, None, None, o.out["loss"], o.out["counts"], o.out["probs"],
                             o.out["tokens"], None, o.ws)
    assert not o.out["loss"][:2].any() and not o.out["counts"][:5].any() and not o.out["tokens"][:2].any()
    fx.flux_moe_router_bwd(0, 5, 2, 1, A, B, None, None, None, None, None, None, None, None, None, None)


def test_another_stream():
    r = Router(500, 8, 2, 1, None)
    want = r.forward()
    for v in r.out.values():
        v.fill_(5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o = r.out
    fx.flux_moe_balance_loss(500, 8, 2, 1, A, B, r.d[0], r.d[1], None, o["loss"], o["counts"], o["probs"], o["tokens"],
                             o["lse"], r.ws, stream=s)
    s.synchronize()
    assert np.array_equal(o["loss"][:2].cpu().numpy(), want["loss"])
    assert np.array_equal(o["lse"][:500].cpu().numpy(), want["lse"])


def test_sum_over_a_long_batch_is_exact_in_the_counts():
    T, E, k = 1 << 18, 40, 3
    r = torch.Generator(device="cuda")
    r.manual_seed(1)
    logits = torch.randn((T, E), device="cuda", generator=r)
    ids = logits.topk(k, dim=1).indices.to(torch.int32).contiguous()
    o = {n: torch.empty(m, dtype=d, device="cuda") for n, m, d in
         (("loss", 2, torch.float32), ("counts", E, torch.int32), ("probs", E, torch.float32), ("tokens", 2, torch.int32),
          ("lse", T, torch.float32))}
    fx.flux_moe_balance_loss(T, E, k, 1, A, B, logits, ids, None, o["loss"], o["counts"], o["probs"], o["tokens"], o["lse"],
                             _ws(fx.flux_moe_balance_workspace_size(T, E, k, 1)))
    assert torch.equal(o["counts"].long(), torch.bincount(ids.reshape(-1).long(), minlength=E))
    p = torch.softmax(logits.double(), 1).mean(0).cpu().numpy()
    check32(o["probs"].cpu().numpy(), p, p * 2, depth=700)
    assert abs(float(o["probs"].double().sum()) - 1) < 700 * U32 * 2


@pytest.mark.parametrize("T,E,k,S", [(512, 8, 2, 1), (700, 256, 4, 1), (640, 16, 2, 64), (4096, 32, 2, 4)])
def test_what_a_workspace_holds_past_its_header_does_not_matter(T, E, k, S):
    # the MoE layers leave their routing in theirs
    r = Router(T, E, k, S, "some")
    want = r.forward()
    r.ws[64:] = 0x7F7F7F7F
    got = r.forward()
    for n in want:
        assert np.array_equal(got[n], want[n]), n
    assert not bool(r.ws[:64].any())
