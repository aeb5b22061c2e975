"""The layer norm, the grouped router and the 8-bit products behind one another and
beside the MoE layers, as a block uses them: eagerly, captured, on two streams."""
import numpy as np
import pytest

import oracle
from tests.rounding import check16, check32

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import reducescatter_tcgen05_tmem_gb300 as fx  # noqa: E402

BF = fx.FLUX_BF16
EPS, P, SEED = 1e-5, 0.1, 99


def _ws(nbytes):
    return torch.zeros(max(nbytes, 256) // 4 + 64, dtype=torch.int32, device="cuda")[:max(nbytes, 256) // 4]


class Block:
    """x -> norm -> router -> experts -> dropout, residual, next norm; and back to the
    gradients of x, of the experts' output and of the router's scores."""

    R, T, H, F, E, K = 2, 96, 256, 512, 32, 4

    def __init__(self, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        R, T, H, F, E, K = self.R, self.T, self.H, self.F, self.E, self.K
        n = lambda *s, std=1.0: torch.randn(s, generator=g, device="cuda") * std  # noqa: E731
        b = lambda *s, std=1.0: n(*s, std=std).bfloat16()  # noqa: E731
        e = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
        self.x, self.w, self.b = b(T, H, std=2.0), b(H, std=0.2) + 1, b(H, std=0.1)
        self.gate, self.bias = n(H, E, std=H ** -0.5), n(E, std=0.05)
        self.w1 = [b(E, H, F // R, std=H ** -0.5) for _ in range(R)]
        self.w2 = [b(E, F // R, H, std=F ** -0.5) for _ in range(R)]
        self.dx1, self.du1, self.dweights = b(T, H, std=0.05), b(T, H, std=0.05), n(T, K, std=0.1)
        self.rng = torch.tensor([SEED, 0], device="cuda")
        self.u, self.y, self.x1, self.u1, self.dx, self.dy = (e(T, H) for _ in range(6))
        self.h = [e(T * K, F // R) for _ in range(R)]
        f = torch.float32
        self.mean, self.rstd, self.mean1, self.rstd1 = (e(T, dt=f) for _ in range(4))
        self.logits, self.dlogits = e(T, E, dt=f), e(T, E, dt=f)
        self.ids, self.weights = e(T, K, dt=torch.int32), e(T, K, dt=f)
        self.dw, self.db = e(H, dt=f), e(H, dt=f)
        self.moe_ws = _ws(fx.flux_moe_workspace_size(fx.FLUX_OP_MOE_LAYERS, R, T, H, F, E, K))
        self.ws = _ws(fx.flux_layer_norm_workspace_size(T, H))

    def rows(self, t):
        return list(t.view(self.R, self.T // self.R, self.H))

    def step(self):
        R, T, H, F, E, K = self.R, self.T, self.H, self.F, self.E, self.K
        fx.flux_layer_norm(R, T, H, BF, 0.0, EPS, self.rows(self.x), None, None, self.w, self.b, None, self.rows(self.u),
                           self.mean, self.rstd)
        torch.matmul(self.u.float(), self.gate, out=self.logits)
        fx.flux_moe_group_gate(T, E, K, fx.FLUX_SCORE_SIGMOID, 4, 2, 2, 1, 2.5, self.logits, self.bias, self.ids, self.weights)
        fx.flux_moe_layers(R, T, H, F, E, K, BF, self.rows(self.u), self.w1, self.w2, self.ids, self.weights, self.h,
                           self.rows(self.y), None, self.moe_ws)
        fx.flux_layer_norm(R, T, H, BF, P, EPS, self.rows(self.x), self.rows(self.y), self.rng, self.w, self.b,
                           self.rows(self.x1), self.rows(self.u1), self.mean1, self.rstd1)
        fx.flux_layer_norm_bwd(R, T, H, BF, P, self.rows(self.x1), self.rng, self.w, self.mean1, self.rstd1, self.rows(self.dx1),
                               self.rows(self.du1), self.rows(self.dx), self.rows(self.dy), self.dw, self.db, self.ws)
        fx.flux_moe_group_gate_bwd(T, E, K, fx.FLUX_SCORE_SIGMOID, 1, 2.5, self.logits, self.ids, self.dweights, 0, self.dlogits)
        self.rng[1] += 1

    def outputs(self):
        return [self.u, self.logits, self.ids, self.weights, self.y, self.x1, self.u1, self.dx, self.dy, self.dw, self.db,
                self.dlogits]

    def check(self, offset):
        d = lambda t: t.double().cpu().numpy()  # noqa: E731
        st, rep = fx.flux_get_status(self.moe_ws)
        assert st == fx.FLUX_OK, rep
        _, u, _, _, _, mag = oracle.layer_norm(d(self.x), None, None, d(self.w), d(self.b), EPS)
        check16(d(self.u), u, mag, "bf16", what="u")
        ids, w = oracle.group_gate(d(self.logits), d(self.bias), self.K, "sigmoid", 4, 2, 2, True, 2.5)
        assert np.array_equal(self.ids.cpu().numpy(), ids)
        check32(d(self.weights), w, np.abs(w), what="weights")
        # the experts with what the router gave them (h is rounded to 16 bits in between)
        bits = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
        h, _ = oracle.moe_layer0([bits(v) for v in self.rows(self.u)], [bits(v) for v in self.w1], ids, self.E, "bf16")
        y = oracle.moe_layer1([oracle.round_to(v, "bf16") for v in h], [bits(v) for v in self.w2], ids, w, self.E, "bf16", h_dtype="f64")
        y = np.concatenate(y)
        assert np.linalg.norm(d(self.y) - y) < 5e-3 * np.linalg.norm(y)
        f = oracle.dropout_factor(self.T, self.H, P, SEED, offset)
        x1, u1, _, _, m1, mu = oracle.layer_norm(d(self.x), d(self.y), f, d(self.w), d(self.b), EPS)
        check16(d(self.x1), x1, m1, "bf16", what="x'")
        check16(d(self.u1), u1, mu, "bf16", what="u'")
        g = oracle.layer_norm_bwd(d(self.x1), d(self.mean1), d(self.rstd1), d(self.w), d(self.dx1), d(self.du1), f)
        check16(d(self.dx), *g["dx"], "bf16", what="dx")
        check16(d(self.dy), *g["dy"], "bf16", what="dy")
        check32(d(self.dw), *g["dw"], what="dw")
        check32(d(self.db), *g["db"], what="db")
        dl, mag = oracle.group_gate_bwd(d(self.logits), ids, d(self.dweights), "sigmoid", True, 2.5)
        check32(d(self.dlogits), dl, mag, what="dlogits")


def test_block_eager_and_captured():
    b = Block()
    b.step()
    torch.cuda.synchronize()
    b.check(0)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b.step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            b.step()
    for i in range(3):
        b.x.mul_(1.0 + 0.25 * i).add_(0.125)
        graph.replay()
        torch.cuda.synchronize()
        b.check(2 + i)


def test_two_blocks_on_two_streams():
    a, b = Block(1), Block(2)
    for k in (a, b):
        k.step()
    torch.cuda.synchronize()
    want = [[t.clone() for t in k.outputs()] for k in (a, b)]
    for k in (a, b):
        k.rng[1] = 0
        for t in k.outputs():
            t.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for k, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                k.rng[1] = 0
                k.step()
    torch.cuda.synchronize()
    for k, w in zip((a, b), want):
        for t, v in zip(k.outputs(), w):
            if t is k.y or t is k.x1 or t is k.u1 or t is k.dx or t is k.dy or t is k.dw:
                continue  # behind the experts' sums, whose order is free
            assert torch.equal(t, v)
    a.check(0)
    b.check(0)


@pytest.mark.parametrize("T", [1, 6, 20, 300])
def test_norm_rows_in_8_bits_and_their_product(T):
    # one call right behind the other, each reading what the last has written, many times over
    H, N = 1024, 2064
    torch.manual_seed(T)
    x = (torch.randn(T, H, device="cuda") * 2).bfloat16()
    w, b = (torch.randn(H, device="cuda") * 0.2 + 1).bfloat16(), (torch.randn(H, device="cuda") * 0.1).bfloat16()
    wt = (torch.randn(N, H, device="cuda") * H ** -0.5).bfloat16()
    wq, wscale = torch.empty(N, H, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    fx.flux_q8_quantize(N, H, BF, wt, wq, wscale)
    u, q, s = torch.empty_like(x), torch.empty(T, H, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    out = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    ws = _ws(fx.flux_q8_workspace_size(T, N, H))
    qw, sw = oracle.q8_quantize(wt.double().cpu().numpy())
    assert np.array_equal(wq.cpu().numpy(), qw) and np.array_equal(wscale.cpu().numpy(), sw)
    for i in range(6):
        x.mul_(1.0 + 0.5 * i)
        for _ in range(3):
            x.add_(0.25)
            fx.flux_layer_norm(1, T, H, BF, 0.0, EPS, [x], None, None, w, b, None, [u])
            fx.flux_q8_quantize(T, H, BF, u, q, s)
            fx.flux_q8_gemm(T, N, H, BF, q, s, wq, wscale, None, out, ws)
        torch.cuda.synchronize()
        _, want, _, _, _, mag = oracle.layer_norm(x.double().cpu().numpy(), None, None, w.double().cpu().numpy(),
                                                  b.double().cpu().numpy(), EPS)
        check16(u.double().cpu().numpy(), want, mag, "bf16", what="u")
        qx, sx = oracle.q8_quantize(u.double().cpu().numpy())
        assert np.array_equal(q.cpu().numpy(), qx) and np.array_equal(s.cpu().numpy(), sx)
        want, mag, reach = oracle.q8_gemm(qx, sx, qw, sw, None)
        assert reach < 1 << 24  # the fp32 sums are exact
        check16(out.double().cpu().numpy(), want, mag, "bf16", depth=4, what="out")


def test_router_and_its_losses_right_behind_one_another():
    T, E, k = 3000, 64, 6
    logits = torch.randn(T, E, device="cuda")
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    ws = _ws(fx.flux_moe_balance_workspace_size(T, E, k, 1))
    loss, probs, lse = torch.empty(2, device="cuda"), torch.empty(E, device="cuda"), torch.empty(T, device="cuda")
    counts, tokens = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    for i in range(10):
        logits.mul_(-1.1)
        fx.flux_moe_group_gate(T, E, k, fx.FLUX_SCORE_SOFTMAX, 8, 3, 1, 0, 1.0, logits, None, ids, w)
        fx.flux_moe_balance_loss(T, E, k, 1, 0.1, 0.01, logits, ids, None, loss, counts, probs, tokens, lse, ws)
        want = torch.bincount(ids.view(-1).long(), minlength=E)
        assert torch.equal(counts.long(), want)
