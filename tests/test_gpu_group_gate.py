"""GPU parity of the routing with expert groups (flux_moe_group_gate,
flux_moe_group_gate_bwd) with its float64 definition, through the C ABI."""
import numpy as np
import pytest

import oracle
from tests.rounding import check32

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import reducescatter_tcgen05_tmem_gb300 as fx  # noqa: E402

SCORE = {"softmax": fx.FLUX_SCORE_SOFTMAX, "sigmoid": fx.FLUX_SCORE_SIGMOID}


class Gate:
    def __init__(self, T, E, k, score, groups=1, kept=1, top=1, renorm=True, scale=1.0, bias=True, seed=0, logits=None):
        r = np.random.default_rng(seed)
        self.args = (T, E, k, SCORE[score], groups, kept, top, int(renorm), scale)
        self.ref = (k, score, groups, kept, top, renorm, scale)
        self.logits = r.standard_normal((T, E)).astype(np.float32) if logits is None else logits
        if bias is True:
            bias = (r.standard_normal(E) * (0.1 if score == "sigmoid" else 0.1 / E)).astype(np.float32)
        self.bias = None if bias is None or bias is False else bias
        self.cu = torch.from_numpy(self.logits).cuda()
        self.cb = None if self.bias is None else torch.from_numpy(self.bias).cuda()
        self.T, self.E, self.k = T, E, k

    def run(self, stream=None):
        ids = torch.full((self.T * self.k + 8,), -7, dtype=torch.int32, device="cuda")
        w = torch.full((self.T * self.k + 8,), 7.0, device="cuda")
        fx.flux_moe_group_gate(*self.args, self.cu, self.cb, ids, w, stream=stream)
        torch.cuda.synchronize()
        assert bool((ids[-8:] == -7).all()) and bool((w[-8:] == 7.0).all())
        n = self.T * self.k
        return ids[:n].view(self.T, self.k).cpu().numpy(), w[:n].view(self.T, self.k).double().cpu().numpy()

    def check(self):
        ids, w = self.run()
        want_ids, want_w = oracle.group_gate(self.logits, None if self.bias is None else self.bias.astype(np.float64), *self.ref)
        assert np.array_equal(ids, want_ids)
        # exponentials, their sum and quotients, the arguments' rounding (up to 20 ulps of scores at most 20)
        check32(w, want_w, np.abs(want_w), depth=128, what="weights")
        self.check_many(want_ids, want_w, 128)
        return ids

    def check_many(self, want_ids, want_w, depth):
        """The same tokens over and over: past 9728 of them a warp takes four at once."""
        if self.T > 9728:
            return
        times = 9800 // self.T + 1
        ids = torch.full((times * self.T * self.k,), -7, dtype=torch.int32, device="cuda")
        w = torch.empty(times * self.T * self.k, device="cuda")
        fx.flux_moe_group_gate(times * self.T, *self.args[1:], self.cu.repeat(times, 1), self.cb, ids, w)
        ids, w = ids.view(times, self.T, self.k).cpu().numpy(), w.view(times, self.T, self.k).double().cpu().numpy()
        assert (ids == want_ids).all()
        check32(w, np.broadcast_to(want_w, w.shape), np.broadcast_to(np.abs(want_w), w.shape), depth=depth, what="weights")


CASES = [
    # T, E, k, score, groups, kept, top, renorm, scale, bias
    (1, 1, 1, "sigmoid", 1, 1, 1, True, 1.0, True),
    (5, 2, 1, "softmax", 2, 1, 1, False, 1.0, True),
    (13, 256, 8, "sigmoid", 8, 4, 2, True, 2.5, True),
    (1000, 256, 8, "sigmoid", 8, 4, 2, True, 2.5, True),
    (333, 256, 8, "softmax", 8, 3, 1, False, 16.0, False),
    (77, 160, 6, "softmax", 8, 3, 1, False, 1.0, True),
    (100, 64, 6, "softmax", 8, 3, 2, True, 1.0, False),
    (100, 64, 64, "sigmoid", 1, 1, 1, True, 1.0, True),     # every expert
    (50, 63, 5, "sigmoid", 9, 2, 2, False, 1.0, True),      # odd sizes
    (50, 33, 3, "softmax", 11, 4, 2, True, 1.0, True),
    (41, 7, 3, "softmax", 7, 5, 2, True, 1.0, True),        # groups of one
    (41, 96, 4, "sigmoid", 32, 7, 2, True, 1.0, True),      # more groups than lanes of a token... of 64 experts
    (19, 64, 4, "sigmoid", 32, 9, 2, True, 1.0, True),
    (29, 1024, 16, "sigmoid", 16, 16, 1, True, 1.0, True),
    (29, 1020, 9, "sigmoid", 30, 29, 2, True, 1.0, True),   # groups of 34: more than 1024 places
    (29, 1023, 40, "softmax", 31, 31, 1, False, 1.0, True),
    (29, 1023, 33, "softmax", 31, 30, 2, True, 1.0, False),
    (29, 999, 12, "sigmoid", 27, 5, 2, True, 1.0, True),
    (9800, 48, 4, "sigmoid", 16, 6, 2, True, 1.0, True),    # long batches of few experts
    (9800, 60, 5, "softmax", 5, 2, 2, True, 1.0, True),
    (9800, 16, 10, "softmax", 1, 1, 1, False, 1.0, False),
    (9800, 64, 33, "sigmoid", 32, 21, 1, True, 1.0, True),
    (9800, 7, 3, "sigmoid", 7, 5, 2, True, 1.0, True),
    (9800, 24, 4, "softmax", 8, 3, 2, False, 1.0, True),
    (29, 1024, 40, "softmax", 32, 11, 2, False, 1.0, True),
    (64, 1021, 33, "softmax", 1, 1, 1, True, 1.0, True),    # prime
    (300, 384, 8, "sigmoid", 1, 1, 1, True, 2.5, True),
    (4099, 8, 2, "softmax", 1, 1, 1, True, 1.0, False),
    (129, 128, 8, "sigmoid", 4, 2, 2, True, 1.0, False),    # ranks of scores, choice of logits
    (129, 66, 8, "sigmoid", 2, 1, 1, True, 1.0, False),
    # eight lanes a token: every number of scores a lane, groups of 1, 2, 4 and 8 lanes
    (70, 24, 5, "sigmoid", 2, 1, 2, True, 1.0, True),
    (70, 40, 8, "softmax", 4, 3, 2, False, 1.0, True),
    (70, 104, 7, "sigmoid", 1, 1, 1, False, 1.0, True),
    (70, 121, 8, "softmax", 1, 1, 1, True, 1.0, True),
    (70, 256, 1, "sigmoid", 2, 1, 1, True, 1.0, False),
    (70, 200, 8, "softmax", 8, 5, 2, False, 2.0, False),
    # one warp a token
    (70, 256, 9, "sigmoid", 8, 4, 2, True, 1.0, True),
    (70, 256, 12, "softmax", 1, 1, 1, False, 1.0, True),
    (70, 260, 8, "sigmoid", 1, 1, 1, True, 1.0, True),
    (70, 128, 10, "softmax", 2, 1, 1, True, 1.0, False),
    (70, 512, 8, "softmax", 16, 5, 2, True, 1.0, True),
    # rows that begin off 16 bytes, more than 64 experts
    (33, 95, 9, "sigmoid", 5, 3, 2, True, 1.0, True),
    (33, 250, 20, "softmax", 1, 1, 1, True, 1.0, True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_choice_and_weights(case):
    Gate(*case, seed=3).check()


def test_as_the_plain_gate():
    g = Gate(500, 40, 4, "softmax", bias=None, seed=5)
    ids, w = g.run()
    i2, w2 = torch.empty(500, 4, dtype=torch.int32, device="cuda"), torch.empty(500, 4, device="cuda")
    fx.flux_moe_topk_gate(500, 40, 4, g.cu, i2, w2)
    assert np.array_equal(ids, i2.cpu().numpy())
    np.testing.assert_allclose(w, w2.cpu().numpy(), rtol=1e-6)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,kept,top", [(1, 1, 1), (8, 3, 1), (8, 3, 2)])
@pytest.mark.parametrize("E", [64, 256])
def test_values_closer_than_fp32(score, groups, kept, top, E):
    # biases that bring every s + bias to within 2^-25 of one value: only 64 bits order them
    r = np.random.default_rng(8)
    row = r.standard_normal(E).astype(np.float32)
    s = oracle.gate_scores(row[None], score)[0]
    bias = (0.75 - s).astype(np.float32)
    logits = np.tile(row, (37, 1))
    logits[1::2] = r.standard_normal((18, E))
    c = s + bias
    assert np.unique(np.sort(c)).size > E // 2 and np.ptp(c) < 2.0 ** -23
    Gate(37, E, 6, score, groups, kept, top, True, 1.0, bias=bias, logits=logits).check()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,kept", [(8, 1, 1), (40, 1, 1), (64, 8, 3), (100, 4, 2), (255, 1, 1), (256, 8, 4), (256, 2, 1),
                                           (512, 1, 1)])
def test_two_neighbours_closer_than_fp32(score, E, groups, kept):
    # two experts whose s + bias are equal to 2^-24 or so in every token, anywhere in the order:
    # both in, both out, or one in and one out
    r = np.random.default_rng(E + groups)
    T, k = 600, min(4, E // groups * kept)
    logits = r.standard_normal((T, E)).astype(np.float32)
    bias = (r.standard_normal(E) * 0.05).astype(np.float32)
    pairs = [(0, E - 1), (1, 2), (E // 2, 3), (E // 2 + 1, E // 2 + 2)]
    if score == "softmax":  # the same sum in every token: permuted rows of one
        base = logits[0].copy()
        for t in range(T):
            logits[t] = base
            rest = np.setdiff1d(np.arange(E), np.array(pairs).ravel())
            logits[t, rest] = base[r.permutation(rest)]
    else:
        logits[:, np.array(pairs).ravel()] = r.standard_normal(8).astype(np.float32) + 1.0
    s = oracle.gate_scores(logits[:1], score)[0]
    for a, b in pairs:
        bias[b] = np.float32(s[a] + np.float64(bias[a]) - s[b])
    c = s + bias.astype(np.float64)
    assert all(0 < abs(c[a] - c[b]) < 2.0 ** -23 for a, b in pairs)
    for top in (1, 2):
        Gate(T, E, k, score, groups, kept, top, True, 1.0, bias=bias, logits=logits).check()


@pytest.mark.parametrize("E,groups", [(64, 8), (256, 8), (256, 4), (96, 3), (512, 16)])
@pytest.mark.parametrize("top", [1, 2])
def test_two_groups_closer_than_fp32(E, groups, top):
    # two groups whose ranks are equal to 2^-23 or so in every token, inside, outside and on the border
    r = np.random.default_rng(E + groups + top)
    n, T = E // groups, 200
    logits = (r.standard_normal((T, E)) * 0.5 - 1.0).astype(np.float32)
    bias = (r.standard_normal(E) * 0.02).astype(np.float32)
    a, b = 1, groups - 1  # the groups; their two largest are the same in every token
    lead = [a * n + 1, a * n + 2, b * n, b * n + 3]
    logits[:, lead] = np.array([2.0, 1.5, 1.75, 1.25], np.float32)
    logits[::5, b * n + 5] = 1.25  # a third beside the second
    s = oracle.gate_scores(logits[:1], "sigmoid")[0]
    c = s + bias.astype(np.float64)
    if top == 1:
        bias[lead[2]] = np.float32(c[lead[0]] - s[lead[2]])
    else:
        bias[lead[3]] = np.float32(c[lead[0]] + c[lead[1]] - c[lead[2]] - s[lead[3]])
    for t in range(T):  # other groups above and below them
        for g in range(groups):
            if g not in (a, b) and r.random() < 0.5:
                logits[t, g * n:g * n + 2] = 3.0 + r.random(2)
    for kept in sorted({1, 2, groups // 2, groups - 1}):
        Gate(T, E, min(5, n * kept), "sigmoid", groups, kept, top, True, 1.0, bias=bias, logits=logits).check()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups", [(64, 8), (60, 5), (95, 5), (256, 8), (256, 4), (512, 16)])
@pytest.mark.parametrize("scale", [1.0, 16.0])
def test_two_sums_of_scores_closer_than_fp32(score, E, groups, scale):
    # no bias: two groups' sums of two scores within some 2^-24 of each other, the last in and the first out
    r = np.random.default_rng(E + groups)
    n, T = E // groups, 400
    logits = (r.standard_normal((T, E)) - 4.0).astype(np.float32)
    a, b = r.permutation(groups)[:2]
    f = (lambda x: np.exp(x)) if score == "softmax" else (lambda x: 1.0 / (1.0 + np.exp(-x)))
    back = np.log if score == "softmax" else (lambda y: -np.log(1.0 / y - 1.0))
    logits[:, a * n], logits[:, a * n + 1], logits[:, b * n + 1] = 0.5, 0.0, 0.25
    x = np.float32(back(f(0.5) + f(0.0) - f(0.25)))
    logits[:, b * n] = x + np.spacing(x) * r.integers(-6, 7, T).astype(np.float32)
    if scale > 1.0:  # one group far above the others: their scores are small beside the sum
        top = [g for g in range(groups) if g not in (a, b)][0]
        logits[:, top * n] = scale
    ids = Gate(T, E, 2, score, groups, 1 if scale == 1.0 else 2, 2, bias=None, logits=logits).check()
    assert {a, b} <= set(np.unique(ids // n)) or scale > 1.0


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", ["zero", "own", None])
@pytest.mark.parametrize("groups,kept,top", [(1, 1, 1), (8, 2, 1), (8, 2, 2)])
def test_equal_scores(score, bias, groups, kept, top):
    # scores of a 16-bit router: many are equal; then rows that are equal throughout
    r = np.random.default_rng(9)
    logits = (np.round(r.standard_normal((200, 128)) * 8) / 8).astype(np.float32)
    logits[::10] = 0.0
    logits[5] = -0.0
    logits[6, ::2] = -0.0
    logits[6, 1::2] = 0.0
    b = {"zero": np.zeros(128, np.float32), "own": (r.standard_normal(128) * 1e-3).astype(np.float32), None: None}[bias]
    Gate(200, 128, 9, score, groups, kept, top, True, 1.0, bias=b, logits=logits).check()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("groups,kept", [(1, 1), (4, 2)])
@pytest.mark.parametrize("pad", [0, 64])
def test_odd_rows(score, renorm, bias, groups, kept, pad):
    r = np.random.default_rng(10)
    z = r.standard_normal((14, 32)).astype(np.float32)
    z[0] = np.nan
    z[1] = -np.inf
    z[2, 3] = np.inf
    z[3, [5, 9]] = np.inf
    z[4, ::3] = np.nan
    z[5, 1:] = -np.inf
    z[6] = -200.0 - np.arange(32)     # sigmoids below fp32's least number still have shares
    z[7] = 100.0 + np.arange(32)      # sigmoids of 1
    z[8] = 1e30
    z[9] = -3e38
    z[10, 0] = 3e38
    z[11] = 45.0                      # equal 64-bit sigmoids from equal and from unequal scores
    z[12] = 40.0 + np.arange(32) % 3
    if pad:  # wide rows: what was every score of a row is every score still
        z = np.concatenate([z, z, z], axis=1)
    g = Gate(14, z.shape[1], 4, score, groups, kept, 2, renorm, 1.5, bias=bias, logits=z)
    ids, w = g.run()
    want_ids, want_w = oracle.group_gate(z, None if g.bias is None else g.bias.astype(np.float64), *g.ref)
    assert np.array_equal(ids, want_ids)
    check32(w, want_w, np.abs(want_w), depth=1024, what="weights")  # arguments up to 200 round by 200 ulps of 1
    if pad:
        g.check_many(want_ids, want_w, 1024)


@pytest.mark.parametrize("E,groups,kept", [(64, 8, 4), (16, 8, 3), (32, 4, 2), (60, 5, 2), (95, 5, 2), (96, 3, 1), (256, 8, 4), (256, 2, 1), (512, 16, 4)])
@pytest.mark.parametrize("top", [1, 2])
def test_biases_whose_sums_pass_fp32(E, groups, kept, top):
    """A rank that is a sum of two may be infinite in fp32; in doubles it is not."""
    r = np.random.default_rng(E + top)
    bias = r.uniform(1.8e38, 3.3e38, E).astype(np.float32)
    Gate(40, E, 2, "sigmoid", groups, kept, top, bias=bias, seed=E).check()
    Gate(40, E, 2, "sigmoid", groups, kept, top, bias=-bias, seed=E).check()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,kept,open_groups", [(64, 8, 4, 2), (16, 8, 3, 1), (60, 5, 2, 1), (95, 5, 2, 1), (256, 8, 4, 3), (512, 16, 4, 2)])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("low", [-np.inf, float(np.finfo(np.float32).min)])
def test_masked_groups(score, E, groups, kept, open_groups, top, low):
    """Fewer groups than are kept have experts that are not masked; a masked one is never chosen."""
    r = np.random.default_rng(E + kept + top)
    n = E // groups
    bias = (r.standard_normal(E) * 0.01).astype(np.float32)
    closed = r.permutation(groups)[open_groups:]
    for g in closed:
        bias[g * n:(g + 1) * n] = low
    ids = Gate(40, E, 2, score, groups, kept, top, bias=bias, seed=E).check()
    assert not np.isin(ids // n, closed).any()


def test_infinite_bias():
    b = np.zeros(64, np.float32)
    b[::3] = -np.inf  # experts that are switched off
    b[7] = np.inf
    ids = Gate(100, 64, 8, "sigmoid", bias=b, seed=12).check()
    assert (ids[:, 0] == 7).all() and not np.isin(ids[ids != 7] % 3, 0).any()
    Gate(20, 64, 40, "sigmoid", bias=b, seed=13).check()  # some of them have to be taken


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c))
@pytest.mark.parametrize("accumulate", [0, 1])
def test_backward(case, accumulate):
    g = Gate(*case, seed=4)
    ids, _ = g.run()
    T, E, k = g.T, g.E, g.k
    r = np.random.default_rng(1)
    dw = r.standard_normal((T, k)).astype(np.float32)
    before = r.standard_normal((T, E)).astype(np.float32)
    buf = torch.full((T * E + 8,), 3.0, device="cuda")
    buf[:T * E] = torch.from_numpy(before).cuda().view(-1) if accumulate else float("nan")
    fx.flux_moe_group_gate_bwd(T, E, k, g.args[3], g.args[7], g.args[8], g.cu, torch.from_numpy(ids).cuda(),
                               torch.from_numpy(dw).cuda(), accumulate, buf)
    want, mag = oracle.group_gate_bwd(g.logits, ids, dw.astype(np.float64), case[3], case[7], case[8])
    got = buf[:T * E].view(T, E).double().cpu().numpy()
    assert bool((buf[T * E:] == 3.0).all())
    if accumulate:
        check32(got, want + before, mag + np.abs(before) / 64, depth=128, what="dlogits")
    else:
        check32(got, want, mag, depth=128, what="dlogits")


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [0, 1])
def test_backward_of_odd_rows(score, renorm):
    z = np.random.default_rng(3).standard_normal((9, 16)).astype(np.float32)
    z[0] = np.nan
    z[1] = -np.inf
    z[2, 3] = np.inf
    z[3] = -200.0 - np.arange(16)
    z[4] = 100.0 + np.arange(16)
    z[5, 2:] = -np.inf
    ids, _ = oracle.group_gate(z, None, 3, score, 1, 1, 1, bool(renorm), 1.0)
    ids[6, 1] = -1
    ids[7, 0] = 16
    dw = np.random.default_rng(4).standard_normal((9, 3)).astype(np.float32)
    dl = torch.full((9, 16), float("nan"), device="cuda")
    fx.flux_moe_group_gate_bwd(9, 16, 3, SCORE[score], renorm, 1.0, torch.from_numpy(z).cuda(), torch.from_numpy(ids).cuda(),
                               torch.from_numpy(dw).cuda(), 0, dl)
    want, mag = oracle.group_gate_bwd(z, ids, dw.astype(np.float64), score, bool(renorm), 1.0)
    # (numbers below fp32's least normal one may be 0)
    check32(dl.double().cpu().numpy(), want, mag + 2.0 ** -100, depth=1024, what="dlogits")


def test_dot_of_zero():
    # the chosen experts' terms cancel: the sum over them is 0
    z = np.zeros((1, 8), np.float32)
    ids = np.array([[0, 1]], np.int32)
    dw = np.array([[1.0, -1.0]], np.float32)
    dl = torch.empty(1, 8, device="cuda")
    fx.flux_moe_group_gate_bwd(1, 8, 2, fx.FLUX_SCORE_SOFTMAX, 0, 1.0, torch.from_numpy(z).cuda(), torch.from_numpy(ids).cuda(),
                               torch.from_numpy(dw).cuda(), 0, dl)
    np.testing.assert_allclose(dl.cpu().numpy(), [[0.125, -0.125] + [0.0] * 6], rtol=1e-6)


def test_sum_with_the_router_losses():
    # the balance loss's gradient, then the gate's added to it
    T, E, k = 300, 32, 4
    g = Gate(T, E, k, "softmax", bias=None, seed=6)
    ids, w = g.run()
    cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    i, wt = cu(ids), cu(w.astype(np.float32))
    ws = torch.zeros(max(64, fx.flux_moe_balance_workspace_size(T, E, k, 1) // 4), dtype=torch.int32, device="cuda")
    loss, probs, lse = torch.empty(2, device="cuda"), torch.empty(E, device="cuda"), torch.empty(T, device="cuda")
    counts, tokens = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    fx.flux_moe_balance_loss(T, E, k, 1, 0.1, 0.01, g.cu, i, None, loss, counts, probs, tokens, lse, ws)
    dw = torch.randn(T, k, device="cuda")
    a, b = torch.empty(T, E, device="cuda"), torch.empty(T, E, device="cuda")
    fx.flux_moe_router_bwd(T, E, k, 1, 0.1, 0.01, g.cu, i, wt, None, lse, counts, tokens, None, dw, a)
    fx.flux_moe_router_bwd(T, E, k, 1, 0.1, 0.01, g.cu, i, None, None, lse, counts, tokens, None, None, b)
    fx.flux_moe_group_gate_bwd(T, E, k, fx.FLUX_SCORE_SOFTMAX, 1, 1.0, g.cu, i, dw, 1, b)
    assert float((a - b).abs().max()) < 1e-5 * float(a.abs().max())


def test_long_batch_repeats():
    g = Gate(70001, 256, 8, "sigmoid", 8, 4, 2, True, 2.5, seed=20)
    a = g.run()
    side = torch.cuda.Stream()
    b = g.run(stream=side)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    rows = np.random.default_rng(0).integers(0, 70001, 500)
    ids, w = oracle.group_gate(g.logits[rows], g.bias.astype(np.float64), *g.ref)
    assert np.array_equal(a[0][rows], ids)
    check32(a[1][rows], w, np.abs(w), depth=128)
