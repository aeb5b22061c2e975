"""GPU parity of the routing with expert groups where some groups or experts are masked with
very low biases (or lifted by very high ones) and others' ranks are closer than fp32 tells."""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import reducescatter_tcgen05_tmem_gb300 as fx  # noqa: E402

SCORE = {"softmax": fx.FLUX_SCORE_SOFTMAX, "sigmoid": fx.FLUX_SCORE_SIGMOID}
LOW = float(np.finfo(np.float32).min)


@pytest.mark.parametrize("E,groups,kept,k", [(16, 8, 3, 4), (64, 8, 3, 8), (48, 16, 5, 4), (60, 5, 2, 5), (95, 5, 2, 5), (256, 8, 4, 8), (256, 4, 2, 8),
                                             (512, 16, 4, 8)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("T", [64, 9856])
def test_masked_and_close_groups(E, groups, kept, k, score, top, T):
    r = np.random.default_rng(E + groups + top)
    n = E // groups
    for trial in range(10):
        z = (r.standard_normal((64, E)) * 0.5 - 1.0).astype(np.float32)
        bias = (r.standard_normal(E) * 0.02).astype(np.float32)
        a, b, *rest = r.permutation(groups)
        # two groups with equal scores in every token (permuted rows of one for the softmax's sum)
        lead = [a * n, a * n + 1, b * n, b * n + n - 1]
        z[:] = z[0]
        other = np.setdiff1d(np.arange(E), lead)
        for t in range(64):
            z[t, other] = z[0, r.permutation(other)]
        z[:, lead] = np.array([2.0, 1.5, 1.75, 1.25], np.float32)
        s = oracle.gate_scores(z[:1], score)[0]
        c = s + bias.astype(np.float64)
        if top == 1:
            bias[lead[2]] = np.float32(c[lead[0]] - s[lead[2]])
        else:
            bias[lead[3]] = np.float32(c[lead[0]] + c[lead[1]] - c[lead[2]] - s[lead[3]])
        for g, kind in zip(rest, r.integers(0, 8, len(rest))):
            mine = slice(g * n, (g + 1) * n)
            if kind == 0:
                bias[mine] = LOW
            elif kind == 1:
                bias[mine] = -np.inf
            elif kind == 2:
                bias[mine] = r.uniform(-3.4e38, -1e38, n)
            elif kind == 3:
                bias[mine] = -1e9
            elif kind == 4:
                bias[mine.start + 1:mine.stop] = LOW  # one expert is open
            elif kind == 5 and trial % 2:
                bias[mine] = 1e30
            elif kind == 6 and trial % 3 == 0:
                bias[mine] = r.uniform(1.8e38, 3.4e38, n)
        times = T // 64
        ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
        fx.flux_moe_group_gate(T, E, k, SCORE[score], groups, kept, top, 1, 1.0, torch.from_numpy(z).cuda().repeat(times, 1),
                               torch.from_numpy(bias).cuda(), ids, w)
        want, _ = oracle.group_gate(z, bias.astype(np.float64), k, score, groups, kept, top, True, 1.0)
        assert (ids.view(times, 64, k).cpu().numpy() == want).all(), trial
