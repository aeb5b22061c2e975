"""GPU parity of the routing with expert groups whose biases are infinite in both signs."""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import reducescatter_tcgen05_tmem_gb300 as fx  # noqa: E402

SCORE = {"softmax": fx.FLUX_SCORE_SOFTMAX, "sigmoid": fx.FLUX_SCORE_SIGMOID}


@pytest.mark.parametrize("E,k,groups,kept", [(16, 2, 8, 3), (64, 8, 8, 3), (48, 4, 16, 6), (256, 8, 8, 4), (95, 5, 5, 2), (512, 8, 16, 4)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("opened", [0, 1, 2])  # groups with finite biases: fewer than are kept
@pytest.mark.parametrize("T", [40, 9800])
def test_infinite_biases(E, k, groups, kept, score, top, opened, T):
    r = np.random.default_rng(E + opened)
    n = E // groups
    z = r.standard_normal((40, E)).astype(np.float32)
    bias = np.full(E, -np.inf, np.float32)
    for g in r.permutation(groups)[:opened]:
        bias[g * n:(g + 1) * n] = (r.standard_normal(n) * 0.05).astype(np.float32)
    bias[(groups - 1) * n] = np.inf        # one of +inf in a group of -inf: its sum counts as -inf
    bias[n // 2] = np.inf if n > 2 else bias[n // 2]
    times = max(T // 40, 1)
    ids, w = torch.empty(times * 40, k, dtype=torch.int32, device="cuda"), torch.empty(times * 40, k, device="cuda")
    fx.flux_moe_group_gate(times * 40, E, k, SCORE[score], groups, kept, top, 1, 1.0, torch.from_numpy(z).cuda().repeat(times, 1),
                           torch.from_numpy(bias).cuda(), ids, w)
    with np.errstate(invalid="ignore"):
        want, _ = oracle.group_gate(z, bias.astype(np.float64), k, score, groups, kept, top, True, 1.0)
    assert (ids.view(times, 40, k).cpu().numpy() == want).all()
