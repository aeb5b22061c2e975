"""GPU parity of the routing with expert groups where the bias holds NaN (a training run
that diverged): each counts as -inf, in every form of the kernel."""
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


@pytest.mark.parametrize("E,k,groups,kept,top", [(8, 2, 1, 1, 1), (16, 8, 1, 1, 1), (48, 4, 16, 6, 2), (64, 8, 8, 3, 2), (64, 20, 1, 1, 1),
                                                 (256, 8, 8, 4, 2), (256, 8, 8, 4, 1), (250, 20, 1, 1, 1), (512, 8, 16, 4, 2)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("which", ["one", "heads", "group", "most", "all"])
@pytest.mark.parametrize("T", [40, 9800])
def test_nan_in_the_bias(E, k, groups, kept, top, score, which, T):
    r = np.random.default_rng(E + k)
    z = r.standard_normal((40, E)).astype(np.float32)
    z[0] = 0.0
    z[1, ::3] = np.nan
    bias = (r.standard_normal(E) * 0.05).astype(np.float32)
    nan = {"one": [E // 2], "heads": range(0, E, 4), "group": range(E // groups), "most": range(k - 1, E), "all": range(E)}[which]
    bias[list(nan)] = np.nan
    times = max(T // 40, 1)
    n = times * 40
    ids = torch.full((n * k + 8,), -7, dtype=torch.int32, device="cuda")
    w = torch.full((n * k + 8,), 7.0, device="cuda")
    fx.flux_moe_group_gate(n, E, k, SCORE[score], groups, kept, top, 0, 1.0, torch.from_numpy(z).cuda().repeat(times, 1),
                           torch.from_numpy(bias).cuda(), ids, w)
    torch.cuda.synchronize()
    assert bool((ids[-8:] == -7).all()) and bool((w[-8:] == 7.0).all())
    want, want_w = oracle.group_gate(z, bias.astype(np.float64), k, score, groups, kept, top, False, 1.0)
    assert (ids[:n * k].view(times, 40, k).cpu().numpy() == want).all()
    w = w[:n * k].view(times, 40, k).double().cpu().numpy()
    check32(w, np.broadcast_to(want_w, w.shape), np.broadcast_to(np.abs(want_w), w.shape), depth=128, what="weights")
