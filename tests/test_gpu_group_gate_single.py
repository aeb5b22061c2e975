"""GPU parity of groups of one expert that are ranked by the sum of two scores: groups whose
64-bit scores are equal are equal in rank, however far apart their logits are."""
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


@pytest.mark.parametrize("E,kept,k", [(2, 1, 1), (4, 2, 1), (8, 3, 3), (8, 5, 4), (7, 5, 3), (16, 9, 4), (32, 9, 9), (31, 30, 20)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("T", [40, 9800])
def test_groups_of_one(E, kept, k, score, top, T):
    r = np.random.default_rng(E)
    z = r.standard_normal((40, E)).astype(np.float32)
    z[0] = 40.0 + np.arange(E)                 # sigmoids of 1, different logits
    z[1] = 36.0 + r.random(E) * 2              # sigmoids of 1 and next to it
    z[2] = -800.0 - np.arange(E)               # sigmoids of 0
    z[3:8] = r.choice(np.array([38, 39, 50, 2, -900, -800], np.float32), (5, E))
    z[8, 1:] = -900.0 + np.arange(E - 1)       # softmax scores of 0 beside one of 1
    z[9] = np.nan
    z[10] = -np.inf
    z[11, E // 2] = np.inf
    z[12, ::2] = np.inf
    z[13, ::2] = -np.inf
    times = max(T // 40, 1)
    n = times * 40
    ids, w = torch.empty(n, k, dtype=torch.int32, device="cuda"), torch.empty(n, k, device="cuda")
    fx.flux_moe_group_gate(n, E, k, SCORE[score], E, kept, top, 0, 1.0, torch.from_numpy(z).cuda().repeat(times, 1), None, ids, w)
    want, want_w = oracle.group_gate(z, None, k, score, E, kept, top, False, 1.0)
    assert (ids.view(times, 40, k).cpu().numpy() == want).all()
    # (arguments up to 1000 round by 1000 ulps of 1; numbers below fp32's least normal one may be 0)
    got = w.view(times, 40, k).double().cpu().numpy()
    check32(got, np.broadcast_to(want_w, got.shape), np.broadcast_to(np.abs(want_w) + 2.0 ** -110, got.shape), depth=2048, what="weights")
