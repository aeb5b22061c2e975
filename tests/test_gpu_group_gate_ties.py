"""GPU parity of the routing with expert groups where scores are equal and every
candidate is chosen: no round of the choice may be left without an expert."""
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


# E, topk, groups, kept: topk is all of the kept groups' experts
@pytest.mark.parametrize("E,k,groups,kept", [(1, 1, 1, 1), (2, 2, 1, 1), (8, 8, 1, 1), (7, 7, 1, 1), (16, 8, 8, 4), (64, 8, 8, 1),
                                             (64, 64, 1, 1), (60, 24, 5, 2), (96, 6, 32, 2), (256, 8, 32, 1), (256, 64, 8, 2),
                                             (250, 250, 1, 1), (512, 32, 16, 1), (1024, 1024, 1, 1), (1020, 34, 30, 1)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("T", [30, 9800])  # a warp a token, or (up to 256 experts) eight lanes a token
def test_every_candidate_chosen_with_ties(E, k, groups, kept, score, biased, T):
    if T == 9800 and E > 256:
        pytest.skip("one form for batches of all lengths")
    r = np.random.default_rng(E + k)
    z = (np.round(r.standard_normal((30, E)) * 2) / 2).astype(np.float32)
    z[0] = 0.0                       # a router whose weights are zero
    z[1] = -np.inf
    z[2:6] = z[2:6, :1]              # one score throughout
    z[6, ::2] = z[6, 0]
    z[7, -2:] = z[7, -1]
    z[8, :2] = z[8, 0]
    bias = (np.round(r.standard_normal(E)) / 64).astype(np.float32) if biased else None
    times = T // 30 + 1 if T > 30 else 1
    cu = torch.from_numpy(z).cuda().repeat(times, 1)
    n = times * 30
    ids = torch.full((n * k + 8,), -7, dtype=torch.int32, device="cuda")
    w = torch.full((n * k + 8,), 7.0, device="cuda")
    fx.flux_moe_group_gate(n, E, k, SCORE[score], groups, kept, 1, 1, 1.0, cu, None if bias is None else torch.from_numpy(bias).cuda(), ids, w)
    torch.cuda.synchronize()
    assert bool((ids[-8:] == -7).all()) and bool((w[-8:] == 7.0).all())
    want, want_w = oracle.group_gate(z, None if bias is None else bias.astype(np.float64), k, score, groups, kept, 1, True, 1.0)
    got = ids[:n * k].view(times, 30, k).cpu().numpy()
    assert (got == want).all()
    w = w[:n * k].view(times, 30, k).double().cpu().numpy()
    check32(w, np.broadcast_to(want_w, w.shape), np.broadcast_to(np.abs(want_w), w.shape), depth=128 + k, what="weights")
