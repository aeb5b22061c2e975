"""Gradient of the grouped routing's scores where slots have no expert (ids outside [0, E)):
they add nothing, whatever their weight's gradient holds."""
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


@pytest.mark.parametrize("E,k", [(8, 2), (16, 3), (33, 4), (64, 8), (64, 20), (256, 8), (250, 40), (1024, 16)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("accumulate", [0, 1])
def test_slots_without_an_expert(E, k, score, renorm, accumulate):
    T = 37
    r = np.random.default_rng(E * k)
    z = r.standard_normal((T, E)).astype(np.float32)
    ids, _ = oracle.group_gate(z, None, k, score, 1, 1, 1, bool(renorm), 1.0)
    dw = r.standard_normal((T, k)).astype(np.float32)
    out = r.random((T, k)) < 0.4
    out[0], out[1] = True, False
    ids[out] = r.choice(np.array([-1, -5, E, E + 3, 2 ** 31 - 1, -2 ** 31], np.int64), out.sum()).astype(np.int32)
    bad = np.where(out, r.choice(np.array([np.nan, np.inf, -np.inf], np.float32), (T, k)), dw)
    before = r.standard_normal((T, E)).astype(np.float32)
    dl = torch.from_numpy(before).cuda() if accumulate else torch.full((T, E), float("nan"), device="cuda")
    cu = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    fx.flux_moe_group_gate_bwd(T, E, k, SCORE[score], renorm, 2.5, cu(z), cu(ids), cu(bad), accumulate, dl)
    want, mag = oracle.group_gate_bwd(z, ids, dw.astype(np.float64), score, bool(renorm), 2.5)
    if accumulate:
        want, mag = want + before, mag + np.abs(before) / 64
    check32(dl.double().cpu().numpy(), want, mag, depth=128, what="dlogits")
