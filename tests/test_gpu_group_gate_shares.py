"""GPU parity of renormalised sigmoid weights whose logits lie far apart: a share that fp32
holds is not lost, whichever form of the kernel a batch takes, and the gradient has it too."""
import numpy as np
import pytest

import oracle
from tests.rounding import check32

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import reducescatter_tcgen05_tmem_gb300 as fx  # noqa: E402


@pytest.mark.parametrize("E,k,groups,kept", [(8, 4, 1, 1), (48, 4, 16, 6), (64, 12, 1, 1), (256, 8, 8, 4), (250, 20, 1, 1), (512, 8, 16, 4)])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T", [30, 9810])
def test_low_shares(E, k, groups, kept, biased, renorm, T):
    r = np.random.default_rng(E + k)
    z = np.full((30, E), -300.0, np.float32) - r.random((30, E)).astype(np.float32)
    for t in range(30):  # the chosen ones: a largest from -80 to 10, the others down to 100 below it
        n = E // groups
        own = np.concatenate([np.arange(g * n, (g + 1) * n) for g in r.permutation(groups)[:kept]])
        at = r.permutation(own)[:k]
        peak = np.linspace(-80, 10, 30)[t]
        z[t, at] = (peak - np.sort(r.random(k)) * np.array([100.0, 60.0, 27.0])[t % 3]).astype(np.float32)
        z[t, at[0]] = peak
    z[0, :4] = [-60, -88, -95, -100]
    bias = np.zeros(E, np.float32) if biased else None
    times = max(T // 30, 1)
    n = times * 30
    ids, w = torch.empty(n, k, dtype=torch.int32, device="cuda"), torch.empty(n, k, device="cuda")
    cu = torch.from_numpy(z).cuda()
    fx.flux_moe_group_gate(n, E, k, fx.FLUX_SCORE_SIGMOID, groups, kept, 1, int(renorm), 1.0, cu.repeat(times, 1),
                           None if bias is None else torch.from_numpy(bias).cuda(), ids, w)
    want_ids, want = oracle.group_gate(z, None if bias is None else bias.astype(np.float64), k, "sigmoid", groups, kept, 1, renorm, 1.0)
    assert (ids.view(times, 30, k).cpu().numpy() == want_ids).all()
    got = w.view(times, 30, k).double().cpu().numpy()
    # an argument of up to 300 is rounded by 2^-24 of itself, which scales its exponential by as
    # much; below fp32's least normal number (2^-126) a weight may lose bits or be 0
    mag = np.abs(want) + 2.0 ** -126 / (512 * 2.0 ** -24)
    check32(got, np.broadcast_to(want, got.shape), np.broadcast_to(mag, got.shape), depth=512, what="weights")
    assert (got[:, want > 2.0 ** -125] > 0).all()
