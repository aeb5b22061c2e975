"""Backward pass of the layer norm on rows far from zero and hardly any spread, whose mean
times 1 / deviation passes fp32: lanes past the row's end must not see it."""
import numpy as np
import pytest

import oracle
from tests.rounding import check16, check32

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import reducescatter_tcgen05_tmem_gb300 as fx  # noqa: E402


@pytest.mark.parametrize("H", [64, 264, 520, 1032, 1544, 2056, 4104, 6152, 8200, 12296])
def test_mean_times_rstd_past_fp32(H):
    T = 5
    g = torch.Generator().manual_seed(H)
    x = torch.full((T, H), 2.0 ** 119, dtype=torch.bfloat16)  # every row one number, 6.6e35
    x[1] = -(2.0 ** 120)
    x[2] = torch.randn(H, generator=g).bfloat16()             # an ordinary one between them
    du = (torch.randn(T, H, generator=g) * 0.05).bfloat16()
    w = (torch.randn(H, generator=g) * 0.2 + 1).bfloat16()
    m = x.double().mean(1).float()
    r = (x.double().var(1, unbiased=False) + 1e-8).rsqrt().float()  # 1e4 for the constant rows
    assert torch.isinf(m[0] * r[0]) and bool((x[0].float() == m[0]).all())
    c = [t.cuda() for t in (x, du, w, m, r)]
    dx, dw, db = torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    ws = torch.zeros(fx.flux_layer_norm_workspace_size(T, H) // 4, dtype=torch.int32, device="cuda")
    fx.flux_layer_norm_bwd(1, T, H, fx.FLUX_BF16, 0.0, [c[0]], None, c[2], c[3], c[4], None, [c[1]], [dx], None, dw, db, ws)
    n = lambda t: t.double().cpu().numpy()  # noqa: E731
    want = oracle.layer_norm_bwd(n(x), n(m), n(r), n(w), None, n(du), None)
    # the constant rows' n is exactly 0: magnitudes by the differences from the mean, not by the mean
    small = n(x) - n(m)[:, None]
    mag = oracle.layer_norm_bwd(np.abs(small) + (np.abs(n(m)) * (np.arange(T) == 2))[:, None], 0 * n(m), n(r), n(w), None, n(du), None)
    check16(n(dx), want["dx"][0], mag["dx"][1], "bf16", what="dx")
    check32(n(dw), want["dw"][0], mag["dw"][1], what="dw")
    check32(n(db), want["db"][0], mag["db"][1], what="db")
