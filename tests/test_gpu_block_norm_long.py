"""The block norms at the most rows that the header allows: 2^31 - 512 of eight columns,
and forward 2^31 - 1."""
import numpy as np
import pytest

import oracle
from tests.rounding import check16, check32
from workloads import gen
from workloads.torch_io import from_device, to_device

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import reducescatter_tcgen05_tmem_gb300 as fx  # noqa: E402

EPS = 1e-5


def test_two_to_the_31_rows():
    T, H, some, more = 2 ** 31 - 512, 8, 700, 511
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB")
    all_x, all_u = (torch.zeros((T + more, H), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    all_rx = torch.empty(T + more, device="cuda")
    x, u, rx = all_x[:T], all_u[:T], all_rx[:T]
    raw = gen.normal16((91, 1), (2 * some, H), 1.0, "bf16")
    x[:some], x[-some:] = to_device(raw[:some], "bf16"), to_device(raw[some:], "bf16")
    fx.flux_block_norm(1, T, H, fx.FLUX_BF16, 0, 0, 0, EPS, [x], None, None, None, None, None, None, [u], None, rx)
    ends = lambda t: torch.cat([t[:some], t[-some:]])  # noqa: E731
    n = oracle.widen(raw, "bf16")
    _, want, _, wrx = oracle.block_norm(n, None, None, None, 1.0, None, EPS)
    check16(oracle.widen(from_device(ends(u)), "bf16"), want, np.abs(want), "bf16", what="u")
    check32(ends(rx).double().cpu().numpy(), wrx, wrx, what="rstd_x")
    assert not bool(u[some:-some].any())
    # 511 rows more, the last of them with values: the rows before keep theirs
    all_x[T + 100:] = 1
    last = u[-some:].clone()
    fx.flux_block_norm(1, T + more, H, fx.FLUX_BF16, 0, 0, 0, EPS, [all_x], None, None, None, None, None, None, [all_u], None, all_rx)
    _, want, _, _ = oracle.block_norm(all_x[-2 * more:].double().cpu().numpy(), None, None, None, 1.0, None, EPS)
    check16(all_u[-2 * more:].double().cpu().numpy(), want, np.abs(want), "bf16", what="u of 2^31 - 1 rows")
    assert torch.equal(u[-some:], last)
    # backward in place: the gradient of u becomes that of x
    rawd = gen.normal16((91, 2), (2 * some, H), 0.1, "bf16")
    u.zero_()
    u[:some], u[-some:] = to_device(rawd[:some], "bf16"), to_device(rawd[some:], "bf16")
    dw = torch.empty(H, device="cuda")
    ws = torch.zeros(fx.flux_block_norm_workspace_size(T, H) // 4, dtype=torch.int32, device="cuda")
    fx.flux_block_norm_bwd(1, T, H, fx.FLUX_BF16, 0, 0, 0, [x], None, None, None, None, None, None, rx, None, [u], [u], None,
                           None, None, None, dw, ws)
    ref = oracle.block_norm_bwd(n, None, None, None, 1.0, None, EPS, None, oracle.widen(rawd, "bf16"))
    check16(oracle.widen(from_device(ends(u)), "bf16"), *ref["dx"], "bf16", what="dx")
    check32(dw.double().cpu().numpy(), *ref["dw_pre"], depth=128 + some, what="dw_pre")
    assert not bool(u[some:-some].any()) and not bool(ws.any())
    del x, u, rx, all_x, all_u, all_rx
    torch.cuda.empty_cache()
