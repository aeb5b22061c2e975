"""8-bit products whose running sums need more than 24 bits: exact up to 8 rows, within the
stated bound of the fp32 sums from 9 rows on."""
import numpy as np
import pytest

import oracle
from tests.rounding import check16

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import reducescatter_tcgen05_tmem_gb300 as fx  # noqa: E402

N = 24


def _codes(pattern, M, K, r):
    """Odd codes from 101 to 127: no partial sum has low bits to spare."""
    x, w = r.integers(50, 64, (M, K)) * 2 + 1, r.integers(50, 64, (N, K)) * 2 + 1
    if pattern == "cancel":  # the second half takes back the first but for some small terms
        h = K // 2
        x[:, h:], w[:, h:] = x[:, :h], -w[:, :h]
        x[:, :3] -= 2 * np.arange(M)[:, None] % 64
    elif pattern == "waves":  # up and down again, eight times
        w[:, (np.arange(K) * 16 // K) % 2 == 1] *= -1
    return x.astype(np.int8), w.astype(np.int8)


@pytest.mark.parametrize("M", [5, 8, 9, 40, 300])
@pytest.mark.parametrize("pattern,K", [("up", 4096), ("up", 28672), ("up", 131056), ("cancel", 28672), ("cancel", 131056),
                                       ("waves", 131056)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_sums_past_24_bits(M, K, pattern, dtype):
    r = np.random.default_rng(K)
    x, w = _codes(pattern, M, K, r)
    steps = np.cumsum((x[0].astype(np.int64) * w[0]).reshape(-1, 16).sum(1))
    assert (steps != steps.astype(np.float32).astype(np.int64)).any(), "fp32 holds every running sum of this input"
    xs = np.full(M, 2.0 ** -8, np.float32)
    ws = np.full(N, 2.0 ** -17 if pattern == "up" else 2.0 ** -9, np.float32)
    cu = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    tdt = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    out = torch.empty(M, N, dtype=tdt, device="cuda")
    ws_ = torch.zeros(fx.flux_q8_workspace_size(M, N, K) // 4, dtype=torch.int32, device="cuda")
    fx.flux_q8_gemm(M, N, K, {"f16": fx.FLUX_F16, "bf16": fx.FLUX_BF16}[dtype], cu(x), cu(xs), cu(w), cu(ws), None, out, ws_)
    torch.cuda.synchronize()
    assert fx.flux_get_status(ws_)[0] == fx.FLUX_OK
    want, mag, _ = oracle.q8_gemm(x, xs, w, ws, None)
    got = out.double().cpu().numpy()
    assert np.abs(want).max() < 65504
    if M <= 8:  # exact integer, rounded to fp32, and two products by powers of two
        check16(got, want, mag, dtype, depth=1)
        return
    # A step adds 16 exact products to the sum, and may cut each of the 17 numbers to the 24 bits of
    # the largest: 17 units of 2^-23 of the magnitudes' sum.  Up to 16 parts of K are added in fp32.
    reach = (np.abs(x.astype(np.float64)) @ np.abs(w.astype(np.float64)).T) * xs[:, None] * ws[None]
    check16(got, want, reach, dtype, depth=17 * 2 * (K // 16 + 1) + 16)
