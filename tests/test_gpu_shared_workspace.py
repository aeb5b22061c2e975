"""One workspace for the operators that need zeros in its first 256 bytes only, behind an
8-bit product of many rows, which leaves its widened tokens and partial sums in it."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import reducescatter_tcgen05_tmem_gb300 as fx  # noqa: E402

BF = fx.FLUX_BF16


def test_calls_behind_an_8_bit_product():
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    e = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    M, N, K, T, H, E, k = 300, 520, 4096, 700, 1032, 32, 4
    xq = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    wq = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    xs, wsc = e(M).fill_(0.01), e(N).fill_(0.001)
    x, du, dx1, w = n(T, H).bfloat16(), n(T, H).bfloat16(), n(T, H).bfloat16(), n(H).bfloat16()
    m, r = x.float().mean(1), (x.float().var(1, unbiased=False) + 1e-5).rsqrt()
    logits = n(T, E)
    ids, wt = e(T, k, dt=torch.int32), e(T, k)
    fx.flux_moe_group_gate(T, E, k, fx.FLUX_SCORE_SOFTMAX, 1, 1, 1, 1, 1.0, logits, None, ids, wt)
    q2, sc2, y = e(fx.flux_w4_weight_bytes(1, K, 512), dt=torch.uint8), e(K // 64, 512, dt=torch.bfloat16), e(6, 512, dt=torch.bfloat16)
    w4 = n(K, 512).bfloat16()
    fx.flux_w4_quantize(1, K, 512, 64, BF, w4, q2, sc2)
    a4 = n(6, K).bfloat16()

    def step(ws):
        out = [e(M, N, dt=torch.bfloat16), e(8, N, dt=torch.bfloat16), e(T, H, dt=torch.bfloat16), e(H), e(H), e(2), e(E, dt=torch.int32),
               torch.empty_like(y)]
        for _ in range(2):
            fx.flux_q8_gemm(M, N, K, BF, xq, xs, wq, wsc, None, out[0], ws())
            fx.flux_layer_norm_bwd(1, T, H, BF, 0.0, [x], None, w, m, r, [dx1], [du], [out[2]], None, out[3], out[4], ws())
            fx.flux_q8_gemm(M, N, K, BF, xq, xs, wq, wsc, None, out[0], ws())
            fx.flux_moe_balance_loss(T, E, k, 1, 0.1, 0.01, logits, ids, None, out[5], out[6], e(E), e(2, dt=torch.int32), e(T), ws())
            fx.flux_q8_gemm(M, N, K, BF, xq, xs, wq, wsc, None, out[0], ws())
            fx.flux_w4_gemv(6, 512, K, 64, BF, a4, q2, sc2, out[7], ws())
            fx.flux_q8_gemm(8, N, K, BF, xq, xs, wq, wsc, None, out[1], ws())
        torch.cuda.synchronize()
        return out

    one = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    want = step(lambda: torch.zeros(64 << 20, dtype=torch.uint8, device="cuda"))
    for a, b in zip(step(lambda: one), want):
        assert torch.equal(a, b)
    assert not bool(one[:256].any()) and bool(one[256:].any())
