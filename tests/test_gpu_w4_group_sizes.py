"""Groups of more inputs than there are: one scale a column, however large the group's
size is, up to the largest that an int holds."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import reducescatter_tcgen05_tmem_gb300 as fx  # noqa: E402

# of the same remainder by 128, which decides how scales are read
LARGE = {32: 2 ** 31 - 96, 64: 2 ** 31 - 64, 96: 2 ** 31 - 32, 128: 2 ** 31 - 128}


@pytest.mark.parametrize("K,rest", [(8, 32), (64, 64), (96, 96), (264, 32), (520, 64), (1000, 96), (1032, 128), (4096, 128)])
def test_one_group_whatever_its_size(K, rest):
    E, N, T, k = 5, 136, 6, 2
    group = -(-K // 128) * 128 + rest
    g = torch.Generator(device="cuda")
    g.manual_seed(K)
    w = torch.randn((E, K, N), device="cuda", generator=g).to(torch.bfloat16)
    x = torch.randn((T, K), device="cuda", generator=g).to(torch.bfloat16)
    h = torch.randn((T * k, K), device="cuda", generator=g).to(torch.bfloat16)
    ids = torch.rand((T, E), device="cuda", generator=g).argsort(1)[:, :k].to(torch.int32).contiguous()
    weights = torch.rand((T, k), device="cuda", generator=g)
    got = []
    for size in (group, LARGE[rest]):
        assert size % 32 == 0 and size % 128 == group % 128 and size < 2 ** 31
        q = torch.full((fx.flux_w4_weight_bytes(E, K, N),), 255, dtype=torch.uint8, device="cuda")
        s = torch.empty((E, 1, N), dtype=torch.bfloat16, device="cuda")
        fx.flux_w4_quantize(E, K, N, size, fx.FLUX_BF16, w, q, s)
        ws = torch.zeros(fx.flux_w4_workspace_size(T * k, N, K, E) // 4, dtype=torch.int32, device="cuda")
        one, rows, sums = (torch.empty((n, N), dtype=torch.bfloat16, device="cuda") for n in (T, T * k, T))
        fx.flux_w4_gemv(T, N, K, size, fx.FLUX_BF16, x, q, s, one, ws)
        fx.flux_moe_w4_layer0(T, K, N, E, k, size, fx.FLUX_BF16, x, q, s, ids, rows, ws)
        fx.flux_moe_w4_layer1(T, N, K, E, k, size, fx.FLUX_BF16, h, q, s, ids, weights, sums, ws)
        got.append((q, s, one, rows, sums))
        # the scale is the column's largest magnitude / 7, and the products are of its codes
        assert torch.equal(s[:, 0], (w.float().abs().amax(1) / 7).to(torch.bfloat16))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    step = got[0][1][0].double()
    bound = x.double().abs() @ (step * (0.5 + 7 * 2.0 ** -8)).expand(K, N) + 2.0 ** -7 * (x.double().abs() @ w[0].double().abs())
    assert bool(((got[0][2].double() - x.double() @ w[0].double()).abs() <= bound).all())
