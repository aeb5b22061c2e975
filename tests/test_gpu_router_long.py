"""The router's losses and gradient at the most tokens that the header allows, where
a CTA's item or its next group of tokens ends near 2^31."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import reducescatter_tcgen05_tmem_gb300 as fx  # noqa: E402


@pytest.mark.parametrize("T", [2 ** 31 - 512, 2 ** 31 - 769])
def test_losses_and_gradient_of_two_to_the_31_tokens(T):
    # one expert: lse is the score, p is 1, and sums and gradient have closed forms
    logits = torch.zeros(T, device="cuda")
    odd = torch.cat([torch.arange(0, 70), torch.arange(2 ** 30 - 40, 2 ** 30 + 40), torch.arange(T - 700, T)]).cuda()
    logits[odd] = (odd % 7).float() - 2.0
    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    e = lambda n, dt=torch.float32: torch.full((n,), 77, dtype=dt, device="cuda")  # noqa: E731
    loss, counts, probs, tokens, lse = e(3), e(2, torch.int32), e(2), e(3, torch.int32), e(T + 8)
    ws = torch.zeros(fx.flux_moe_balance_workspace_size(T, 1, 1, 1) // 4, dtype=torch.int32, device="cuda")
    fx.flux_moe_balance_loss(T, 1, 1, 1, 0.5, 1.0, logits, ids, None, loss, counts, probs, tokens, lse, ws)
    assert counts.tolist() == [T, 77] and tokens.tolist() == [T, T, 77]
    assert torch.equal(lse[:T], logits) and bool((lse[T:] == 77).all())
    z = float(logits[odd].double().square().sum()) / T
    assert abs(float(probs[0]) - 1) < 1e-5 and abs(float(loss[0]) - 0.5) < 1e-5 and abs(float(loss[1]) - z) < 1e-5 * z
    assert float(loss[2]) == 77 and float(probs[1]) == 77 and not bool(ws.any())
    dlogits = e(T + 8)
    fx.flux_moe_router_bwd(T, 1, 1, 1, 0.0, 1.0, logits, ids, None, None, lse, counts, tokens, None, None, dlogits)
    # 2 lse / n, each a rounding to fp32
    z_scale = float(torch.tensor(2.0) / torch.tensor(float(T)))
    assert torch.equal(dlogits[:T], lse[:T].mul_(z_scale)) and bool((dlogits[T:] == 77).all())
    del logits, ids, lse, dlogits
    torch.cuda.empty_cache()
