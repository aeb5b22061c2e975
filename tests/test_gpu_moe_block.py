"""The block of examples/moe_block.py, end to end: its norms, router, experts and
4-bit decoding against the same block in plain float32, with its gradients."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import reducescatter_tcgen05_tmem_gb300 as fx  # noqa: E402
from examples.moe_block import BALANCE, EPS, ZLOSS, Block  # noqa: E402


def _norm(x, w):
    return x * (x.square().mean(1, keepdim=True) + EPS).rsqrt() * w.float()


def _near(got, ref, rel, what):
    off = float((got.double() - ref.double()).norm() / ref.double().norm())
    assert off <= rel, (what, off)


@pytest.mark.parametrize("R", [1, 4])
def test_training_step(R):
    b = Block(R=R, T=128, H=256, F=512, seqs=2, seed=R)
    x = torch.randn((b.T, b.H), device="cuda").to(torch.bfloat16)
    mask = torch.ones(b.T, dtype=torch.uint8, device="cuda")
    mask[50:64] = 0
    dx1, du1 = (torch.randn_like(x) * 0.01 for _ in range(2))
    x1, u1, s = b.forward(x, mask)
    g = b.backward(s, dx1, du1)
    assert fx.flux_get_status(b.ws)[0] == fx.FLUX_OK and not bool(b.ws.any())

    # the same block in float32 from the stored routing and block output
    _near(s["u"], _norm(x.float(), b.w_in), 4e-3, "u")
    y = torch.zeros((b.T, b.H), device="cuda")
    for e in range(b.E):
        t, j = (s["ids"] == e).nonzero(as_tuple=True)
        y[t] += s["weights"][t, j, None] * (s["u"][t].float() @ b.w1[e].float() @ b.w2[e].float())
    _near(s["y"], y, 1e-2, "y")
    leaves = {"x": x.float(), "y": s["y"].float(), "w_out": b.w_out.float(), "gate": b.gate.float(),
              "res": b.res_scale.clone(), "w_next": b.w_next.float(), "logits": s["logits"].clone()}
    for v in leaves.values():
        v.requires_grad_(True)
    r1 = leaves["res"] * leaves["x"] + leaves["gate"] * _norm_of(leaves["y"], leaves["w_out"])
    r2 = _norm_of(r1, leaves["w_next"])
    _near(x1, r1.detach(), 4e-3, "x'")
    _near(u1, r2.detach(), 4e-3, "u'")
    z = leaves["logits"]
    chosen = z.gather(1, s["ids"].long())
    w = chosen.softmax(1)
    keep = mask.float()
    counts = s["counts"].float()
    n = keep.view(b.seqs, -1).sum(1)
    P = (z.softmax(1) * keep[:, None]).view(b.seqs, -1, b.E).sum(1) / n[:, None]
    loss0 = BALANCE * b.E / (b.topk * b.seqs) * (counts / n[:, None] * P).sum()
    loss1 = ZLOSS * (z.logsumexp(1).square() * keep).sum() / keep.sum()
    _near(s["loss"], torch.stack([loss0, loss1]).detach(), 1e-5, "losses")
    total = (r1 * dx1.float()).sum() + (r2 * du1.float()).sum() + loss0 + loss1 + (w * g["dweights"]).sum()
    total.backward()
    for got, leaf, rel in (("dx", "x", 4e-3), ("dy", "y", 4e-3), ("dw_out", "w_out", 1e-4), ("dgate", "gate", 1e-4),
                           ("dres", "res", 1e-4), ("dw_next", "w_next", 1e-4), ("dlogits", "logits", 1e-5)):
        _near(g[got].view(leaves[leaf].shape), leaves[leaf].grad, rel, got)


def _norm_of(x, w):
    return x * (x.square().mean(1, keepdim=True) + EPS).rsqrt() * w


def test_decoding_is_the_16_bit_block_with_rounded_experts():
    b = Block(R=2, seed=5)
    x = torch.randn((b.T, b.H), device="cuda").to(torch.bfloat16)
    want, _, s = b.forward(x)
    got, _ = b.decode(x[:6].contiguous())
    assert fx.flux_get_status(b.ws)[0] == fx.FLUX_OK and not bool(b.ws.any())
    # a code is off by up to half a step of about 2.7 / 7 standard deviations: 0.11 of
    # a weight on the root mean square, in each of two layers; the residual stream dilutes it
    off = float((got.float() - want[:6].float()).norm() / want[:6].float().norm())
    assert 1e-3 < off < 0.16, off
    # the 4-bit experts' own values, in float32
    (q1, s1), (q2, s2) = b.quantize()
    u, _ = b.norm_in(x[:6].contiguous(), 6)
    import oracle
    W1 = torch.from_numpy(oracle.w4_weights(q1.cpu().numpy().reshape(b.E, b.F, -1), s1.double().cpu().numpy(), b.H, b.group)).cuda()
    W2 = torch.from_numpy(oracle.w4_weights(q2.cpu().numpy().reshape(b.E, b.H, -1), s2.double().cpu().numpy(), b.F, b.group)).cuda()
    _, ids, w = b.route(u, 6)
    y = torch.zeros((6, b.H), dtype=torch.float64, device="cuda")
    for t in range(6):
        for j in range(b.topk):
            h = (u[t].double() @ W1[ids[t, j]]).to(torch.bfloat16).double()
            y[t] += w[t, j].double() * (h @ W2[ids[t, j]])
    ref = b.res_scale.double() * x[:6].double() + b.gate.double() * _norm_of(y, b.w_out.double())
    _near(got, ref, 4e-3, "x' with 4-bit experts")
