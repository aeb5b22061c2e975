"""One MoE block of a transformer, as a training step sees it and as decoding does.

Training (R virtual ranks, tokens sharded by rows):

    u        = norm(x)                         flux_block_norm
    scores   = u . W_router                    flux_gemm
    ids, w   = top-k gate                      flux_moe_topk_gate
    losses   = balance and z losses, counts    flux_moe_balance_loss
    y        = the experts' two layers         flux_moe_layers
    x', u'   = residual + gated norm(y), next norm   flux_block_norm

and back from the gradients of x' and u': through the norms
(flux_block_norm_bwd), and from the gate weights' gradient and the losses to
the router scores (flux_moe_router_bwd).

Decoding: the same block for a few tokens with 4-bit experts
(flux_w4_quantize once, then flux_moe_w4_layer0 / flux_moe_w4_layer1).

    python -c "import __graft_entry__ as g; g.build()" && python examples/moe_block.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import reducescatter_tcgen05_tmem_gb300 as fx  # noqa: E402

DTYPE, CODE, EPS = torch.bfloat16, fx.FLUX_BF16, 1e-6
BALANCE, ZLOSS = 0.01, 0.001


class Block:
    """Weights of one block and the workspaces its calls keep."""

    def __init__(self, R=2, T=256, H=512, F=1024, E=8, topk=2, seqs=4, group=64, seed=0):
        self.R, self.T, self.H, self.F, self.E, self.topk, self.seqs, self.group = R, T, H, F, E, topk, seqs, group
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def normal(shape, std, mean=0.0):
            return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(DTYPE)

        self.w_in, self.w_out, self.w_next = (normal((H,), 0.1, 1.0) for _ in range(3))
        self.gate = normal((1, H), 0.1, 0.5)                   # of the block's output, per channel
        self.res_scale = torch.tensor([0.95], device="cuda")   # of the residual stream
        self.w_router = normal((H, E), H ** -0.5)
        self.w1, self.w2 = normal((E, H, F), H ** -0.5), normal((E, F, H), F ** -0.5)
        # the layers take each rank's block of every expert
        f = F // R
        self.w1_shards = [self.w1[:, :, r * f:(r + 1) * f].contiguous() for r in range(R)]
        self.w2_shards = [self.w2[:, r * f:(r + 1) * f].contiguous() for r in range(R)]
        def workspace(*sizes):
            return torch.zeros(max(sizes) // 4, dtype=torch.int32, device="cuda")

        # the MoE layers leave their routing in theirs; one serves all the others
        self.ws_moe = workspace(fx.flux_moe_workspace_size(fx.FLUX_OP_MOE_LAYERS, R, T, H, F, E, topk))
        self.ws = workspace(fx.flux_workspace_size(fx.FLUX_OP_GEMM, 1, T, E, H),
                            fx.flux_moe_balance_workspace_size(T, E, topk, seqs),
                            fx.flux_block_norm_workspace_size(T, H, 1, H),
                            fx.flux_w4_workspace_size(min(T * topk, fx.FLUX_W4_MAX_ROWS), max(H, F), max(H, F), E))
        self.quantized = None

    def rows(self, t, T):
        """A [T, H] tensor as the ranks' row shards."""
        return list(t.view(self.R, T // self.R, self.H))

    def route(self, u, T):
        scores = torch.empty((T, self.E), dtype=DTYPE, device="cuda")
        fx.flux_gemm(T, self.E, self.H, CODE, u, self.w_router, scores, self.ws)
        logits = scores.float()
        ids = torch.empty((T, self.topk), dtype=torch.int32, device="cuda")
        weights = torch.empty((T, self.topk), device="cuda")
        fx.flux_moe_topk_gate(T, self.E, self.topk, logits, ids, weights)
        return logits, ids, weights

    def norm_in(self, x, T, keep=False):
        u = torch.empty_like(x)
        r = torch.empty(T, device="cuda") if keep else None
        fx.flux_block_norm(self.R, T, self.H, CODE, 0, 0, 0, EPS, self.rows(x, T), None, None, None, None, self.w_in,
                           None, self.rows(u, T), None, r)
        return u, r

    def norm_out(self, x, y, T, keep=False):
        x1, u1 = torch.empty_like(x), torch.empty_like(x)
        ry, rx = (torch.empty(T, device="cuda") if keep else None for _ in range(2))
        fx.flux_block_norm(self.R, T, self.H, CODE, 1, 1, self.H, EPS, self.rows(x, T), self.rows(y, T), self.w_out, self.gate,
                           self.res_scale, self.w_next, self.rows(x1, T), self.rows(u1, T), ry, rx)
        return x1, u1, ry, rx

    # ------------------------------------------------------------ training
    def forward(self, x, mask=None):
        T, s = self.T, {}
        u, s["r_in"] = self.norm_in(x, T, keep=True)
        s["logits"], s["ids"], s["weights"] = self.route(u, T)
        s["loss"] = torch.empty(2, device="cuda")
        s["counts"] = torch.empty((self.seqs, self.E), dtype=torch.int32, device="cuda")
        s["probs"] = torch.empty((self.seqs, self.E), device="cuda")
        s["tokens"] = torch.empty(self.seqs + 1, dtype=torch.int32, device="cuda")
        s["lse"] = torch.empty(T, device="cuda")
        fx.flux_moe_balance_loss(T, self.E, self.topk, self.seqs, BALANCE, ZLOSS, s["logits"], s["ids"], mask, s["loss"],
                                 s["counts"], s["probs"], s["tokens"], s["lse"], self.ws)
        h = [torch.empty((T * self.topk, self.F // self.R), dtype=DTYPE, device="cuda") for _ in range(self.R)]
        y = torch.empty_like(x)
        fx.flux_moe_layers(self.R, T, self.H, self.F, self.E, self.topk, CODE, self.rows(u, T), self.w1_shards,
                           self.w2_shards, s["ids"], s["weights"], h, self.rows(y, T), None, self.ws_moe)
        x1, u1, s["ry"], s["rx"] = self.norm_out(x, y, T, keep=True)
        s.update(x=x, y=y, u=u, mask=mask)
        return x1, u1, s

    def backward(self, s, dx1, du1):
        """Gradients of the residual stream before the block (the part that passes it by),
        of the block's output, of the norms' weights and of the router scores."""
        T, H = self.T, self.H
        g = {"dx": torch.empty_like(dx1), "dy": torch.empty_like(dx1), "dw_out": torch.empty(H, device="cuda"),
             "dgate": torch.empty((1, H), device="cuda"), "dres": torch.empty(1, device="cuda"),
             "dw_next": torch.empty(H, device="cuda")}
        fx.flux_block_norm_bwd(self.R, T, H, CODE, 1, 1, H, self.rows(s["x"], T), self.rows(s["y"], T), self.w_out, self.gate,
                               self.res_scale, self.w_next, s["ry"], s["rx"], self.rows(dx1, T), self.rows(du1, T),
                               self.rows(g["dx"], T), self.rows(g["dy"], T), g["dw_out"], g["dgate"], g["dres"],
                               g["dw_next"], self.ws)
        # gradient of a gate weight: its expert's output for the token, against dy
        g["dweights"] = torch.empty((T, self.topk), device="cuda")
        for e in range(self.E):
            t, j = (s["ids"] == e).nonzero(as_tuple=True)
            out = s["u"][t].float() @ self.w1[e].float() @ self.w2[e].float()
            g["dweights"][t, j] = (out * g["dy"][t].float()).sum(1)
        g["dlogits"] = torch.empty((T, self.E), device="cuda")
        fx.flux_moe_router_bwd(T, self.E, self.topk, self.seqs, BALANCE, ZLOSS, s["logits"], s["ids"], s["weights"], s["mask"],
                               s["lse"], s["counts"], s["tokens"], None, g["dweights"], g["dlogits"])
        return g

    # ------------------------------------------------------------ decoding
    def quantize(self):
        """The experts in 4 bits, once."""
        if self.quantized is None:
            self.quantized = []
            for w, K, N in ((self.w1, self.H, self.F), (self.w2, self.F, self.H)):
                q = torch.empty(fx.flux_w4_weight_bytes(self.E, K, N), dtype=torch.uint8, device="cuda")
                scales = torch.empty((self.E, -(-K // self.group), N), dtype=DTYPE, device="cuda")
                fx.flux_w4_quantize(self.E, K, N, self.group, CODE, w, q, scales)
                self.quantized.append((q, scales))
        return self.quantized

    def decode(self, x):
        """x' and u' for a few tokens (a multiple of R) with 4-bit experts."""
        T = x.shape[0]
        (q1, s1), (q2, s2) = self.quantize()
        u, _ = self.norm_in(x, T)
        _, ids, weights = self.route(u, T)
        h = torch.empty((T * self.topk, self.F), dtype=DTYPE, device="cuda")
        y = torch.empty_like(x)
        fx.flux_moe_w4_layer0(T, self.H, self.F, self.E, self.topk, self.group, CODE, u, q1, s1, ids, h, self.ws)
        fx.flux_moe_w4_layer1(T, self.H, self.F, self.E, self.topk, self.group, CODE, h, q2, s2, ids, weights, y, self.ws)
        x1, u1, _, _ = self.norm_out(x, y, T)
        return x1, u1


def main():
    b = Block()
    x = torch.randn((b.T, b.H), device="cuda").to(DTYPE)
    x1, u1, saved = b.forward(x)
    grads = b.backward(saved, torch.randn_like(x) * 0.01, torch.randn_like(x) * 0.01)
    few = 4
    y1, _ = b.decode(x[:few].contiguous())
    status, report = fx.flux_get_status(b.ws)
    if status != fx.FLUX_OK:
        raise RuntimeError(f"device status {status}: {report}")
    print("balance loss %.6f, z loss %.6f, tokens per expert %s" % (*saved["loss"].tolist(), saved["counts"].sum(0).tolist()))
    print("gradient norms: " + ", ".join(f"{k} {float(v.float().norm()):.3e}" for k, v in grads.items()))
    off = (y1.float() - x1[:few].float()).norm() / x1[:few].float().norm()
    print(f"decoding with 4-bit experts: {float(off):.3f} of the 16-bit block's output off")


if __name__ == "__main__":
    main()
