"""The block-norm, router and 4-bit calls captured into one CUDA graph and replayed:
the same results as called one by one, on inputs that change between replays."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import reducescatter_tcgen05_tmem_gb300 as fx  # noqa: E402

T, H, F, E, K, GROUP, S = 24, 1024, 512, 16, 2, 64, 2


def test_captured_and_replayed():
    bf, dev = torch.bfloat16, "cuda"
    x, y = (torch.randn((T, H), device=dev).to(bf) for _ in range(2))
    w = torch.rand(H, device=dev).to(bf)
    logits = torch.randn((T, E), device=dev)
    q1 = torch.randint(0, 256, (fx.flux_w4_weight_bytes(E, H, F),), dtype=torch.uint8, device=dev)
    q2 = torch.randint(0, 256, (fx.flux_w4_weight_bytes(E, F, H),), dtype=torch.uint8, device=dev)
    s1 = (torch.rand((E, H // GROUP, F), device=dev) * 0.01).to(bf)
    s2 = (torch.rand((E, F // GROUP, H), device=dev) * 0.01).to(bf)
    need = max(fx.flux_block_norm_workspace_size(T, H), fx.flux_moe_balance_workspace_size(T, E, K, S),
               fx.flux_w4_workspace_size(T * K, max(H, F), max(H, F), E))
    ws = torch.zeros(need // 4, dtype=torch.int32, device=dev)
    o = {"x1": torch.empty_like(x), "u": torch.empty_like(x), "ry": torch.empty(T, device=dev), "rx": torch.empty(T, device=dev),
         "dx": torch.empty_like(x), "dy": torch.empty_like(x), "dw": torch.empty(H, device=dev), "dp": torch.empty(H, device=dev),
         "ids": torch.empty((T, K), dtype=torch.int32, device=dev), "gw": torch.empty((T, K), device=dev),
         "loss": torch.empty(2, device=dev), "counts": torch.empty((S, E), dtype=torch.int32, device=dev),
         "probs": torch.empty((S, E), device=dev), "tokens": torch.empty(S + 1, dtype=torch.int32, device=dev),
         "lse": torch.empty(T, device=dev), "dl": torch.empty((T, E), device=dev),
         "h": torch.empty((T * K, F), dtype=bf, device=dev), "out": torch.empty((T, H), dtype=bf, device=dev),
         "one": torch.empty((3, H), dtype=bf, device=dev)}

    def calls():
        fx.flux_block_norm(1, T, H, fx.FLUX_BF16, 1, 0, 0, 1e-6, [x], [y], w, None, None, w, [o["x1"]], [o["u"]], o["ry"], o["rx"])
        fx.flux_block_norm_bwd(1, T, H, fx.FLUX_BF16, 1, 0, 0, [x], [y], w, None, None, w, o["ry"], o["rx"], [x], [y], [o["dx"]],
                               [o["dy"]], o["dw"], None, None, o["dp"], ws)
        fx.flux_moe_topk_gate(T, E, K, logits, o["ids"], o["gw"])
        fx.flux_moe_balance_loss(T, E, K, S, 0.01, 0.001, logits, o["ids"], None, o["loss"], o["counts"], o["probs"],
                                 o["tokens"], o["lse"], ws)
        fx.flux_moe_router_bwd(T, E, K, S, 0.01, 0.001, logits, o["ids"], o["gw"], None, o["lse"], o["counts"], o["tokens"],
                               None, o["gw"], o["dl"])
        fx.flux_moe_w4_layer0(T, H, F, E, K, GROUP, fx.FLUX_BF16, o["u"], q1, s1, o["ids"], o["h"], ws)
        fx.flux_moe_w4_layer1(T, H, F, E, K, GROUP, fx.FLUX_BF16, o["h"], q2, s2, o["ids"], o["gw"], o["out"], ws)
        fx.flux_w4_gemv(3, H, F, GROUP, fx.FLUX_BF16, o["h"], q2, s2, o["one"], ws)

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for seed in range(3):
        torch.manual_seed(seed)
        x.copy_(torch.randn((T, H), device=dev))
        y.copy_(torch.randn((T, H), device=dev))
        logits.copy_(torch.randn((T, E), device=dev))
        calls()
        torch.cuda.synchronize()
        want = {k: v.clone() for k, v in o.items()}
        for v in o.values():
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for k, v in o.items():
            assert torch.equal(v, want[k]), (seed, k)
        assert not bool(ws.any())
