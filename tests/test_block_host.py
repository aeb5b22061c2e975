"""Refusals of the block-norm, router and 4-bit entry points, and their workspace
sizes, on the host before any GPU work (CPU only: no compute calls)."""
import math

import pytest

FAKE = 1 << 20  # never dereferenced: every refused case fails validation first


@pytest.fixture(scope="module")
def fx():
    from tests.conftest import ensure_built
    ensure_built()
    import reducescatter_tcgen05_tmem_gb300 as m
    return m


class WS:
    def __init__(self, n, addr=FAKE):
        self.n, self.addr = n, addr

    def data_ptr(self):
        return self.addr

    def numel(self):
        return self.n

    def element_size(self):
        return 1


def _status(fx, fn, kw):
    with pytest.raises(fx.FluxError) as e:
        fn(**kw)
    return e.value.status


def _norm(fx, **kw):
    p = [FAKE] * 16
    base = dict(R=2, T=8, H=64, dtype=fx.FLUX_F16, post_norm=1, gate_rows=1, gate_cols=64, eps=1e-6, x_shards=p, y_shards=p,
                w_post=FAKE, gate=FAKE, res_scale=FAKE, w_pre=FAKE, x_out=p, u_out=p, rstd_y=FAKE, rstd_x=FAKE, stream=0)
    base.update(kw)
    return base


def _norm_bwd(fx, **kw):
    p = [FAKE] * 16
    base = dict(R=2, T=8, H=64, dtype=fx.FLUX_F16, post_norm=1, gate_rows=1, gate_cols=64, x_shards=p, y_shards=p, w_post=FAKE,
                gate=FAKE, res_scale=FAKE, w_pre=FAKE, rstd_y=FAKE, rstd_x=FAKE, dx_out=p, du=p, dx=p, dy=p, dw_post=FAKE,
                dgate=FAKE, dres_scale=FAKE, dw_pre=FAKE, workspace=WS(1 << 30), stream=0)
    base.update(kw)
    return base


COMMON = [  # (changes, FLUX_ERR_*)
    (dict(R=0), "INVALID_ARG"), (dict(R=17), "INVALID_ARG"), (dict(T=7), "INVALID_ARG"), (dict(T=-2), "INVALID_ARG"),
    (dict(dtype=2), "INVALID_ARG"), (dict(gate_rows=0), "INVALID_ARG"), (dict(gate_rows=3), "INVALID_ARG"),
    (dict(gate_cols=2), "INVALID_ARG"), (dict(H=60, gate_cols=60), "UNSUPPORTED"),
    (dict(H=16392, gate_cols=1), "UNSUPPORTED"), (dict(x_shards=None), "INVALID_ARG"),
    (dict(x_shards=[FAKE, None]), "INVALID_ARG"), (dict(x_shards=[FAKE, FAKE + 2]), "UNSUPPORTED"),
    (dict(y_shards=[None, FAKE]), "INVALID_ARG"), (dict(post_norm=0), "INVALID_ARG"),  # w_post without its norm
    (dict(w_post=FAKE + 4), "UNSUPPORTED"), (dict(gate=FAKE + 2), "UNSUPPORTED"), (dict(w_pre=FAKE + 8), "UNSUPPORTED"),
    (dict(res_scale=FAKE + 4), "UNSUPPORTED"), (dict(rstd_y=FAKE + 4), "UNSUPPORTED"),
]


@pytest.mark.parametrize("kw,err", COMMON + [
    (dict(eps=-1.0), "INVALID_ARG"), (dict(eps=math.nan), "INVALID_ARG"), (dict(eps=math.inf), "INVALID_ARG"),
    (dict(x_out=None), "INVALID_ARG"), (dict(y_shards=None), "INVALID_ARG"),
    (dict(y_shards=None, x_out=None, rstd_y=None), "INVALID_ARG"),  # w_post, gate, res_scale of no block
    (dict(u_out=None), "INVALID_ARG"), (dict(u_out=None, w_pre=None), "INVALID_ARG"),  # rstd_x of no norm
    (dict(y_shards=None, x_out=None, rstd_y=None, w_post=None, gate=None, res_scale=None, u_out=None, w_pre=None,
          rstd_x=None), "INVALID_ARG"),
    (dict(post_norm=0, w_post=None), "INVALID_ARG"),  # rstd_y without its norm
], ids=str)
def test_norm_refusals(fx, kw, err):
    assert _status(fx, fx.flux_block_norm, _norm(fx, **kw)) == getattr(fx, "FLUX_ERR_" + err)


@pytest.mark.parametrize("kw,err", COMMON + [
    (dict(dy=None), "INVALID_ARG"), (dict(dx=None), "INVALID_ARG"), (dict(rstd_y=None), "INVALID_ARG"),
    (dict(rstd_x=None), "INVALID_ARG"), (dict(du=None), "INVALID_ARG"), (dict(gate=None), "INVALID_ARG"),
    (dict(res_scale=None), "INVALID_ARG"), (dict(dw_pre=FAKE + 4), "UNSUPPORTED"), (dict(dx=[FAKE, FAKE + 8]), "UNSUPPORTED"),
    (dict(workspace=WS(256)), "WORKSPACE"), (dict(workspace=WS(1 << 30, FAKE + 16)), "WORKSPACE"),
], ids=str)
def test_norm_bwd_refusals(fx, kw, err):
    assert _status(fx, fx.flux_block_norm_bwd, _norm_bwd(fx, **kw)) == getattr(fx, "FLUX_ERR_" + err)


def _balance(fx, **kw):
    base = dict(T=8, E=4, topk=2, seqs=2, balance_coef=0.01, z_coef=0.0, logits=FAKE, topk_ids=FAKE, token_mask=FAKE,
                loss=FAKE, counts=FAKE, probs=FAKE, tokens=FAKE, lse=FAKE, workspace=WS(1 << 20), stream=0)
    base.update(kw)
    return base


ROUTER = [
    (dict(T=-1), "INVALID_ARG"), (dict(E=0), "INVALID_ARG"), (dict(E=1025), "INVALID_ARG"), (dict(topk=0), "INVALID_ARG"),
    (dict(topk=5), "INVALID_ARG"), (dict(seqs=0), "INVALID_ARG"), (dict(seqs=3), "INVALID_ARG"),
    (dict(T=1 << 30, topk=4), "INVALID_ARG"), (dict(balance_coef=math.nan), "INVALID_ARG"),
    (dict(z_coef=math.inf), "INVALID_ARG"), (dict(logits=None), "INVALID_ARG"), (dict(counts=None), "INVALID_ARG"),
    (dict(tokens=None), "INVALID_ARG"), (dict(lse=None), "INVALID_ARG"), (dict(logits=FAKE + 4), "UNSUPPORTED"),
    (dict(token_mask=FAKE + 1), "UNSUPPORTED"),
]


@pytest.mark.parametrize("kw,err", ROUTER + [
    (dict(loss=None), "INVALID_ARG"), (dict(probs=None), "INVALID_ARG"), (dict(topk_ids=None), "INVALID_ARG"),
    (dict(workspace=WS(256)), "WORKSPACE"),
], ids=str)
def test_balance_refusals(fx, kw, err):
    assert _status(fx, fx.flux_moe_balance_loss, _balance(fx, **kw)) == getattr(fx, "FLUX_ERR_" + err)


@pytest.mark.parametrize("kw,err", ROUTER + [
    (dict(dlogits=None), "INVALID_ARG"), (dict(topk_ids=None), "INVALID_ARG"), (dict(topk_weights=None), "INVALID_ARG"),
    (dict(dlogits=FAKE + 4), "UNSUPPORTED"),
], ids=str)
def test_router_bwd_refusals(fx, kw, err):
    base = dict(T=8, E=4, topk=2, seqs=2, balance_coef=0.01, z_coef=0.0, logits=FAKE, topk_ids=FAKE, topk_weights=FAKE,
                token_mask=FAKE, lse=FAKE, counts=FAKE, tokens=FAKE, dloss=FAKE, dweights=FAKE, dlogits=FAKE, stream=0)
    base.update(kw)
    assert _status(fx, fx.flux_moe_router_bwd, base) == getattr(fx, "FLUX_ERR_" + err)


@pytest.mark.parametrize("kw,err", [
    (dict(M=-1), "INVALID_ARG"), (dict(N=-8), "INVALID_ARG"), (dict(K=-8), "INVALID_ARG"), (dict(group=0), "INVALID_ARG"),
    (dict(dtype=5), "INVALID_ARG"), (dict(N=12), "UNSUPPORTED"), (dict(K=100), "UNSUPPORTED"), (dict(group=48), "UNSUPPORTED"),
    (dict(M=1025), "UNSUPPORTED"), (dict(x=None), "INVALID_ARG"), (dict(q=None), "INVALID_ARG"), (dict(scales=None), "INVALID_ARG"),
    (dict(out=None), "INVALID_ARG"), (dict(q=FAKE + 8), "UNSUPPORTED"), (dict(out=FAKE + 2), "UNSUPPORTED"),
    (dict(workspace=WS(128)), "WORKSPACE"),
], ids=str)
def test_gemv_refusals(fx, kw, err):
    base = dict(M=4, N=64, K=128, group=64, dtype=fx.FLUX_BF16, x=FAKE, q=FAKE, scales=FAKE, out=FAKE, workspace=WS(1 << 30), stream=0)
    base.update(kw)
    assert _status(fx, fx.flux_w4_gemv, base) == getattr(fx, "FLUX_ERR_" + err)


@pytest.mark.parametrize("kw,err", [
    (dict(T=-1), "INVALID_ARG"), (dict(E=0), "INVALID_ARG"), (dict(E=2000), "INVALID_ARG"), (dict(topk=0), "INVALID_ARG"),
    (dict(topk=5), "INVALID_ARG"), (dict(T=513), "UNSUPPORTED"), (dict(T=1 << 30), "UNSUPPORTED"), (dict(H=132), "UNSUPPORTED"),
    (dict(F=4), "UNSUPPORTED"), (dict(topk_ids=None), "INVALID_ARG"), (dict(topk_ids=FAKE + 4), "UNSUPPORTED"),
    (dict(workspace=WS(64)), "WORKSPACE"),
], ids=str)
def test_moe_refusals(fx, kw, err):
    base = dict(T=4, H=64, F=128, E=4, topk=2, group=64, dtype=fx.FLUX_BF16, topk_ids=FAKE, workspace=WS(1 << 30), stream=0)
    base.update(kw)
    want = getattr(fx, "FLUX_ERR_" + err)
    assert _status(fx, fx.flux_moe_w4_layer0, dict(base, x=FAKE, q1=FAKE, scales1=FAKE, h=FAKE)) == want
    one = dict(base, h=FAKE, q2=FAKE, scales2=FAKE, topk_weights=FAKE, out=FAKE)
    assert _status(fx, fx.flux_moe_w4_layer1, one) == want
    if not kw:
        assert _status(fx, fx.flux_moe_w4_layer1, dict(one, topk_weights=None)) == fx.FLUX_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,err", [
    (dict(E=0), "INVALID_ARG"), (dict(w=None), "INVALID_ARG"), (dict(group=33), "UNSUPPORTED"), (dict(K=4), "UNSUPPORTED"),
    (dict(q=FAKE + 4), "UNSUPPORTED"), (dict(dtype=-1), "INVALID_ARG"),
], ids=str)
def test_quantize_refusals(fx, kw, err):
    base = dict(E=2, K=128, N=64, group=32, dtype=fx.FLUX_F16, w=FAKE, q=FAKE, scales=FAKE, stream=0)
    base.update(kw)
    assert _status(fx, fx.flux_w4_quantize, base) == getattr(fx, "FLUX_ERR_" + err)


def test_workspace_sizes(fx):
    for T, H, g in [(1, 8, (0, 0)), (4096, 4096, (0, 0)), (32768, 4096, (1, 4096)), (4061, 12288, (31, 12288)),
                    (64, 16384, (64, 16384)), (1000, 2048, (1000, 1)), (0, 64, (1, 64))]:
        n = fx.flux_block_norm_workspace_size(T, H, *g)
        assert n >= 256 and n % 256 == 0 and n <= 64 << 20, (T, H, g)
    for T, H, g in [(-1, 8, (0, 0)), (4, 12, (0, 0)), (4, 16392, (0, 0)), (4, 8, (3, 8)), (4, 8, (2, 4))]:
        assert fx.flux_block_norm_workspace_size(T, H, *g) == 0
    for T, E, k, S in [(1, 1, 1, 1), (131072, 256, 8, 64), (600, 1024, 2, 600), (0, 4, 2, 3)]:
        n = fx.flux_moe_balance_workspace_size(T, E, k, S)
        assert n >= 256 and n % 256 == 0 and n <= 64 << 20
    assert fx.flux_moe_balance_workspace_size(4, 4, 5, 1) == 0 and fx.flux_moe_balance_workspace_size(4, 4, 2, 3) == 0
    assert fx.flux_w4_workspace_size(16, 8192, 28672) >= 256
    assert fx.flux_w4_workspace_size(1025, 8, 8) == 0 and fx.flux_w4_workspace_size(-1, 8, 8) == 0
    assert fx.flux_w4_weight_bytes(2, 200, 24) == 2 * 24 * 2 * 64 and fx.flux_w4_weight_bytes(0, 8, 8) == 0


def test_constants_are_the_headers(fx):
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "flux_gb300.h")).read()
    for name in ("FLUX_BLOCK_MAX_H", "FLUX_W4_MAX_ROWS", "FLUX_MAX_EXPERTS", "FLUX_MAX_RANKS"):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == getattr(fx, name)
