"""Refusals of the layer-norm, grouped routing and 8-bit entry points, and their
workspace sizes, on the host before any GPU work (CPU only: no compute calls)."""
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


def _check(fx, fn, base, kw, err):
    base = dict(base)
    base.update(kw)
    assert _status(fx, fn, base) == getattr(fx, "FLUX_ERR_" + err)


P = [FAKE] * 16
LN = dict(R=2, T=8, H=64, dtype=0, p=0.1, rng=FAKE, weight=FAKE, mean=FAKE, rstd=FAKE, stream=0)
COMMON = [
    (dict(R=0), "INVALID_ARG"), (dict(R=17), "INVALID_ARG"), (dict(T=7), "INVALID_ARG"), (dict(T=-2), "INVALID_ARG"),
    (dict(H=-8), "INVALID_ARG"), (dict(dtype=2), "INVALID_ARG"), (dict(p=1.0), "INVALID_ARG"), (dict(p=-0.1), "INVALID_ARG"),
    (dict(p=math.nan), "INVALID_ARG"), (dict(p=1.0 - 2.0 ** -20), "INVALID_ARG"),  # keeps 0 of 65536
    (dict(p=0.0), "INVALID_ARG"), (dict(rng=None), "INVALID_ARG"), (dict(H=60), "UNSUPPORTED"), (dict(H=16392), "UNSUPPORTED"),
    (dict(rng=FAKE + 8), "UNSUPPORTED"), (dict(weight=FAKE + 2), "UNSUPPORTED"), (dict(mean=FAKE + 4), "UNSUPPORTED"),
    (dict(rstd=FAKE + 4), "UNSUPPORTED"),
]


@pytest.mark.parametrize("kw,err", COMMON + [
    (dict(eps=-1.0), "INVALID_ARG"), (dict(eps=math.nan), "INVALID_ARG"), (dict(eps=math.inf), "INVALID_ARG"),
    (dict(x_out=None), "INVALID_ARG"), (dict(y_shards=None), "INVALID_ARG"),
    (dict(y_shards=None, x_out=None), "INVALID_ARG"),  # dropout of no block
    (dict(y_shards=None, x_out=None, p=0.0, rng=None, x_shards=None), "INVALID_ARG"),
    (dict(y_shards=None, x_out=None, p=0.0, rng=None, u_out=None), "INVALID_ARG"),
    (dict(u_out=None), "INVALID_ARG"), (dict(u_out=None, weight=None, bias=None, mean=None), "INVALID_ARG"),
    (dict(x_shards=[FAKE, None]), "INVALID_ARG"), (dict(y_shards=[FAKE, FAKE + 2]), "UNSUPPORTED"),
    (dict(u_out=[FAKE, FAKE + 8]), "UNSUPPORTED"), (dict(bias=FAKE + 2), "UNSUPPORTED"),
], ids=str)
def test_layer_norm_refusals(fx, kw, err):
    _check(fx, fx.flux_layer_norm, dict(LN, eps=1e-5, x_shards=P, y_shards=P, bias=FAKE, x_out=P, u_out=P), kw, err)


@pytest.mark.parametrize("kw,err", COMMON + [
    (dict(dx=None, dy=None), "INVALID_ARG"), (dict(du=None), "INVALID_ARG"), (dict(x_out=None), "INVALID_ARG"),
    (dict(mean=None), "INVALID_ARG"), (dict(rstd=None), "INVALID_ARG"), (dict(dx=[None, FAKE]), "INVALID_ARG"),
    (dict(du=None, x_out=None, weight=None, mean=None, rstd=None), "INVALID_ARG"),  # dweight of no norm
    (dict(dy=[FAKE, FAKE + 8]), "UNSUPPORTED"), (dict(dweight=FAKE + 4), "UNSUPPORTED"), (dict(dbias=FAKE + 4), "UNSUPPORTED"),
    (dict(T=(1 << 31) - 2, H=8), "UNSUPPORTED"),
    (dict(workspace=WS(256)), "WORKSPACE"), (dict(workspace=WS(1 << 30, FAKE + 16)), "WORKSPACE"),
], ids=str)
def test_layer_norm_bwd_refusals(fx, kw, err):
    _check(fx, fx.flux_layer_norm_bwd, dict(LN, x_out=P, dx_out=P, du=P, dx=P, dy=P, dweight=FAKE, dbias=FAKE,
                                            workspace=WS(1 << 30)), kw, err)


def test_layer_norm_workspace(fx):
    size = fx.flux_layer_norm_workspace_size
    assert size(-1, 64) == size(8, 60) == size(8, 16392) == size((1 << 31) - 1, 64) == 0
    assert size(0, 64) == size(64, 0) == 256
    for H in (8, 64, 264, 520, 1032, 4096, 8200, 16384):
        last = 0
        for T in (1, 2, 7, 64, 1000, 100000, (1 << 31) - 512):
            s = size(T, H)
            assert s >= 256 + 8 * H and s >= last  # enough for every smaller batch
            last = s
        assert last <= 256 + 2 * (8 * 456 * H * 4 + 256)


GATE = dict(T=8, E=16, topk=4, score=1, groups=4, topk_groups=2, group_top=2, renorm=1, scale=1.0, logits=FAKE, bias=FAKE,
            topk_ids=FAKE, topk_weights=FAKE, stream=0)
GATE_COMMON = [
    (dict(T=-1), "INVALID_ARG"), (dict(E=0), "INVALID_ARG"), (dict(E=1028), "INVALID_ARG"), (dict(topk=0), "INVALID_ARG"),
    (dict(topk=17), "INVALID_ARG"), (dict(score=2), "INVALID_ARG"), (dict(score=-1), "INVALID_ARG"),
    (dict(scale=math.nan), "INVALID_ARG"), (dict(scale=math.inf), "INVALID_ARG"), (dict(logits=None), "INVALID_ARG"),
    (dict(topk_ids=None), "INVALID_ARG"), (dict(logits=FAKE + 4), "UNSUPPORTED"), (dict(topk_ids=FAKE + 4), "UNSUPPORTED"),
]


@pytest.mark.parametrize("kw,err", GATE_COMMON + [
    (dict(groups=0), "INVALID_ARG"), (dict(groups=3), "INVALID_ARG"), (dict(groups=33, E=66), "INVALID_ARG"),
    (dict(topk_groups=0), "INVALID_ARG"), (dict(topk_groups=5), "INVALID_ARG"), (dict(topk=9), "INVALID_ARG"),
    (dict(group_top=0), "INVALID_ARG"), (dict(group_top=3), "INVALID_ARG"), (dict(topk_weights=None), "INVALID_ARG"),
    (dict(bias=FAKE + 4), "UNSUPPORTED"), (dict(topk_weights=FAKE + 8), "UNSUPPORTED"),
], ids=str)
def test_group_gate_refusals(fx, kw, err):
    _check(fx, fx.flux_moe_group_gate, GATE, kw, err)


@pytest.mark.parametrize("kw,err", GATE_COMMON + [
    (dict(dweights=None), "INVALID_ARG"), (dict(dlogits=None), "INVALID_ARG"), (dict(dweights=FAKE + 4), "UNSUPPORTED"),
    (dict(dlogits=FAKE + 8), "UNSUPPORTED"),
], ids=str)
def test_group_gate_bwd_refusals(fx, kw, err):
    _check(fx, fx.flux_moe_group_gate_bwd, dict(T=8, E=16, topk=4, score=1, renorm=1, scale=1.0, logits=FAKE, topk_ids=FAKE,
                                                dweights=FAKE, accumulate=0, dlogits=FAKE, stream=0), kw, err)


@pytest.mark.parametrize("kw,err", [
    (dict(rows=-1), "INVALID_ARG"), (dict(K=-16), "INVALID_ARG"), (dict(dtype=2), "INVALID_ARG"), (dict(K=24), "UNSUPPORTED"),
    (dict(K=131072), "UNSUPPORTED"), (dict(x=None), "INVALID_ARG"), (dict(q=None), "INVALID_ARG"), (dict(scales=None), "INVALID_ARG"),
    (dict(x=FAKE + 2), "UNSUPPORTED"), (dict(q=FAKE + 1), "UNSUPPORTED"), (dict(scales=FAKE + 4), "UNSUPPORTED"),
], ids=str)
def test_q8_quantize_refusals(fx, kw, err):
    _check(fx, fx.flux_q8_quantize, dict(rows=4, K=64, dtype=0, x=FAKE, q=FAKE, scales=FAKE, stream=0), kw, err)


@pytest.mark.parametrize("M", [4, 400])
@pytest.mark.parametrize("kw,err", [
    (dict(M=-1), "INVALID_ARG"), (dict(N=-8), "INVALID_ARG"), (dict(K=-16), "INVALID_ARG"), (dict(dtype=2), "INVALID_ARG"),
    (dict(K=24), "UNSUPPORTED"), (dict(K=131072), "UNSUPPORTED"), (dict(N=12), "UNSUPPORTED"), (dict(N=(1 << 30) + 8), "UNSUPPORTED"),
    (dict(x=None), "INVALID_ARG"), (dict(w=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"),
    (dict(x_scales=None), "INVALID_ARG"), (dict(w_scales=None), "INVALID_ARG"), (dict(x=FAKE + 8), "UNSUPPORTED"),
    (dict(w=FAKE + 8), "UNSUPPORTED"), (dict(out=FAKE + 8), "UNSUPPORTED"), (dict(bias=FAKE + 2), "UNSUPPORTED"),
    (dict(x_scales=FAKE + 4), "UNSUPPORTED"), (dict(w_scales=FAKE + 4), "UNSUPPORTED"), (dict(workspace=WS(255)), "WORKSPACE"),
    (dict(workspace=WS(1 << 30, FAKE + 16)), "WORKSPACE"),
], ids=str)
def test_q8_gemm_refusals(fx, kw, err, M):
    _check(fx, fx.flux_q8_gemm, dict(M=M, N=64, K=64, dtype=0, x=FAKE, x_scales=FAKE, w=FAKE, w_scales=FAKE, bias=FAKE,
                                     out=FAKE, workspace=WS(1 << 30), stream=0), kw, err)


def test_q8_workspace(fx):
    size = fx.flux_q8_workspace_size
    assert size(-1, 64, 64) == size(4, 12, 64) == size(4, 64, 24) == size(4, 64, 131072) == 0
    assert size(0, 64, 64) == size(4, 0, 64) == size(4, 64, 0) == 256
    assert size(4, 64, 64) == 256  # whole blocks of channels: no partial sums
    assert size(4, 8192, 28672) > 256
    assert size(400, 64, 64) > 256


@pytest.mark.parametrize("N,K", [(8, 16), (256, 512), (4096, 4096), (4096, 14336), (8192, 28672), (14336, 4096), (264, 131056)])
def test_a_q8_workspace_is_enough_for_every_smaller_batch(fx, N, K):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the calls would run")
    last = 0
    for M in (1, 8, 9, 16, 100, 333, 1000, 4096):
        size = fx.flux_q8_workspace_size(M, N, K)
        assert size >= last
        last = size
    for M in list(range(1, 200)) + list(range(200, 4097, 61)):
        # everything is in order but the machine
        assert _status(fx, fx.flux_q8_gemm, dict(M=M, N=N, K=K, dtype=0, x=FAKE, x_scales=FAKE, w=FAKE, w_scales=FAKE, bias=None,
                                                 out=FAKE, workspace=WS(last), stream=0)) in (fx.FLUX_ERR_CUDA, fx.FLUX_ERR_NO_DEVICE)


def test_empty_calls_return_without_a_gpu(fx):
    fx.flux_layer_norm(1, 0, 64, 0, 0.0, 1e-5, None, None, None, None, None, None, P, stream=0)
    fx.flux_moe_group_gate(0, 8, 2, 0, 1, 1, 1, 0, 1.0, None, None, None, None, stream=0)
    fx.flux_moe_group_gate_bwd(0, 8, 2, 0, 0, 1.0, None, None, None, 0, None, stream=0)
    fx.flux_q8_quantize(0, 64, 0, None, None, None, stream=0)
    fx.flux_q8_gemm(0, 64, 64, 0, None, None, None, None, None, None, WS(256), stream=0)


def test_row_shards_in_python(fx):
    for bad in (1.5, "1048576", b"1048576", [FAKE], object()):
        for shards in ([bad], [FAKE, bad]):
            with pytest.raises((AttributeError, TypeError)):
                fx.flux_layer_norm(len(shards), 0, 64, 0, 0.0, 1e-5, shards, None, None, None, None, None, P, stream=0)
    with pytest.raises(ValueError):  # fewer than ranks: the library would read past them
        fx.flux_layer_norm(4, 8, 64, 0, 0.0, 1e-5, [FAKE] * 3, None, None, None, None, None, P, stream=0)
    assert fx.binding._row_ptrs(2, [FAKE, None]) == (FAKE).to_bytes(8, "little") + bytes(8)
