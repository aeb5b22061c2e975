"""GPU parity of the products with 4-bit weights (flux_w4_gemv, flux_moe_w4_layer0,
flux_moe_w4_layer1, flux_w4_quantize) with their float64 definitions."""
import numpy as np
import pytest

import oracle
from tests.rounding import check16
from workloads import gen
from workloads.torch_io import from_device, to_device, torch_dtype

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import reducescatter_tcgen05_tmem_gb300 as fx  # noqa: E402

DT = {"f16": fx.FLUX_F16, "bf16": fx.FLUX_BF16}


def _ws(rows, N, K, E=1):
    n = fx.flux_w4_workspace_size(rows, N, K, E) // 4
    assert n >= 64
    ws = torch.zeros(n + 64, dtype=torch.int32, device="cuda")
    off = (-ws.data_ptr()) % 256 // 4
    return ws[off:off + n]


class Weights:
    """Random codes and scales, on the host as values and on the device as the calls take them."""

    def __init__(self, E, K, N, group, dtype, seed):
        r = np.random.default_rng(seed)
        self.codes = r.integers(0, 16, (E, N, K))
        raw = gen.normal16((seed, 5), (E, -(-K // group), N), 0.02, dtype)
        self.scales = oracle.widen(raw, dtype)
        q = oracle.w4_pack(self.codes)
        pad = r.integers(0, 256, q.shape, dtype=np.uint8)  # what lies past K does not matter
        if K % 128:
            for k in range(K, q.shape[-1] * 2):
                byte, shift = oracle.w4_place(k)
                q[..., byte] = (q[..., byte] & ~np.uint8(15 << shift)) | (pad[..., byte] & np.uint8(15 << shift))
        self.q = torch.from_numpy(q).cuda()
        self.s = to_device(raw, dtype)
        self.W = oracle.w4_weights(q, self.scales, K, group)
        assert self.q.numel() == fx.flux_w4_weight_bytes(E, K, N)


def _out(rows, N, dtype):
    flat = torch.full((rows * N + 256,), 7.0, dtype=torch_dtype(dtype), device="cuda")
    flat[128:128 + rows * N] = float("nan")
    return flat, flat[128:128 + rows * N].view(rows, N)


def _read(flat, t, dtype):
    assert bool((flat[:128] == 7.0).all()) and bool((flat[128 + t.numel():] == 7.0).all()), "write outside the output"
    return oracle.widen(from_device(t), dtype)


# a lane sums up to K / 4 products of its group's inputs in fp32 one after another
def _depth(K):
    return 64 + K


GEMV = [
    # M, N, K, group, dtype
    (1, 8, 8, 32, "bf16"),
    (1, 16, 128, 128, "f16"),
    (1, 4096, 1024, 128, "bf16"),
    (2, 24, 264, 64, "f16"),
    (3, 200, 1000, 32, "bf16"),
    (5, 136, 4104, 128, "f16"),
    (7, 72, 520, 96, "bf16"),      # groups that cross the runs of 128
    (8, 512, 2048, 64, "f16"),
    (9, 512, 2048, 64, "bf16"),
    (13, 1032, 3592, 256, "f16"),
    (16, 264, 1792, 1792, "bf16"),  # one group
    (17, 88, 640, 32, "f16"),
    (33, 40, 384, 128, "bf16"),
    (64, 128, 896, 64, "f16"),
    (100, 56, 136, 32, "bf16"),
    (1024, 16, 256, 64, "f16"),
    (1, 8, 28672, 128, "bf16"),
    (4, 8200, 72, 64, "f16"),
]


@pytest.mark.parametrize("case", GEMV, ids=lambda c: "-".join(str(v) for v in c))
def test_gemv(case):
    M, N, K, group, dtype = case
    w = Weights(1, K, N, group, dtype, 11)
    raw = gen.normal16((11, 6), (M, K), 1.0, dtype)
    flat, out = _out(M, N, dtype)
    ws = _ws(M, N, K)
    for _ in range(2):
        fx.flux_w4_gemv(M, N, K, group, DT[dtype], to_device(raw, dtype), w.q, w.s, out, ws)
        got = _read(flat, out, dtype)
        if _ == 0:
            first = got
    assert np.array_equal(first, got), "repeat calls differ"
    assert not bool(ws.any())
    ref, mag = oracle.w4_gemv(oracle.widen(raw, dtype), w.W[0])
    check16(got, ref, mag, dtype, depth=_depth(K))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_exact_integers(dtype):
    # small whole inputs and scales of powers of two: every order of sums is exact
    M, N, K, group = 6, 48, 512, 32
    r = np.random.default_rng(3)
    codes = r.integers(0, 16, (1, N, K))
    scales = 2.0 ** r.integers(-6, 3, (1, K // group, N))
    x = r.integers(-1, 2, (M, K)).astype(np.float64)
    x[:, 16:] = 0  # few terms: the result stays in the type
    x[:, 500] = 1
    q = torch.from_numpy(oracle.w4_pack(codes)).cuda()
    W = oracle.w4_weights(oracle.w4_pack(codes), scales, K, group)[0]
    ref = x @ W
    dt = torch_dtype(dtype)
    out = torch.empty((M, N), dtype=dt, device="cuda")
    fx.flux_w4_gemv(M, N, K, group, DT[dtype], torch.from_numpy(x).to(dt).cuda(), q, torch.from_numpy(scales).to(dt).cuda(),
                    out, _ws(M, N, K))
    assert np.array_equal(out.double().cpu().numpy(), oracle.round_to(ref, dtype))


MOE = [
    # T, H, F, E, topk, group, dtype
    (1, 128, 64, 1, 1, 32, "bf16"),
    (1, 256, 136, 8, 2, 64, "f16"),
    (4, 264, 200, 8, 2, 32, "bf16"),
    (7, 520, 384, 5, 5, 128, "f16"),
    (24, 384, 128, 64, 6, 64, "bf16"),
    (33, 128, 96, 3, 2, 32, "f16"),
    (128, 136, 72, 4, 2, 32, "bf16"),   # 64 rows an expert
    (512, 64, 40, 2, 2, 32, "f16"),     # the most rows
    (16, 1792, 256, 200, 4, 128, "bf16"),
]


def _routing(T, E, k, seed):
    r = np.random.default_rng(seed)
    ids = np.argsort(r.random((T, E)), axis=1)[:, :k].astype(np.int32)
    w = r.random((T, k)).astype(np.float32)
    return ids, w


@pytest.mark.parametrize("case", MOE, ids=lambda c: "-".join(str(v) for v in c))
def test_moe_layers(case):
    T, H, F, E, k, group, dtype = case
    ids, gw = _routing(T, E, k, 21)
    cids, cw = torch.from_numpy(ids).cuda(), torch.from_numpy(gw).cuda()
    w1, w2 = Weights(E, H, F, group, dtype, 22), Weights(E, F, H, group, dtype, 23)
    x, h = gen.normal16((24, 1), (T, H), 1.0, dtype), gen.normal16((24, 2), (T * k, F), 1.0, dtype)
    flat, out = _out(T * k, F, dtype)
    ws = _ws(T * k, F, H, E)
    for _ in range(2):
        fx.flux_moe_w4_layer0(T, H, F, E, k, group, DT[dtype], to_device(x, dtype), w1.q, w1.s, cids, out, ws)
    ref, mag = oracle.w4_layer0(oracle.widen(x, dtype), w1.W, ids)
    check16(_read(flat, out, dtype), ref, mag, dtype, depth=_depth(H), what="layer0")
    assert not bool(ws.any())
    flat, out = _out(T, H, dtype)
    ws = _ws(T * k, H, F, E)
    for _ in range(2):
        fx.flux_moe_w4_layer1(T, H, F, E, k, group, DT[dtype], to_device(h, dtype), w2.q, w2.s, cids, cw, out, ws)
        got = _read(flat, out, dtype)
        if _ == 0:
            first = got
    assert np.array_equal(first, got), "repeat calls differ"
    ref, mag = oracle.w4_layer1(oracle.widen(h, dtype), w2.W, ids, gw.astype(np.float64))
    check16(got, ref, mag, dtype, depth=_depth(F) + k, what="layer1")
    assert not bool(ws.any())


def test_ids_out_of_range():
    T, H, F, E, k, group = 6, 128, 64, 4, 2, 32
    ids, gw = _routing(T, E, k, 31)
    ids[1, 0], ids[4] = 4, (-1, 1 << 20)
    cids, cw = torch.from_numpy(ids).cuda(), torch.from_numpy(gw).cuda()
    w1, w2 = Weights(E, H, F, group, "f16", 32), Weights(E, F, H, group, "f16", 33)
    x, h = gen.normal16((34, 1), (T, H), 1.0, "f16"), gen.normal16((34, 2), (T * k, F), 1.0, "f16")
    flat, out = _out(T * k, F, "f16")
    ws = _ws(T * k, F, H, E)
    fx.flux_moe_w4_layer0(T, H, F, E, k, group, fx.FLUX_F16, to_device(x, "f16"), w1.q, w1.s, cids, out, ws)
    got = _read(flat, out, "f16")
    ref, mag = oracle.w4_layer0(oracle.widen(x, "f16"), w1.W, ids)
    check16(got, ref, mag, "f16", depth=_depth(H))
    assert not got[[2, 8, 9]].any()
    assert fx.flux_get_status(ws)[0] == fx.FLUX_ERR_INVALID_ARG
    flat, out = _out(T, H, "f16")
    ws = _ws(T * k, H, F, E)
    fx.flux_moe_w4_layer1(T, H, F, E, k, group, fx.FLUX_F16, to_device(h, "f16"), w2.q, w2.s, cids, cw, out, ws)
    got = _read(flat, out, "f16")
    ref, mag = oracle.w4_layer1(oracle.widen(h, "f16"), w2.W, ids, gw.astype(np.float64))
    check16(got, ref, mag, "f16", depth=_depth(F) + k)
    assert not got[4].any()
    assert fx.flux_get_status(ws)[0] == fx.FLUX_ERR_INVALID_ARG
    assert fx.flux_get_status(ws)[0] == fx.FLUX_OK


def test_every_id_out_of_range_writes_zeros():
    T, H, F, E, k, group = 3, 128, 64, 4, 2, 32
    cids = torch.full((T, k), 9, dtype=torch.int32, device="cuda")
    cw = torch.ones((T, k), device="cuda")
    w2 = Weights(E, F, H, group, "bf16", 33)
    h = to_device(gen.normal16((34, 2), (T * k, F), 1.0, "bf16"), "bf16")
    flat, out = _out(T, H, "bf16")
    ws = _ws(T * k, H, F, E)
    fx.flux_moe_w4_layer1(T, H, F, E, k, group, fx.FLUX_BF16, h, w2.q, w2.s, cids, cw, out, ws)
    assert not _read(flat, out, "bf16").any()
    assert fx.flux_get_status(ws)[0] == fx.FLUX_ERR_INVALID_ARG


def test_empty_products():
    out = torch.full((3, 16), 5.0, dtype=torch.float16, device="cuda")
    ws = _ws(3, 16, 0)
    fx.flux_w4_gemv(0, 16, 64, 32, fx.FLUX_F16, None, None, None, None, ws)
    assert bool((out == 5.0).all())
    fx.flux_w4_gemv(3, 16, 0, 32, fx.FLUX_F16, None, None, None, out, ws)
    assert not bool(out.any())


def test_infinities_and_nan_stay_in_their_rows_and_columns():
    M, N, K, group, dtype = 9, 64, 256, 64, "bf16"
    w = Weights(1, K, N, group, dtype, 41)
    x = to_device(gen.normal16((42, 6), (M, K), 1.0, dtype), dtype)
    out, ws = torch.empty((M, N), dtype=torch.bfloat16, device="cuda"), _ws(M, N, K)
    fx.flux_w4_gemv(M, N, K, group, DT[dtype], x, w.q, w.s, out, ws)
    clean = out.clone()
    x[4, 100] = float("nan")
    w.s[0, 2, 33] = float("inf")
    fx.flux_w4_gemv(M, N, K, group, DT[dtype], x, w.q, w.s, out, ws)
    rows = [i for i in range(M) if i != 4]
    cols = [i for i in range(N) if i != 33]
    assert torch.equal(out[rows][:, cols], clean[rows][:, cols])
    assert bool(out[4].isnan().all()) and not bool(out[rows][:, 33].isfinite().any())


@pytest.mark.parametrize("E,K,N,group,dtype", [(1, 128, 16, 32, "bf16"), (2, 200, 24, 64, "f16"), (3, 520, 136, 128, "bf16"), (2, 264, 16, 96, "f16"),
                                               (1, 1000, 8, 1024, "f16")])
def test_quantize(E, K, N, group, dtype):
    raw = gen.normal16((51, 1), (E, K, N), 0.02, dtype)
    wide = oracle.widen(raw, dtype)
    wide[0, :group, 3] = 0  # a group of zeros
    dev = to_device(raw, dtype)
    dev[0, :group, 3] = 0
    q = torch.full((fx.flux_w4_weight_bytes(E, K, N),), 255, dtype=torch.uint8, device="cuda")
    s = torch.empty((E, -(-K // group), N), dtype=torch_dtype(dtype), device="cuda")
    fx.flux_w4_quantize(E, K, N, group, DT[dtype], dev, q, s)
    codes, scales = oracle.w4_quantize(wide, group, lambda v: oracle.round_to(v, dtype))
    assert np.array_equal(oracle.widen(from_device(s), dtype), scales)
    got = q.cpu().numpy().reshape(E, N, -1)
    assert np.array_equal(oracle.w4_codes(got, K), codes)
    back = oracle.w4_weights(got, scales, K, group)
    step = np.repeat(scales, group, axis=1)[:, :K]
    assert (np.abs(back - wide) <= step * (0.5 + 7 * 2.0 ** -8)).all()


def test_quantized_layer_is_near_the_16_bit_one():
    # the same weights through flux_gemm: each is off by at most half a step
    M, N, K, group = 8, 256, 1024, 64
    w = gen.normal16((61, 1), (K, N), 0.02, "bf16")
    x = gen.normal16((61, 2), (M, K), 1.0, "bf16")
    q = torch.empty(fx.flux_w4_weight_bytes(1, K, N), dtype=torch.uint8, device="cuda")
    s = torch.empty((K // group, N), dtype=torch.bfloat16, device="cuda")
    fx.flux_w4_quantize(1, K, N, group, fx.FLUX_BF16, to_device(w, "bf16"), q, s)
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    fx.flux_w4_gemv(M, N, K, group, fx.FLUX_BF16, to_device(x, "bf16"), q, s, out, _ws(M, N, K))
    xv, wv = oracle.widen(x, "bf16"), oracle.widen(w, "bf16")
    step = np.repeat(oracle.widen(from_device(s), "bf16"), group, axis=0)
    bound = np.abs(xv) @ (step * (0.5 + 7 * 2.0 ** -8)) + 2.0 ** -8 * np.abs(xv) @ np.abs(wv)
    assert (np.abs(oracle.widen(from_device(out), "bf16") - xv @ wv) <= bound).all()


def test_another_stream():
    M, N, K, group = 4, 512, 1024, 128
    w = Weights(1, K, N, group, "f16", 71)
    x = to_device(gen.normal16((72, 6), (M, K), 1.0, "f16"), "f16")
    a, b = (torch.empty((M, N), dtype=torch.float16, device="cuda") for _ in range(2))
    ws, ws2 = _ws(M, N, K), _ws(M, N, K)
    fx.flux_w4_gemv(M, N, K, group, fx.FLUX_F16, x, w.q, w.s, a, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    fx.flux_w4_gemv(M, N, K, group, fx.FLUX_F16, x, w.q, w.s, b, ws2, stream=s)
    s.synchronize()
    assert torch.equal(a, b)


def test_what_a_workspace_holds_past_its_header_does_not_matter():
    T, H, F, E, k, group = 5, 640, 392, 6, 2, 64
    ids, gw = _routing(T, E, k, 81)
    cids, cw = torch.from_numpy(ids).cuda(), torch.from_numpy(gw).cuda()
    w2 = Weights(E, F, H, group, "bf16", 82)
    h = to_device(gen.normal16((83, 2), (T * k, F), 1.0, "bf16"), "bf16")
    outs = []
    for fill in (0, 0x7F7F7F7F):
        ws = _ws(T * k, H, F, E)
        ws[64:] = fill
        out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        fx.flux_moe_w4_layer1(T, H, F, E, k, group, fx.FLUX_BF16, h, w2.q, w2.s, cids, cw, out, ws)
        one = torch.empty((T * k, H), dtype=torch.bfloat16, device="cuda")
        fx.flux_w4_gemv(T * k, H, F, group, fx.FLUX_BF16, h, w2.q[:H], w2.s[0], one, ws)
        assert not bool(ws[:64].any())
        outs.append((out, one))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
