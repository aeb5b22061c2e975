"""GPU parity of the 8-bit rows and products (flux_q8_quantize, flux_q8_gemm) with
their definitions, through the C ABI."""
import numpy as np
import pytest

import oracle
from tests.rounding import check16
from workloads import gen
from workloads.torch_io import to_device, torch_dtype

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import reducescatter_tcgen05_tmem_gb300 as fx  # noqa: E402

DT = {"f16": fx.FLUX_F16, "bf16": fx.FLUX_BF16}


def _ws(nbytes, fill=0):
    n = max(nbytes, 256) // 4
    ws = torch.full((n + 64,), fill, dtype=torch.int32, device="cuda")
    off = (-ws.data_ptr()) % 256 // 4
    ws = ws[off:off + n]
    ws[:64] = 0
    return ws


def _quantize(x, dtype):
    rows, K = x.shape
    q = torch.full((rows * K + 64,), 99, dtype=torch.int8, device="cuda")
    s = torch.full((rows + 8,), 7.0, device="cuda")
    fx.flux_q8_quantize(rows, K, DT[dtype], x, q, s)
    assert bool((q[rows * K:] == 99).all()) and bool((s[rows:] == 7.0).all())
    return q[:rows * K].view(rows, K), s[:rows]


@pytest.mark.parametrize("rows,K", [(1, 16), (3, 64), (7, 4096), (2, 4112), (5, 16384), (2, 16400), (3, 32768), (2, 32784),
                                    (1, 131056), (1000, 1024)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_quantize(rows, K, dtype):
    x = gen.normal16((rows, K), (rows, K), 1.7, dtype)
    q, s = _quantize(to_device(x, dtype), dtype)
    want_q, want_s = oracle.q8_quantize(oracle.widen(x, dtype))
    assert np.array_equal(s.cpu().numpy(), want_s)
    assert np.array_equal(q.cpu().numpy(), want_q)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_quantize_borders(dtype):
    # every 16-bit pattern, in rows whose scales put many quotients on or next to a half
    bits = np.arange(65536, dtype=np.uint16).view(np.int16)
    t = torch.from_numpy(bits.copy()).view(torch_dtype(dtype))
    t = t[torch.isfinite(t.float())]
    rows = []
    for top in (127.0, 63.5, 1.0, 254.0, 3.0, 1e-4, 0.0078125 * 127):
        v = t[t.float().abs() <= top]
        v = torch.cat([torch.tensor([top], dtype=t.dtype), v])
        v = torch.cat([v, v.new_zeros(-v.numel() % 16)])
        rows.append(v)
    for v in rows:
        q, s = _quantize(v.view(1, -1).cuda(), dtype)
        want_q, want_s = oracle.q8_quantize(v.double().numpy()[None])
        assert np.array_equal(s.cpu().numpy(), want_s)
        assert np.array_equal(q.cpu().numpy(), want_q)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_quantize_least_numbers_and_not_finite(dtype):
    least = float(torch.finfo(torch_dtype(dtype)).smallest_normal)
    x = torch.zeros(6, 64, dtype=torch_dtype(dtype))
    x[0] = torch.arange(64) * least
    x[1, 5] = torch.tensor([1], dtype=torch.int16).view(x.dtype)[0]  # the least number of all
    x[2, 7] = float("nan")
    x[3, 7] = float("-inf")
    x[4] = torch.finfo(x.dtype).max
    q, s = _quantize(x.cuda(), dtype)
    want_q, want_s = oracle.q8_quantize(x.double().numpy())
    assert np.array_equal(s.cpu().numpy(), want_s, equal_nan=True)
    assert np.array_equal(q.cpu().numpy(), want_q)
    w = torch.ones(8, 64, dtype=torch.int8, device="cuda")
    out = torch.empty(6, 8, dtype=x.dtype, device="cuda")
    fx.flux_q8_gemm(6, 8, 64, DT[dtype], q.contiguous(), s.contiguous(), w, torch.ones(8, device="cuda"), None, out,
                    _ws(fx.flux_q8_workspace_size(6, 8, 64)))
    assert bool(torch.isnan(out[2:4]).all()) and bool((out[5] == 0).all())


class Product:
    def __init__(self, M, N, K, dtype, bias=False, seed=0, spread=40.0):
        r = np.random.default_rng(seed)
        self.M, self.N, self.K, self.dtype = M, N, K, dtype
        draw = lambda n: np.clip(np.rint(r.standard_normal((n, K)) * spread), -128, 127).astype(np.int8)  # noqa: E731
        self.x, self.w = draw(M), draw(N)
        self.xs = (r.random(M) * 0.02 + 0.005).astype(np.float32)
        self.ws = (r.random(N) * 0.02 / np.sqrt(K) + 1e-4).astype(np.float32)
        self.b = oracle.widen(gen.normal16((seed, 5), (N,), 0.5, dtype), dtype) if bias else None
        cu = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        self.d = [cu(self.x), cu(self.xs), cu(self.w), cu(self.ws),
                  None if self.b is None else torch.from_numpy(self.b).to(torch_dtype(dtype)).cuda()]

    def run(self, ws=None, stream=None):
        M, N, K = self.M, self.N, self.K
        buf = torch.full((M * N + 128,), 7.0, dtype=torch_dtype(self.dtype), device="cuda")
        buf[64:64 + M * N] = float("nan")
        if ws is None:
            ws = _ws(fx.flux_q8_workspace_size(M, N, K), fill=0x7FC07FC1)  # NaN in any type: only the header counts
        fx.flux_q8_gemm(M, N, K, DT[self.dtype], *self.d, buf[64:64 + M * N], ws, stream=stream)
        torch.cuda.synchronize()
        st, rep = fx.flux_get_status(ws)
        assert st == fx.FLUX_OK, rep
        assert bool((buf[:64] == 7.0).all()) and bool((buf[64 + M * N:] == 7.0).all())
        return buf[64:64 + M * N].view(M, N).double().cpu().numpy()

    def check(self):
        got = self.run()
        want, mag, reach = oracle.q8_gemm(self.x, self.xs, self.w, self.ws, self.b)
        # exact sums (up to 8 rows: whole numbers): the scales' two roundings, the bias's; else one rounding to 24 bits for 16 codes too
        if self.M > 8 and reach >= 1 << 24:
            big = (np.abs(self.x.astype(np.float64)) @ np.abs(self.w.astype(np.float64)).T) * self.xs[:, None] * self.ws[None]
            check16(got, want, mag + big, self.dtype, depth=8 + 2 * self.K // 16)
        else:
            check16(got, want, mag, self.dtype, depth=4)


FEW = [(1, 8, 16), (1, 16, 512), (2, 24, 528), (3, 136, 1040), (7, 4096, 4096), (8, 4104, 1024), (9, 1000, 2064), (13, 8192, 3584),
       (16, 64, 28672), (17, 264, 1536), (24, 512, 4096), (31, 40, 272), (32, 4096, 512), (1, 131072, 64), (32, 8, 131056)]
MANY = [(33, 8, 16), (33, 256, 64), (64, 128, 80), (100, 264, 400), (128, 4096, 1024), (129, 520, 1040), (256, 256, 4096),
        (257, 1000, 528), (333, 4096, 1424), (512, 8, 128), (1000, 72, 2064), (2048, 2056, 512), (700, 11272, 64), (64, 128, 16384)]


@pytest.mark.parametrize("size", FEW + MANY, ids=str)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_product(size, dtype):
    Product(*size, dtype, bias=size[0] % 2 == 1, seed=size[0]).check()


@pytest.mark.parametrize("M", [5, 32, 40, 300])
def test_largest_codes(M):
    # every product 2^14, sums up to 2^28: the integer sums stay exact, the fp32 ones round
    p = Product(M, 24, 16384, "bf16")
    p.x[:], p.w[:] = -128, -128
    p.w[3] = 127
    p.d[0], p.d[2] = torch.from_numpy(p.x).cuda(), torch.from_numpy(p.w).cuda()
    p.check()


@pytest.mark.parametrize("M", [3, 30, 200])
def test_no_inputs(M):
    p = Product(M, 24, 16, "f16", bias=True)
    p.K = 0
    p.d[0] = p.d[2] = None
    assert np.array_equal(p.run(_ws(256)), np.tile(p.b, (M, 1)))
    p.d[4] = None
    assert not p.run(_ws(256)).any()


def test_one_workspace_for_several_sizes():
    sizes = [(300, 520, 512), (8, 4096, 1024), (16, 1000, 4096), (600, 264, 272), (30, 4096, 1024), (1, 64, 16384)]
    ws = _ws(max(fx.flux_q8_workspace_size(*s) for s in sizes))
    for _ in range(2):
        for s in sizes:
            p = Product(*s, "bf16", seed=sum(s))
            want, mag, _ = oracle.q8_gemm(p.x, p.xs, p.w, p.ws, None)
            check16(p.run(ws), want, mag, "bf16", depth=4, what=str(s))


@pytest.mark.parametrize("M", [6, 200])
def test_captured_and_repeated(M):
    p = Product(M, 1032, 2048, "f16", seed=2)
    first = p.run()
    x = torch.from_numpy(gen.normal16((1, 2), (M, 2048), 1.0, "f16")).cuda()
    x = x.view(torch.float16) if x.dtype != torch.float16 else x
    q, s = torch.empty(M, 2048, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    out = torch.empty(M, 1032, dtype=torch.float16, device="cuda")
    ws = _ws(fx.flux_q8_workspace_size(M, 1032, 2048))

    def step():
        fx.flux_q8_quantize(M, 2048, fx.FLUX_F16, x, q, s)
        fx.flux_q8_gemm(M, 1032, 2048, fx.FLUX_F16, q, s, p.d[2], p.d[3], None, out, ws)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    for i in range(3):
        x.mul_(1.25)
        graph.replay()
        torch.cuda.synchronize()
        qq, ss = oracle.q8_quantize(x.double().cpu().numpy())
        want, mag, _ = oracle.q8_gemm(qq, ss, p.w, p.ws, None)
        check16(out.double().cpu().numpy(), want, mag, "f16", depth=4)
    assert np.array_equal(p.run(), first)
