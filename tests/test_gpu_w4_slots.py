"""flux_moe_w4_layer1 with more slots a token than warps join: the slots are added in
slot order, whatever their number."""
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


def _layer1(T, H, F, E, k, group, dtype, h, q, scales, ids, weights):
    out = torch.full((T, H), float("nan"), dtype=torch_dtype(dtype), device="cuda")
    ws = torch.zeros(fx.flux_w4_workspace_size(T * k, H, F, E) // 4, dtype=torch.int32, device="cuda")
    fx.flux_moe_w4_layer1(T, H, F, E, k, group, DT[dtype], h, q, scales, ids, weights, out, ws)
    return out, ws


@pytest.mark.parametrize("k", [2, 8, 9, 15, 16, 17, 33])
def test_slots_are_added_in_slot_order(k):
    # 2^24, ones, -2^24: in slot order every one is rounded away (ties go to the even
    # 2^24) and the sum is 0; in any order that adds the ends first it is not
    T, H, F, E = 3, 136, 8, 64
    values = torch.ones((T, k), device="cuda")
    values[:, 0], values[:, k - 1] = 2.0 ** 24, -2.0 ** 24
    h = torch.zeros((T * k, F), dtype=torch.bfloat16, device="cuda")
    h[:, 0] = values.reshape(-1)
    codes = np.full((E, H, F), 9)  # a weight of 1
    q = torch.from_numpy(oracle.w4_pack(codes)).cuda()
    scales = torch.ones((E, 1, H), dtype=torch.bfloat16, device="cuda")
    ids = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t))[:k] for t in range(T)]).to(torch.int32).cuda()
    out, ws = _layer1(T, H, F, E, k, 32, "bf16", h, q, scales, ids, torch.ones((T, k), device="cuda"))
    assert not bool(out.any()) and not bool(ws.any())


@pytest.mark.parametrize("case", [(4, 136, 264, 16, 9, 32, "bf16"), (7, 264, 72, 20, 16, 64, "f16"), (3, 72, 1032, 64, 40, 128, "bf16"),
                                  (31, 520, 128, 33, 33, 32, "f16")], ids=lambda c: "-".join(str(v) for v in c))
def test_many_slots(case):
    T, H, F, E, k, group, dtype = case
    r = np.random.default_rng(17)
    ids = np.argsort(r.random((T, E)), axis=1)[:, :k].astype(np.int32)
    ids[0, k // 2], ids[T - 1, 0] = E, -1  # slots of no expert
    gw = r.random((T, k)).astype(np.float32)
    codes = r.integers(0, 16, (E, H, F))
    raw = gen.normal16((17, 5), (E, -(-F // group), H), 0.02, dtype)
    q = oracle.w4_pack(codes)
    h = gen.normal16((17, 6), (T * k, F), 1.0, dtype)
    args = (to_device(h, dtype), torch.from_numpy(q).cuda(), to_device(raw, dtype), torch.from_numpy(ids).cuda(),
            torch.from_numpy(gw).cuda())
    out, ws = _layer1(*case, *args)
    again, _ = _layer1(*case, *args)
    assert torch.equal(out, again)
    W = oracle.w4_weights(q, oracle.widen(raw, dtype), F, group)
    ref, mag = oracle.w4_layer1(oracle.widen(h, dtype), W, ids, gw.astype(np.float64))
    # a product's inputs one after another, then the slots
    check16(oracle.widen(from_device(out), dtype), ref, mag, dtype, depth=64 + F + k)
    assert fx.flux_get_status(ws)[0] == fx.FLUX_ERR_INVALID_ARG
