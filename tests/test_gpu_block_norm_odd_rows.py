"""Rows that are not finite stay in their rows in the backward pass of the block
norm: at every width class, with and without lanes past the row, and with enough
rows that a CTA uses each of its places for a row several times."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import reducescatter_tcgen05_tmem_gb300 as fx  # noqa: E402


def _run(form, T, H, x, y, du, dx1):
    """(dx, dy) with statistics of the forward call; eps 0."""
    ry = torch.empty(T, device="cuda") if form != "pre" else None
    rx = torch.empty(T, device="cuda") if form != "post" else None
    out = [torch.empty_like(x)]
    fx.flux_block_norm(1, T, H, fx.FLUX_BF16, 1, 0, 0, 0.0, [x], None if form == "pre" else [y], None, None, None, None,
                       None if form == "pre" else out, None if form == "post" else [torch.empty_like(x)], ry, rx)
    n = fx.flux_block_norm_workspace_size(T, H) // 4
    dx, dy = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    fx.flux_block_norm_bwd(1, T, H, fx.FLUX_BF16, 1, 0, 0, [x], None if form == "pre" else [y], None, None, None, None, ry, rx,
                           [dx1], None if form == "post" else [du], [dx], None if form == "pre" else [dy], None, None, None,
                           None, torch.zeros(n, dtype=torch.int32, device="cuda"))
    return dx, dy


# lanes past the row at 264, 1032, 4104, 7000, 8200, 10240, 12296 and 16376 columns
@pytest.mark.parametrize("form", ["both", "pre", "post"])
@pytest.mark.parametrize("H", [264, 1032, 4104, 7000, 8192, 8200, 10240, 12288, 12296, 16376])
def test_rows_that_are_not_finite_stay_in_their_rows(H, form):
    T = 1301  # eight or nine rows of a CTA of one row
    g = torch.Generator(device="cuda")
    g.manual_seed(H)
    x, y, du, dx1 = (torch.randn((T, H), device="cuda", generator=g).to(torch.bfloat16) for _ in range(4))
    want = _run(form, T, H, x, y, du, dx1)
    assert bool(want[0].isfinite().all()) and bool(want[1].isfinite().all())
    # in the first rows of a CTA's stretch: every later one shares a place with one of them
    odd = {0: (du, 3, float("nan")), 2: (du, H - 1, float("inf")), 9: (x, 0, float("nan")), 650: (y, 5, -float("inf")),
           651: (x, H // 2, float("inf")), 652: (dx1, 1, float("nan"))}
    for row, (t, col, value) in odd.items():
        t[row, col] = value
    x[1], y[1] = 0, 0
    got = _run(form, T, H, x, y, du, dx1)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[[*odd, 1]] = False
    for name, a, b in zip(("dx", "dy"), got, want):
        assert torch.equal(a[keep], b[keep]), f"{name}: rows {(~(a == b).all(1) & keep).nonzero().reshape(-1).tolist()[:12]}"
