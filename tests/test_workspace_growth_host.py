"""A workspace that is enough for a batch is enough for every smaller one: the number
of tokens changes from call to call where these operators are used (CPU only)."""
import pytest


@pytest.fixture(scope="module")
def fx():
    from tests.conftest import ensure_built
    ensure_built()
    import reducescatter_tcgen05_tmem_gb300 as m
    return m


def _never_shrinks(sizes, what):
    last = 0
    for n, size in sizes:
        assert size >= last, (what, n, size, last)
        last = size


@pytest.mark.parametrize("S", [1, 2, 7, 64, 300, 600])
@pytest.mark.parametrize("E", [1, 3, 8, 16, 33, 64, 100, 256, 300, 512, 1000, 1024])
def test_balance_loss(fx, E, S):
    k = min(E, 2)
    steps = [*range(1, 1500), *range(1500, 40000, 37), *range(40000, 400000, 1009)]
    _never_shrinks(((n * S, fx.flux_moe_balance_workspace_size(n * S, E, k, S)) for n in steps), (E, S))


@pytest.mark.parametrize("H", [8, 256, 264, 1024, 4096, 5120, 12296, 16384])
@pytest.mark.parametrize("gate", ["none", "one", "scalar"])
def test_block_norm(fx, H, gate):
    g = {"none": (0, 0), "one": (1, H), "scalar": (1, 1)}[gate]
    _never_shrinks(((T, fx.flux_block_norm_workspace_size(T, H, *g)) for T in [*range(1, 4000), *range(4000, 100000, 997)]), H)


@pytest.mark.parametrize("N", [8, 4096, 14336])
def test_w4(fx, N):
    _never_shrinks(((m, fx.flux_w4_workspace_size(m, N, 4096, 8)) for m in range(0, 1025)), N)


def test_what_a_batch_needs_is_what_the_smaller_one_gets(fx):
    # 9000 tokens make 450 items of 256 experts, 8664 tokens 456
    assert fx.flux_moe_balance_workspace_size(8664, 256, 8, 1) <= fx.flux_moe_balance_workspace_size(9000, 256, 8, 1)
