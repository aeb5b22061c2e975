"""The router's entry points refuse more tokens than their kernels count, on the host
before any GPU work (CPU only: no compute calls)."""
import pytest

FAKE = 1 << 20  # never dereferenced: every case is refused
MOST = 2 ** 31 - 512


class WS:
    def data_ptr(self):
        return FAKE

    def numel(self):
        return 1 << 50

    def element_size(self):
        return 1


@pytest.fixture(scope="module")
def fx():
    from tests.conftest import ensure_built
    ensure_built()
    import reducescatter_tcgen05_tmem_gb300 as m
    return m


@pytest.mark.parametrize("T,E,S", [(MOST + 1, 1, 1), (2 ** 31 - 1, 1, 1), (2 ** 31 - 8, 4, 8), (2 ** 31 - 1, 1, 2 ** 31 - 1)])
def test_more_tokens_than_are_counted(fx, T, E, S):
    def status(fn, *args):
        with pytest.raises(fx.FluxError) as e:
            fn(*args, stream=0)
        return e.value.status

    p = [FAKE] * 8
    assert status(fx.flux_moe_balance_loss, T, E, 1, S, 0.1, 0.1, *p, WS()) == fx.FLUX_ERR_INVALID_ARG
    assert status(fx.flux_moe_router_bwd, T, E, 1, S, 0.1, 0.1, *p, FAKE, FAKE) == fx.FLUX_ERR_INVALID_ARG
    assert fx.flux_moe_balance_workspace_size(T, E, 1, S) == 0


@pytest.mark.parametrize("E", [1, 4, 1000])
@pytest.mark.parametrize("S", [1, 2, 228, 256, 456, 512])
def test_the_most_tokens_have_a_workspace(fx, E, S):
    n = fx.flux_moe_balance_workspace_size(MOST // S * S, E, 1, S)
    assert 256 <= n <= 64 << 20
