"""The norms' backward pass refuses more rows than its kernel counts, on the host before any
GPU work (CPU only: no compute calls)."""
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


@pytest.mark.parametrize("R,T", [(1, MOST + 1), (1, 2 ** 31 - 1), (8, 2 ** 31 - 8)])
def test_more_rows_than_are_counted(fx, R, T):
    def status(fn, *args):
        with pytest.raises(fx.FluxError) as e:
            fn(*args, stream=0)
        return e.value.status

    p = [FAKE] * R
    assert status(fx.flux_block_norm_bwd, R, T, 8, fx.FLUX_BF16, 0, 0, 0, p, p, None, None, None, None, None, FAKE, p, p, p, p,
                  None, None, None, None, WS()) == fx.FLUX_ERR_UNSUPPORTED
    assert fx.flux_block_norm_workspace_size(T, 8) == 0


@pytest.mark.parametrize("H", [8, 264, 1024, 4096, 16384])
def test_the_most_rows_have_a_workspace(fx, H):
    assert 256 <= fx.flux_block_norm_workspace_size(MOST, H) <= 128 << 20
