"""The 4-bit entry points refuse sizes whose tiles would pass 32 bits, on the host
before any GPU work (CPU only: no compute calls)."""
import pytest

FAKE = 1 << 20  # never dereferenced: every case is refused


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


# the largest multiples of eight past the limit: rounded up to a tile of columns or a
# run of inputs they are 2^31
@pytest.mark.parametrize("N,K", [(2 ** 31 - 8, 8), (8, 2 ** 31 - 8), (2 ** 31 - 1016, 8), (8, 2 ** 31 - 1016)])
def test_sizes_past_the_limit_are_refused(fx, N, K):
    def status(fn, *args):
        with pytest.raises(fx.FluxError) as e:
            fn(*args, stream=0)
        return e.value.status

    ws = WS()
    assert status(fx.flux_w4_quantize, 1, K, N, 32, fx.FLUX_F16, FAKE, FAKE, FAKE) == fx.FLUX_ERR_UNSUPPORTED
    assert status(fx.flux_w4_gemv, 1, N, K, 32, fx.FLUX_F16, FAKE, FAKE, FAKE, FAKE, ws) == fx.FLUX_ERR_UNSUPPORTED
    assert status(fx.flux_moe_w4_layer0, 1, K, N, 2, 1, 32, fx.FLUX_F16, FAKE, FAKE, FAKE, FAKE, FAKE, ws) == fx.FLUX_ERR_UNSUPPORTED
    assert status(fx.flux_moe_w4_layer1, 1, N, K, 2, 1, 32, fx.FLUX_F16, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, ws) == fx.FLUX_ERR_UNSUPPORTED
    assert fx.flux_w4_weight_bytes(1, K, N) == 0 and fx.flux_w4_workspace_size(1, N, K) == 0


def test_the_limit_itself_has_sizes(fx):
    top = 2 ** 31 - 1024
    assert fx.flux_w4_weight_bytes(1, top, 8) == 8 * (top // 128) * 64
    assert fx.flux_w4_weight_bytes(1, 8, top) == top * 64
    assert fx.flux_w4_workspace_size(1, top, 8) > 4 * top and fx.flux_w4_workspace_size(1, 8, top) >= 256
