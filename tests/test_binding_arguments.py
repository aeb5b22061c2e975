"""What the binding takes for a pointer: None, an address or an object with
data_ptr(); anything else is refused in Python (CPU only).  Lists of
shards may be None only where a call has optional ones."""
import pytest

FAKE = 1 << 20


@pytest.fixture(scope="module")
def fx():
    from tests.conftest import ensure_built
    ensure_built()
    import reducescatter_tcgen05_tmem_gb300 as m
    return m


class Address(int):
    """An address as a subclass of int, as an enum or a handle type may be."""


@pytest.mark.parametrize("bad", [1.5, float(FAKE), "1048576", b"1048576", [FAKE], (FAKE,), object()], ids=repr)
def test_what_is_no_pointer_is_refused(fx, bad):
    with pytest.raises((AttributeError, TypeError)):
        fx.flux_w4_quantize(1, 0, 0, 32, fx.FLUX_F16, bad, FAKE, FAKE, stream=0)
    with pytest.raises((AttributeError, TypeError)):
        fx.flux_block_norm(1, 0, 8, fx.FLUX_F16, 0, 0, 0, 0.0, [bad], None, None, None, None, None, None, [FAKE], stream=0)
    with pytest.raises((AttributeError, TypeError)):
        fx.flux_block_norm(2, 0, 8, fx.FLUX_F16, 0, 0, 0, 0.0, [FAKE, bad], None, None, None, None, None, None, [FAKE, FAKE],
                           stream=0)


def test_pointers_are_taken(fx):
    class Tensor:
        def data_ptr(self):
            return FAKE

    for good in (None, FAKE, Address(FAKE), Tensor()):
        assert fx.binding._ptr(good) == (None if good is None else FAKE)
        for n in (1, 3):
            assert list(fx.binding._ptrs([good] * n)) == [None if good is None else FAKE] * n
    assert len(fx.binding._ptrs([])) == 0


class WS:
    def data_ptr(self):
        return FAKE

    def numel(self):
        return 1 << 40

    def element_size(self):
        return 1


def test_missing_shards_are_refused_before_anything_runs(fx):
    # the second layer's lists of a call that launches two kernels
    p = [FAKE] * 2
    for w2, out in ((None, p), (p, None)):
        with pytest.raises(TypeError):
            fx.flux_mlp_ag_rs(2, 512, 512, 512, fx.FLUX_F16, p, p, p, w2, out, None, WS(), stream=0)
    with pytest.raises(TypeError):
        fx.flux_tune_gemm_rs(2, 512, 512, 512, fx.FLUX_F16, None, p, p, WS(), stream=0)
    # and where they are optional
    fx.flux_block_norm(1, 0, 8, fx.FLUX_F16, 0, 0, 0, 0.0, None, None, None, None, None, None, None, [FAKE], stream=0)
