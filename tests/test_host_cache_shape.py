"""The binding's check of a cache whose shape is not [pages or sequences][rows][row
width], on CPU: the number of rows is taken from the first two sizes, so that
with any other shape the calls would reach past the tensor."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def m():
    from mla_latent_kv_33_b200 import build
    build.build()
    from mla_latent_kv_33_b200 import mla
    return mla


class Data:
    def __init__(self, *shape):
        self.shape, self.dtype, self.device = shape, torch.bfloat16, "cuda:0"

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def get_device(self):
        return 0


def cache(m, *shape):
    c = m.Cache.__new__(m.Cache)
    c.data, c.block_table = Data(*shape), None
    c.desc = m.CacheDesc(0x10000, 0, 0, None, 0, shape[0], shape[1], 0)
    return c


@pytest.mark.parametrize("shape", [(2560, 576), (576, 576), (4, 2, 64, 576), (64, 4, 144, 576)])
def test_a_cache_of_another_shape_is_refused(m, shape):
    p = m.dims(5120, 128, 128, 512, 1536, 64)
    with pytest.raises(ValueError, match="mla_cache_write: a cache of"):
        m._take_cache(p, cache(m, *shape), 0, "mla_cache_write")


@pytest.mark.parametrize("shape", [(40, 64, 576), (1, 1, 576), (40, 64, 1, 576)])
def test_a_cache_of_rows_is_taken(m, shape):
    p, c = m.dims(5120, 128, 128, 512, 1536, 64), cache(m, *shape)
    m._take_cache(p, c, 0, "mla_cache_write")
