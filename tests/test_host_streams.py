"""A workspace that the binding makes itself belongs to the stream of the call,
on CPU: blocks are handed out and taken back in the order of the stream they were
allocated on, so a block of another stream may still be written or read by work
queued there when the call's kernels start."""
import contextlib

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def m():
    from mla_latent_kv_33_b200 import build
    build.build()
    from mla_latent_kv_33_b200 import mla
    return mla


class Tensor:
    """Stands for a device tensor; T rows unless a shape is given."""

    def __init__(self, *shape, dtype=torch.bfloat16):
        self.shape, self.dtype, self.device = shape, dtype, "cuda:0"

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000


class Allocated(Exception):
    pass


class Stream:
    device_index, cuda_stream = 0, 0


def calls(m, stream):
    """Every call that makes a workspace when it is given none."""
    p = m.dims(5120, 128, 128, 512, 1536, 64)
    c = m.Cache.__new__(m.Cache)
    c.data, c.block_table = Tensor(40, 64, 576), Tensor(8, 32, dtype=torch.int32)
    c.desc = m.CacheDesc(0x10000, 1, 64, 0x10000, 32, 8, 0, 40)
    h, x, lens = Tensor(8, 5120), Tensor(8, 1), Tensor(8, dtype=torch.int32)
    o_lat, o, w = Tensor(8, 128, 512), Tensor(8, 16384), Tensor(16384, 512)
    kc, kr, qa = Tensor(128, 64, 128), Tensor(64, 64), Tensor(8, 128, 192)
    return {
        "mla_cache_append": lambda: m.mla_cache_append(p, h, x, x, x, x, c, stream=stream),
        "mla_absorb_q": lambda: m.mla_absorb_q(p, h, x, x, x, x, x, x, stream=stream),
        "mla_decode": lambda: m.mla_decode(p, x, c, lens, 1, o_lat, stream=stream),
        "mla_o_proj": lambda: m.mla_o_proj(p, o, x, x, stream=stream),
        "mla_o_proj_latent": lambda: m.mla_o_proj_latent(p, o_lat, x, x, stream=stream),
        "mla_absorb_q_merged": lambda: m.mla_absorb_q_merged(p, h, x, x, x, x, x, stream=stream),
        "mla_front_end": lambda: m.mla_front_end(p, h, x, x, x, x, x, x, x, x, c, x, stream=stream),
        "mla_query_heads": lambda: m.mla_query_heads(p, h, x, x, x, x, x, stream=stream),
        "mla_attend_order_a": lambda: m.mla_attend_order_a(p, x, x, x, c, lens, 1, o, stream=stream),
        "mla_decode_shared": lambda: m.mla_decode_shared(p, qa, kc, kc, kr, c, lens, 1, w, w, o, stream=stream),
        # a workspace on the CUDA cores only
        "mla_out_proj": lambda: m.mla_out_proj(m.dims(5120, 128, 128, 512, 1536, 64, dtype="fp32"), o_lat, x, x,
                                               stream=stream),
    }


NAMES = ["mla_cache_append", "mla_absorb_q", "mla_decode", "mla_out_proj", "mla_o_proj", "mla_o_proj_latent",
         "mla_absorb_q_merged", "mla_front_end", "mla_query_heads", "mla_attend_order_a", "mla_decode_shared"]


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_own_workspace_is_allocated_on_the_stream_of_the_call(m, monkeypatch, name, given):
    current = ["the current stream"]
    made = []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def empty(*size, **kw):
        made.append(current[-1])
        raise Allocated

    stream = Stream() if given else None
    call = calls(m, stream)[name]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", empty)
    with pytest.raises(Allocated):
        call()
    assert made == [stream if given else "the current stream"]
