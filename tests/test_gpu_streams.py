"""A call on a side stream that makes its own workspace, while the current stream
still has work queued that writes a block of the same size, freed just before."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mla_latent_kv_33_b200 import mla as m
    return m


@pytest.mark.parametrize("what", ["decode", "query_heads", "decode_shared"])
def test_work_queued_on_the_current_stream_does_not_reach_the_workspace(mla, what):
    import torch
    p = mla.dims(512, 128, 128, 512, 192, 64)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)
    B, P = 24, 256
    table = torch.randperm(B * 8, generator=g, device="cuda").to(torch.int32).view(B, 8)
    cache = mla.Cache(normal(B * 8, 64, 576), table)
    lens = torch.randint(P + 1, 513, (B,), generator=g, device="cuda").to(torch.int32)
    W_UK, W_UV, W_DQ = normal(16384, 512, std=0.04), normal(16384, 512, std=0.04), normal(192, 512, std=0.04)
    W_UQ, W_QR = normal(16384, 192, std=0.07), normal(8192, 192, std=0.07)
    h, q, qa = normal(B, 512), normal(B, 128, 576), normal(B, 128, 192)
    kc, v, kr = normal(128, P, 128), normal(128, P, 128), normal(P, 64)
    pos = torch.arange(B, dtype=torch.int32, device="cuda")
    if what == "decode":
        o = torch.zeros((B, 128, 512), dtype=torch.bfloat16, device="cuda")
        nbytes = mla.workspace_size(p, mla.OP_DECODE, B, 1, mla.cache_capacity(cache))

        def call(stream=None):
            mla.mla_decode(p, q, cache, lens, 1, o, stream=stream)
    elif what == "query_heads":
        o = torch.zeros((B, 128, 192), dtype=torch.bfloat16, device="cuda")
        nbytes = mla.workspace_size(p, mla.OP_QUERY_HEADS, B)

        def call(stream=None):
            mla.mla_query_heads(p, h, W_DQ, W_UQ, W_QR, pos, o, stream=stream)
    else:
        o = torch.zeros((B, 16384), dtype=torch.bfloat16, device="cuda")
        nbytes = mla.workspace_size(p, mla.OP_DECODE_SHARED, B, 1, P)

        def call(stream=None):
            mla.mla_decode_shared(p, qa, kc, v, kr, cache, lens, 1, W_UK, W_UV, o, stream=stream)
    call()
    want = o.clone()
    side, x = torch.cuda.Stream(), normal(8192, 8192)
    y = x @ x
    torch.cuda.synchronize()
    for _ in range(3):
        for _ in range(10):  # some milliseconds of work ahead of the fill; the side stream is idle
            torch.matmul(x, x, out=y)
        block = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        block.fill_(255)
        del block  # free for the current stream, its fill still queued
        with torch.cuda.stream(side):
            o.zero_()
        call(side)
    torch.cuda.synchronize()
    assert mla.mla_get_device_error() == mla.MLA_OK
    assert o.equal(want)
