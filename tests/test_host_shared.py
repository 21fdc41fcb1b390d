"""Host-side refusals of the shared-prefix calls, on CPU: every call below is
rejected before it touches the device (its pointers are never dereferenced), with
the status and the message that mla_last_error_message reports. The binding's
own checks (types, sizes and devices of the tensors) raise before the library is
called."""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only checks with fake device pointers")

A, MIS, WS = 0x10000, 0x10008, 1 << 34
INV, UNS, WSP = "MLA_ERR_INVALID_ARG", "MLA_ERR_UNSUPPORTED", "MLA_ERR_WORKSPACE"


@pytest.fixture(scope="module")
def m():
    from mla_latent_kv_33_b200 import build
    build.build()
    from mla_latent_kv_33_b200 import mla
    return mla


def v2(m, **kw):
    return m.dims(**{**dict(d=5120, n_h=128, d_h=128, d_c=512, d_cq=1536, d_r=64, dtype="bf16"), **kw})


def cache(m, **kw):
    c = m.CacheDesc(A, 1, 64, A, 128, 64, 0, 4096)  # 64 sequences of up to 8192 positions
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def refused(m, status, want, words):
    assert status == getattr(m, want), (status, m._lib.mla_last_error_message())
    assert words in m._lib.mla_last_error_message().decode()


def plan(m, c=None, table=1 << 24, ctx=A, new=A, B=8, free=A, num_free=4, shared=A, num_shared=2, T=16, seq_lens=2 * A,
         row_start=2 * A, seq_idx=2 * A, positions=2 * A, slots=2 * A, used=2 * A, null_cache=False):
    c = c if c is not None else cache(m)
    return m._lib.mla_batch_plan(None if null_cache else C.byref(c), table, ctx, new, B, free, num_free, shared,
                                 num_shared, T, seq_lens, row_start, seq_idx, positions, slots, used, None)


@pytest.mark.parametrize("kw,want,words", [
    (dict(null_cache=True), INV, "NULL"), (dict(B=0), INV, "positive"), (dict(T=0), INV, "positive"),
    (dict(B=65), INV, "num_seqs"), (dict(num_free=-1), INV, "num_free"), (dict(num_shared=-1), INV, "num_shared"),
    (dict(num_shared=129), INV, "max_blocks_per_seq"), (dict(table=None), INV, "NULL"), (dict(ctx=None), INV, "NULL"),
    (dict(free=None), INV, "NULL"), (dict(shared=None), INV, "NULL"), (dict(seq_lens=None), INV, "NULL"),
    (dict(row_start=None), INV, "NULL"), (dict(seq_idx=None), INV, "NULL"), (dict(positions=None), INV, "NULL"),
    (dict(slots=None), INV, "NULL"), (dict(used=None), INV, "NULL"),
])
def test_batch_plan_arguments(m, kw, want, words):
    refused(m, plan(m, **kw), want, words)


@pytest.mark.parametrize("out", ["table", "seq_lens", "row_start", "seq_idx", "positions", "slots", "used"])
@pytest.mark.parametrize("src", ["ctx", "new", "free", "shared"])
def test_batch_plan_outputs_may_not_overlap_inputs(m, out, src):
    """An output that starts on an input's last element (its table of 8 x 128
    entries starts before it and reaches into it)."""
    last = {"ctx": 7, "new": 7, "free": 3, "shared": 1}[src]
    x = 1 << 26
    refused(m, plan(m, **{src: x, out: x + 4 * last if out != "table" else x - 4 * 1023}), INV, "overlaps")


def test_batch_plan_cache(m):
    refused(m, plan(m, cache(m, paged=0, max_len=100)), INV, "paged")
    refused(m, plan(m, cache(m, block_size=0)), INV, "block_size")
    refused(m, plan(m, cache(m, num_seqs=20000), B=16385), UNS, "16384")


@pytest.mark.parametrize("kw,want,words", [
    (dict(rows=None), INV, "NULL"), (dict(slots=None), INV, "NULL"), (dict(rows=MIS), INV, "aligned"),
    (dict(T=0), INV, "positive"), (dict(T=-4), INV, "positive"),
])
def test_cache_write_arguments(m, kw, want, words):
    a = {**dict(rows=A, slots=A, T=4), **kw}
    d, c = v2(m), cache(m)
    refused(m, m._lib.mla_cache_write(C.byref(d), a["rows"], a["slots"], a["T"], C.byref(c), None), want, words)


def test_cache_write_cache(m):
    d = v2(m)
    refused(m, m._lib.mla_cache_write(C.byref(d), A, A, 4, None, None), INV, "NULL")
    refused(m, m._lib.mla_cache_write(C.byref(d), A, A, 4, C.byref(cache(m, data=MIS)), None), INV, "aligned")
    refused(m, m._lib.mla_cache_write(None, A, A, 4, C.byref(cache(m)), None), INV, "NULL")


@pytest.mark.parametrize("kw,want,words", [
    (dict(P=0), INV, "positive"), (dict(P=-1), INV, "positive"), (dict(P=8193), INV, "capacity"),
    (dict(seq=-1), INV, "seq"), (dict(seq=64), INV, "seq"), (dict(W_UK=None), INV, "NULL"), (dict(W_UV=None), INV, "NULL"),
    (dict(kc=None), INV, "NULL"), (dict(v=None), INV, "NULL"), (dict(kr=None), INV, "NULL"), (dict(kc=MIS), INV, "aligned"),
    (dict(v=MIS), INV, "aligned"), (dict(kr=MIS), INV, "aligned"), (dict(W_UV=MIS), INV, "aligned"),
    (dict(block_size=48), UNS, "multiple of 64"),
    (dict(num_blocks=1 << 26), UNS, "too many cache rows"),
])
def test_prefix_expand_arguments(m, kw, want, words):
    a = {**dict(seq=1, P=100, W_UK=A, W_UV=A, kc=A, v=A, kr=A), **kw}
    c = cache(m, **{k: a[k] for k in ("block_size", "num_blocks") if k in a})
    s = m._lib.mla_prefix_expand(C.byref(v2(m)), C.byref(c), a["seq"], a["P"], a["W_UK"], a["W_UV"], a["kc"], a["v"],
                                 a["kr"], None)
    refused(m, s, want, words)


def shared(m, d=None, c=None, qa=A, kc=A, v=A, kr=A, P=128, seq_lens=A, B=8, n_q=1, W_UK=A, W_UV=A, o=A, lse=A, ws=A,
           ws_bytes=WS):
    d, c = d if d is not None else v2(m), c if c is not None else cache(m)
    return m._lib.mla_decode_shared(C.byref(d), qa, kc, v, kr, P, C.byref(c), seq_lens, B, n_q, W_UK, W_UV, o, lse, ws,
                                    ws_bytes, None)


@pytest.mark.parametrize("kw,want,words", [
    (dict(B=0), INV, "positive"), (dict(n_q=0), INV, "positive"), (dict(P=-1), INV, "prefix_len"),
    (dict(qa=None), INV, "NULL"), (dict(seq_lens=None), INV, "NULL"), (dict(W_UK=None), INV, "NULL"),
    (dict(W_UV=None), INV, "NULL"), (dict(o=None), INV, "NULL"), (dict(kc=None), INV, "NULL"), (dict(v=None), INV, "NULL"),
    (dict(kr=None), INV, "NULL"), (dict(qa=MIS), INV, "aligned"), (dict(kc=MIS), INV, "aligned"),
    (dict(v=MIS), INV, "aligned"), (dict(kr=MIS), INV, "aligned"), (dict(o=MIS), INV, "aligned"),
    (dict(W_UK=MIS), INV, "aligned"), (dict(ws=MIS), INV, "aligned"), (dict(B=65), INV, "num_seqs"),
    (dict(P=8192), INV, "capacity"), (dict(P=2 ** 31 - 1), INV, "capacity"), (dict(P=100), UNS, "multiple of 64"),
    (dict(n_q=4000), UNS, "B*n_q"), (dict(ws=None), WSP, "workspace"), (dict(ws_bytes=100), WSP, "workspace"),
])
def test_decode_shared_arguments(m, kw, want, words):
    refused(m, shared(m, **kw), want, words)


def test_decode_shared_pages_and_dims(m):
    refused(m, shared(m, c=cache(m, block_size=32, max_blocks_per_seq=512)), UNS, "block_size")
    refused(m, shared(m, c=cache(m, num_blocks=1 << 26)), UNS, "too many rows")
    refused(m, shared(m, d=v2(m, d_h=300)), UNS, "d_h")
    refused(m, shared(m, c=cache(m, max_blocks_per_seq=2 ** 30), P=2 ** 31 - 64, n_q=100), UNS, "prefix_len")


def test_decode_shared_workspace_is_exactly_what_it_asks_for(m):
    d = v2(m)
    for B, n_q, P in ((1, 1, 64), (64, 1, 4096), (100, 2, 2112), (8, 1, 0)):
        need = m.workspace_size(d, m.OP_DECODE_SHARED, B, n_q, P)
        assert need > B * n_q * 128 * 576 * 2
        c = cache(m, num_seqs=128)
        refused(m, shared(m, B=B, n_q=n_q, P=P, c=c, ws_bytes=need - 1), WSP, str(need))
    # CUDA-core dims keep nothing in a workspace; a call too large for any has none
    assert m.workspace_size(m.dims(256, 4, 32, 64, 96, 16, dtype="fp32"), m.OP_DECODE_SHARED, 4, 1, 100) == 0
    assert m.workspace_size(d, m.OP_DECODE_SHARED, 1 << 20, 1, 64) == 0
    assert m.workspace_size(d, m.OP_PREFIX_EXPAND, 1, 1, 64) == 0


def test_tensor_core_ops_are_reported(m):
    assert m.uses_tensor_cores(v2(m), m.OP_PREFIX_EXPAND) and m.uses_tensor_cores(v2(m), m.OP_DECODE_SHARED)
    assert not m.uses_tensor_cores(v2(m, dtype="fp32"), m.OP_DECODE_SHARED)
    assert not m.uses_tensor_cores(v2(m, n_h=64), m.OP_DECODE_SHARED)


class Fake:
    """Stands for a device tensor in the binding's checks."""

    def __init__(self, shape, dtype=torch.int32, dev=0, dense=True):
        self.shape, self.dtype, self.dev, self.dense, self.device = shape, dtype, dev, dense, f"cuda:{dev}"

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return self.dense

    def data_ptr(self):
        raise AssertionError("a wrong tensor's address was taken")


@pytest.mark.parametrize("bad", [dict(dtype=torch.int64), dict(dev=1), dict(dev=-1), dict(dense=False), dict(shape=(9,))])
def test_the_binding_refuses_wrong_tensors(m, bad):
    t = Fake(**{**dict(shape=(8,)), **bad})
    with pytest.raises(ValueError, match="ctx_lens: a contiguous torch.int32 tensor of 8 elements on cuda:0"):
        m._take(t, torch.int32, 8, 0, "ctx_lens")


@pytest.mark.parametrize("current,of_stream,ok", [(0, 0, True), (1, 1, True), (0, 1, False), (1, 0, False), (0, None, True)])
def test_the_binding_refuses_a_stream_of_another_device(m, monkeypatch, current, of_stream, ok):
    class Stream:
        device_index = of_stream
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
    stream = None if of_stream is None else Stream()
    if ok:
        assert m._call_device(stream) == current
    else:
        with pytest.raises(ValueError, match=f"the stream belongs to cuda:{of_stream}, the current device is cuda:{current}"):
            m._call_device(stream)
