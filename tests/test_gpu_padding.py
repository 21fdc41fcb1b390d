"""Padding rows of mla_batch_plan (seq_idx -1) through the calls that read
seq_idx: they store nothing and raise no error, the other rows are as without
them; any other sequence outside the cache is still an error."""
import math

import numpy as np
import pytest

from mla_latent_kv_33_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mla_latent_kv_33_b200 import mla as m
    return m


CASES = {
    "v2_paged_T5": synth.shrink(synth.WORKLOADS["v2_b64_paged"], B=5, L_lo=1, L_hi=300),
    "v3_paged_T300": synth.shrink(synth.WORKLOADS["v3_b128_nq2"], B=150, L_lo=2, L_hi=150, median=60.0),
    "v2_contig_T3": synth.shrink(synth.WORKLOADS["v2_b16_4k"], B=3, L=77),
    "tiny_fp32_T12": synth.shrink(synth.WORKLOADS["tiny_fp32"], B=12),
    "small_bf16": synth.Workload("small_bf16", 9, d=96, n_h=3, d_h=16, d_c=32, d_cq=48, d_r=8, B=4,
                                 n_q=1, lens="uniform", L_lo=1, L_hi=40, paged=True, block_size=16),
}


def step(mla, w, x, seq_idx, positions, h, front):
    """(cache, q or None, error) after an append (or the whole front end)."""
    import torch
    from tests.gpu_util import dev, dims_of, store
    W = {k: store(x.weights[k], x.weights_bits.get(k), w.dtype) for k in x.weights}
    data = dev(x.cache, w.dtype)
    cache = mla.Cache(data, None if x.block_table is None else torch.from_numpy(x.block_table).cuda())
    s, pos = (torch.from_numpy(np.asarray(a, np.int32)).cuda() for a in (seq_idx, positions))
    q = torch.zeros((w.T, w.n_h, w.D), dtype=data.dtype, device="cuda")
    if front:
        mla.mla_front_end(dims_of(w, mla), h, W["W_DKV"], W["W_KR"], W["W_DQ"], W["W_UQ"], W["W_QR"], W["W_UK"], s, pos,
                          cache, q)
    else:
        mla.mla_cache_append(dims_of(w, mla), h, W["W_DKV"], W["W_KR"], s, pos, cache)
    return data, q, mla.mla_get_device_error()


def bits(t):
    import torch
    return t.contiguous().view(torch.uint8).view(-1, t.element_size() * t.shape[-1])


@pytest.mark.parametrize("front", [False, True])
@pytest.mark.parametrize("overlap", [False, True])
@pytest.mark.parametrize("case", list(CASES))
def test_padding_rows_are_skipped_without_an_error(mla, case, overlap, front):
    import torch
    from tests.gpu_util import store
    w = CASES[case]
    x = synth.generate(w, seed=31)
    h = store(x.h, x.h_bits, w.dtype)
    was = mla.get_launch_overlap()
    mla.set_launch_overlap(overlap)
    try:
        full, q_full, err = step(mla, w, x, x.seq_idx, x.positions, h, front)
        assert err == mla.MLA_OK
        pad = np.zeros(w.T, bool)
        pad[[0, w.T - 1]] = True
        pad[3::7] = True
        seq_idx, positions = np.where(pad, -1, x.seq_idx), x.positions.copy()
        positions[pad] = np.resize([0, -5, 2 ** 30, 7], int(pad.sum()))
        h[torch.from_numpy(np.nonzero(pad)[0]).cuda()] = float("nan")
        got, q, err = step(mla, w, x, seq_idx, positions, h, front)
    finally:
        mla.set_launch_overlap(was)
    assert err == mla.MLA_OK
    # as the run without padding, but for the cache rows of the padding rows, which are as before
    row = [int(s) * x.cache.shape[1] + int(p) if x.block_table is None else
           int(x.block_table[s, p // w.block_size]) * w.block_size + int(p) % w.block_size
           for s, p in zip(x.seq_idx, x.positions)]
    from tests.gpu_util import dev
    want = bits(full).clone()
    at = torch.tensor([r for r, k in zip(row, pad) if k], device="cuda")
    want[at] = bits(dev(x.cache, w.dtype))[at]
    assert torch.equal(bits(got), want)
    keep = torch.from_numpy(np.nonzero(~pad)[0]).cuda()
    assert torch.equal(bits(q[keep]), bits(q_full[keep]))


@pytest.mark.parametrize("front", [False, True])
@pytest.mark.parametrize("case", ["v2_paged_T5", "tiny_fp32_T12"])
@pytest.mark.parametrize("bad", [-2, -2 ** 31, "num_seqs"])
def test_other_sequences_outside_the_cache_are_reported(mla, case, bad, front):
    import torch
    from tests.gpu_util import store
    w = CASES[case]
    x = synth.generate(w, seed=32)
    h = store(x.h, x.h_bits, w.dtype)
    seq_idx = x.seq_idx.copy()
    seq_idx[1] = w.B if bad == "num_seqs" else bad
    _, _, err = step(mla, w, x, seq_idx, x.positions, h, front)
    assert err == mla.MLA_ERR_DEVICE_DATA


def test_a_mixed_step_with_padded_row_buffers(mla):
    """Requests with one new token, then two with a prompt chunk, in row buffers
    with spare rows: planned, sent through the front end, and attended as the
    calls take them: the one-token requests together, each chunk by itself over
    its own row of the table."""
    import torch
    from tests.gpu_util import ATOL, RTOL
    p = mla.dims(512, 128, 128, 512, 192, 64)
    g = torch.Generator(device="cuda")
    g.manual_seed(41)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)
    i32 = dict(dtype=torch.int32, device="cuda")
    W = [normal(m, n, std=n ** -0.5) for m, n in ((512, 512), (64, 512), (192, 512), (16384, 192), (8192, 192),
                                                  (16384, 512))]
    ctx, new = [5, 64, 700, 0, 129, 300, 64, 0], [1, 1, 1, 1, 1, 1, 37, 150]
    B, T, width, nb = 8, sum(new) + 23, 12, 60
    data = normal(nb, 64, 576)
    pool = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, width), -1, **i32)
    at = 0
    for b, c in enumerate(ctx):
        n = -(-c // 64)
        table[b, :n] = pool[at:at + n]
        at += n
    cache = mla.Cache(data, table)
    seq_lens, row_start, used = torch.zeros(B, **i32), torch.zeros(B + 1, **i32), torch.zeros(1, **i32)
    seq_idx, pos = torch.zeros(T, **i32), torch.zeros(T, **i32)
    slots = torch.zeros(T, dtype=torch.int64, device="cuda")
    mla.mla_batch_plan(cache, torch.tensor(ctx, **i32), torch.tensor(new, **i32), pool[at:].contiguous(), seq_lens,
                       row_start, seq_idx, pos, slots, used)
    h, q = normal(T, 512), torch.zeros((T, 128, 576), dtype=torch.bfloat16, device="cuda")
    before = data.clone()
    mla.mla_front_end(p, h, *W, seq_idx, pos, cache, q)
    assert mla.mla_get_device_error() == mla.MLA_OK
    assert row_start.tolist() == [sum(new[:b]) for b in range(B + 1)] and (seq_idx[sum(new):] == -1).all()
    changed = (bits(data) != bits(before)).any(dim=1).nonzero().view(-1)
    assert changed.tolist() == sorted(slots[:sum(new)].tolist())
    o, lse = torch.zeros((T, 128, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((T, 128), device="cuda")
    mla.mla_decode(p, q[:6], cache, seq_lens[:6], 1, o[:6], lse[:6])
    for b in (6, 7):
        rows = slice(sum(new[:b]), sum(new[:b + 1]))
        mla.mla_decode(p, q[rows], mla.Cache(data, table[b:b + 1]), seq_lens[b:b + 1], new[b], o[rows], lse[rows])
    assert mla.mla_get_device_error() == mla.MLA_OK
    assert (o[sum(new):] == 0).all() and (lse[sum(new):] == 0).all()
    flat = data.view(-1, 576).double()
    for b in range(B):
        L = ctx[b] + new[b]
        i = torch.arange(L, device="cuda")
        keys = flat[table[b, i // 64].long() * 64 + i % 64]
        for j in range(new[b]):
            t, n = sum(new[:b]) + j, ctx[b] + j + 1
            s = q[t].double() @ keys[:n].t() / math.sqrt(192)
            ref, rl = torch.softmax(s, dim=1) @ keys[:n, :512], torch.logsumexp(s, dim=1)
            assert ((o[t].double() - ref).abs() <= ATOL + RTOL * ref.abs()).all(), (b, j)
            assert ((lse[t].double() - rl).abs() <= ATOL + RTOL * rl.abs()).all(), (b, j)
