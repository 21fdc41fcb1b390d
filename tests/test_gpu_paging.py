"""GPU parity of mla_batch_plan (block tables and slot maps from the requests'
lengths) against a plain planner written from its definition, every entry
compared, and of mla_cache_write (rows stored by a slot map), bit for bit."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mla_latent_kv_33_b200 import mla as m
    return m


def plan_reference(ctx, new, free, shared, table, bs, num_blocks, T):
    """The definition, one request after the other."""
    table = table.copy()
    B, width = table.shape
    seq_lens, row_start = np.zeros(B, np.int64), np.zeros(B + 1, np.int64)
    seq_idx, positions, slots = np.full(T, -1), np.zeros(T, np.int64), np.full(T, -1, np.int64)
    first = used = 0
    error = False
    row = 0
    for b in range(B):
        c, n = int(ctx[b]), int(new[b])
        row_start[b] = row
        ok = c >= 0 and n >= 0 and c >= len(shared) * bs and c + n <= width * bs
        need = -(-(c + n) // bs) - -(-c // bs) if ok else 0
        rows = max(n, 0)
        fits = ok and (need == 0 or first + need <= len(free)) and (rows == 0 or row + rows <= T)
        error |= not fits
        if fits:
            table[b, :len(shared)] = shared
            for k in range(need):
                table[b, -(-c // bs) + k] = free[first + k]
            if need:
                used = first + need
            seq_lens[b] = c + n
            for i in range(rows):
                pos = c + i
                blk = int(table[b, pos // bs])
                seq_idx[row + i], positions[row + i] = b, pos
                if 0 <= blk < num_blocks:
                    slots[row + i] = blk * bs + pos % bs
                else:
                    error = True
        first += need
        row += rows
    row_start[B] = row
    return dict(table=table, seq_lens=seq_lens, row_start=row_start, seq_idx=seq_idx, positions=positions, slots=slots,
                used=np.array([used]), error=error)


def run_plan(mla, ctx, new, free, shared, table, bs, num_blocks, T, stream=None, times=1):
    import torch

    def i32(x):
        return torch.tensor(np.asarray(x, np.int32), dtype=torch.int32, device="cuda")
    B = len(ctx)
    # one canary element behind every output
    z = {k: torch.full((n + 1,), -99, dtype=torch.int64 if k == "slots" else torch.int32, device="cuda")
         for k, n in dict(seq_lens=B, row_start=B + 1, seq_idx=T, positions=T, slots=T, used=1).items()}
    t = i32(table)
    cache = mla.Cache(torch.empty((num_blocks, bs, 1), dtype=torch.bfloat16, device="cuda"), t)
    args = (i32(ctx), None if new is None else i32(new), i32(free))
    for _ in range(times):
        mla.mla_batch_plan(cache, *args, *(z[k][:-1] for k in ("seq_lens", "row_start", "seq_idx", "positions",
                                                               "slots", "used")),
                           shared_blocks=i32(shared) if len(shared) else None, stream=stream)
    err = mla.mla_get_device_error(stream)
    assert all(int(x[-1]) == -99 for x in z.values())
    out = {k: x[:-1].cpu().numpy() for k, x in z.items()}
    out["table"] = t.cpu().numpy()
    return out, err


def same(got, ref):
    for k in ("table", "seq_lens", "row_start", "seq_idx", "positions", "slots", "used"):
        assert np.array_equal(got[k], ref[k]), (k, np.argwhere(got[k] != ref[k])[:5])


def draw_plan(seed, B, bs, ctx_hi, new_hi, nshared, pad):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(nshared * bs, nshared * bs + ctx_hi + 1, B)
    new = rng.integers(0, new_hi + 1, B)
    width = int((ctx + new).max() + bs - 1) // bs + 1
    held = -(-ctx // bs)
    need = -(-(ctx + new) // bs) - held
    num_blocks = int(nshared + (held - nshared).sum() + need.sum() + 5)
    pool = rng.permutation(num_blocks).astype(np.int32)
    table = np.full((B, width), -7, np.int32)
    at = nshared
    for b in range(B):
        k = held[b] - nshared
        table[b, nshared:held[b]] = pool[at:at + k]
        at += k
    return dict(ctx=ctx, new=new, free=pool[at:], shared=pool[:nshared], table=table, bs=bs, num_blocks=num_blocks,
                T=max(1, int(new.sum()) + pad))


CASES = {
    "one_request_first_token": dict(B=1, bs=64, ctx_hi=0, new_hi=1, nshared=0, pad=0),
    "one_long_prompt": dict(B=1, bs=16, ctx_hi=40, new_hi=5000, nshared=0, pad=3),
    "step_b64": dict(B=64, bs=64, ctx_hi=8191, new_hi=1, nshared=0, pad=0),
    "shared_b37": dict(B=37, bs=64, ctx_hi=300, new_hi=70, nshared=5, pad=11),
    "pages_of_one": dict(B=9, bs=1, ctx_hi=7, new_hi=6, nshared=2, pad=1),
    "odd_pages_b513": dict(B=513, bs=48, ctx_hi=200, new_hi=9, nshared=1, pad=0),
    "many_b16384": dict(B=16384, bs=32, ctx_hi=20, new_hi=3, nshared=0, pad=100),
}


@pytest.mark.parametrize("case", list(CASES))
@pytest.mark.parametrize("seed", [1, 2])
def test_plan_matches_its_definition(mla, case, seed):
    c = draw_plan(100 * seed + len(case), **CASES[case])
    ref = plan_reference(**c)
    got, err = run_plan(mla, **c)
    assert err == mla.MLA_OK and not ref["error"]
    same(got, ref)


def test_plan_of_one_token_each_and_planned_twice(mla):
    c = draw_plan(7, B=50, bs=64, ctx_hi=500, new_hi=1, nshared=2, pad=0)
    c["new"], c["T"] = np.ones(50, np.int64), 60
    c["free"] = np.concatenate([c["free"], np.arange(50, dtype=np.int32)])
    ref = plan_reference(**c)
    got, err = run_plan(mla, **{**c, "new": None}, times=2)
    assert err == mla.MLA_OK
    same(got, ref)


def _broken(kind):
    c = draw_plan(11, B=40, bs=16, ctx_hi=100, new_hi=30, nshared=2, pad=0)
    if kind == "negative_new":
        c["new"][[0, 17]] = -3
    elif kind == "negative_ctx":
        c["ctx"][5] = -1
    elif kind == "below_the_shared_pages":
        c["ctx"][9] = 31
    elif kind == "past_the_table":
        c["new"][20], c["T"] = c["table"].shape[1] * 16 - c["ctx"][20] + 1, 4000
    elif kind == "huge":
        c["new"][3], c["ctx"][4] = 2 ** 31 - 1, 2 ** 31 - 1
    elif kind == "pool_short":
        c["free"] = c["free"][:7]
    elif kind == "pool_empty":
        c["free"] = c["free"][:0]
    elif kind == "rows_short":
        c["T"] = int(c["new"].sum()) // 2
    elif kind == "bad_free_page":
        c["free"] = c["free"].copy()
        c["free"][[0, 3]] = [-1, c["num_blocks"]]
    elif kind == "bad_held_page":
        b = int(np.argmax((c["ctx"] % 16 > 0) & (c["new"] > 0)))
        c["table"][b, c["ctx"][b] // 16] = c["num_blocks"] + 9
    return c


@pytest.mark.parametrize("kind", ["negative_new", "negative_ctx", "below_the_shared_pages", "past_the_table", "huge",
                                  "pool_short", "pool_empty", "rows_short", "bad_free_page", "bad_held_page"])
def test_requests_that_cannot_be_planned_are_skipped_and_reported(mla, kind):
    c = _broken(kind)
    ref = plan_reference(**c)
    assert ref["error"]
    ref["row_start"] = np.minimum(ref["row_start"], 2 ** 31 - 1)
    got, err = run_plan(mla, **c)
    assert err == mla.MLA_ERR_DEVICE_DATA
    same(got, ref)
    assert mla.mla_get_device_error() == mla.MLA_OK


def test_plan_in_a_graph_and_on_another_stream(mla):
    import torch
    c = draw_plan(21, B=33, bs=64, ctx_hi=900, new_hi=40, nshared=3, pad=5)
    ref = plan_reference(**c)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got, err = run_plan(mla, **c, stream=s)
    assert err == mla.MLA_OK
    same(got, ref)

    def i32(x):
        return torch.tensor(np.asarray(x, np.int32), dtype=torch.int32, device="cuda")
    B, T = 33, c["T"]
    t = i32(c["table"])
    cache = mla.Cache(torch.empty((c["num_blocks"], 64, 1), dtype=torch.bfloat16, device="cuda"), t)
    ins = (i32(c["ctx"]), i32(c["new"]), i32(c["free"]))
    outs = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (B, B + 1, T, T)]
    outs += [torch.zeros(T, dtype=torch.int64, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")]
    sh = i32(c["shared"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.mla_batch_plan(cache, *ins, *outs, shared_blocks=sh)
    for seed in (31, 32):  # the graph reads the lengths of the replay
        n = draw_plan(seed, B=33, bs=64, ctx_hi=900, new_hi=c["new"].max(), nshared=3, pad=5)
        n.update(T=T, table=np.full_like(c["table"], 0), free=np.resize(n["free"], ins[2].numel()), shared=c["shared"],
                 num_blocks=c["num_blocks"])
        n["ctx"] = np.minimum(n["ctx"], c["ctx"])
        n["new"] = np.minimum(n["new"], c["new"])
        n["free"] = np.minimum(n["free"], c["num_blocks"] - 1)
        for dst, key in zip(ins, ("ctx", "new", "free")):
            dst.copy_(i32(n[key]))
        t.zero_()
        g.replay()
        assert mla.mla_get_device_error() == mla.MLA_OK
        ref = plan_reference(**n)
        for k, x in zip(("seq_lens", "row_start", "seq_idx", "positions", "slots", "used"), outs):
            assert np.array_equal(x.cpu().numpy(), ref[k]), k
        assert np.array_equal(t.cpu().numpy(), ref["table"])


# -------------------------------------------------------------- slot writes --

WRITES = {  # dims (d_c, d_r), dtype, rows, blocks, block size, paged
    "v2_one_row": (512, 64, "bf16", 1, 3, 64, True),
    "v2_64": (512, 64, "bf16", 64, 16, 64, True),
    "v2_5000": (512, 64, "bf16", 5000, 90, 64, True),
    "v2_fp32_777": (512, 64, "fp32", 777, 30, 32, True),
    "tiny_fp32_contiguous": (64, 16, "fp32", 33, 3, 20, False),
    "four_byte_rows": (13, 6, "fp32", 50, 9, 7, True),       # 76-byte rows
    "two_byte_rows": (13, 6, "bf16", 50, 9, 7, True),        # 38-byte rows
}


@pytest.mark.parametrize("case", list(WRITES))
@pytest.mark.parametrize("overlap", [False, True])
def test_cache_write_stores_rows_and_nothing_else(mla, case, overlap):
    import torch
    d_c, d_r, dtype, T, nb, bs, paged = WRITES[case]
    p = mla.dims(256, 4, 32, d_c, 96, d_r, dtype=dtype)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(len(case))
    rows = torch.randn((T, d_c + d_r), generator=g).to(dt)
    rows[0, 0] = float("nan")
    slots = torch.randperm(nb * bs, generator=g)[:T].clone()
    if T > 8:
        slots[torch.randperm(T, generator=g)[:5]] = torch.tensor([-1, -1, -5, -1, -2 ** 40])
    data = torch.randn((nb, bs, d_c + d_r), generator=g).to(dt)
    want = data.clone().view(-1, d_c + d_r)
    keep = slots >= 0
    want[slots[keep]] = rows[keep]
    dev = data.cuda()
    table = torch.zeros((1, nb), dtype=torch.int32, device="cuda") if paged else None
    was = mla.get_launch_overlap()
    mla.set_launch_overlap(overlap)
    try:
        mla.mla_cache_write(p, rows.cuda(), slots.cuda(), mla.Cache(dev, table))
    finally:
        mla.set_launch_overlap(was)
    assert mla.mla_get_device_error() == mla.MLA_OK
    it = torch.int16 if dtype == "bf16" else torch.int32
    assert torch.equal(dev.cpu().view(it), want.view(dev.shape).view(it))


def test_cache_write_reports_a_slot_past_the_cache(mla):
    import torch
    p = mla.dims(5120, 128, 128, 512, 1536, 64)
    rows = torch.ones((4, 576), dtype=torch.bfloat16, device="cuda")
    data = torch.zeros((2, 64, 576), dtype=torch.bfloat16, device="cuda")
    cache = mla.Cache(data, torch.zeros((1, 2), dtype=torch.int32, device="cuda"))
    mla.mla_cache_write(p, rows, torch.tensor([3, 128, 2 ** 40, 127], device="cuda"), cache)
    assert mla.mla_get_device_error() == mla.MLA_ERR_DEVICE_DATA
    got = data.view(128, 576).float().sum(dim=1).cpu()
    assert got[3] == 576 and got[127] == 576 and got.sum() == 2 * 576
