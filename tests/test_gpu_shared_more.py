"""Further forms of the shared-prefix calls against the definition in 64 bits:
heads whose prefix is cut into three partials, accumulator rescales on SM pairs,
fp32 storage at the DeepSeek widths, many new tokens per request, and a prefix
whose last page is not full.

Tolerances: those of test_gpu_shared.py (every bf16 rounding counted). Where keys
are scaled up or the arithmetic is fp32 only, the error ds of a score comes on
top, bounded below by the number of its fp32 roundings: a score error ds moves
the lse by at most ds and o by at most ds * (sum_i w_i |v_i| + |o|)."""
import math

import pytest

from tests.test_gpu_shared import V2, Problem, check, layer, mla, reference, run_shared  # noqa: F401

pytestmark = pytest.mark.gpu

KTILE, ABS = 128, 4  # keys per tile, absorb tiles of a unit


def partials(T, P):
    """How many clusters' ranges hold key tiles of each (row group, head) unit."""
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    cg = 2 if T > 128 else 1
    nt = -(-P // KTILE)
    units, per = -(-T // (128 * cg)) * 128, nt + ABS
    G = min(sms // cg, units * 3 // 2, units * per)
    start = [units * per * c // G for c in range(G + 1)]
    return [sum(start[c] < (u + 1) * per and start[c + 1] > u * per + ABS for c in range(G)) for u in range(units)]


@pytest.mark.parametrize("B,P,suffix", [(2, 5568, [1, 90]), (3, 8192, [300, 2, 64]),
                                        (128, 6144, [1 + i % 20 for i in range(128)])])
def test_three_partials_of_a_head_are_joined(mla, B, P, suffix):  # noqa: F811
    cut = partials(B, P)
    assert max(cut) == 3 and min(cut) >= 1
    pr = Problem(V2, "bf16", P, suffix, 1, seed=B)
    o, lse, err = run_shared(mla, pr)
    assert err == mla.MLA_OK
    check(pr, o, lse)


@pytest.mark.parametrize("B,n_q", [(5, 1), (140, 1), (128, 2), (260, 1)])
def test_growing_scores_rescale_the_accumulator(mla, B, n_q):  # noqa: F811
    """Tiles 3 and 6 of the prefix carry keys 6 and 14 times as long, so that the
    running maximum of nearly every row grows by more than 2^8 there: once for
    each softmax group, in both CTAs of a pair above 128 rows."""
    import torch
    P = 1344
    pr = Problem(V2, "bf16", P, [n_q + (5 * i) % 40 for i in range(B)], n_q, seed=60 + B)
    pr.kc[:, 3 * KTILE:4 * KTILE] *= 6
    pr.kc[:, 6 * KTILE:7 * KTILE] *= 14
    scale = 1 / math.sqrt(192)
    q, k = pr.qa.double(), pr.kc.double()
    s = (torch.einsum("thd,hpd->thp", q[..., :128], k) + torch.einsum("thr,pr->thp", q[..., 128:], pr.kr.double())) * scale
    top = torch.stack([t.amax(dim=2) for t in s.split(KTILE, dim=2)], dim=2)
    for tile in (3, 6):  # 5.55 nats are 2^8
        grown = top[:, :, tile] - top[:, :, :tile].amax(dim=2) > 5.6
        assert grown.double().mean() > 0.9 and all(g.any(dim=0).all() for g in grown.split(32))
    o, lse, err = run_shared(mla, pr)
    assert err == mla.MLA_OK
    ro, rl, tol, ltol = reference(pr, scale)
    # scores: 12 K steps, each of at most two fp32 roundings of partial sums no larger than size, and the shift by the maximum
    size = (torch.einsum("thd,hpd->thp", q[..., :128].abs(), k.abs()).amax(dim=2) +
            torch.einsum("thr,pr->thp", q[..., 128:].abs(), pr.kr.double().abs()).amax(dim=2)) * scale
    ds = 26 * 2.0 ** -23 * size
    vmax = torch.maximum(pr.v.double().abs().amax(dim=1), torch.full((128, 1), 6.0, device="cuda", dtype=torch.float64))
    tol = tol + (2 * ds[:, :, None] * vmax).view(pr.T, -1)
    err_o, err_l = (o.double() - ro).abs(), (lse.double() - rl).abs()
    assert (err_o <= tol).all(), float((err_o / tol).max())
    assert (err_l <= ltol + ds).all(), float((err_l / (ltol + ds)).max())


WIDE = dict(n_h=8, d_h=256, d_c=960, d_r=64)


@pytest.mark.parametrize("s,P,suffix,n_q,bs,paged", [
    (V2, 300, [1, 90, 17], 1, 16, True), (V2, 1100, [2, 40], 2, 64, True), (V2, 0, [5, 1030], 5, 64, False),
    (V2, 65, [64], 60, 1, True), (WIDE, 130, [3, 50], 3, 16, True)])
def test_fp32_storage_at_full_widths(mla, s, P, suffix, n_q, bs, paged):  # noqa: F811
    import torch
    pr = Problem(s, "fp32", P, suffix, n_q, bs, paged, seed=P + 7)
    o, lse, err = run_shared(mla, pr, dtype="fp32")
    assert err == mla.MLA_OK
    n_h, d_h, d_c, d_r = s["n_h"], s["d_h"], s["d_c"], s["d_r"]
    scale, e = 1 / math.sqrt(d_h + d_r), 2.0 ** -24
    wk, wv = pr.W_UK.double().view(n_h, d_h, d_c), pr.W_UV.double().view(n_h, d_h, d_c)
    for b, L in enumerate(pr.lens):
        rows = pr.suffix[b].double()
        c, kr = rows[:, :d_c], rows[:, d_c:]
        for j in range(n_q):
            t, n = b * n_q + j, L - P - n_q + 1 + j
            q = pr.qa[t].double()
            q_lat = torch.einsum("hd,hdc->hc", q[:, :d_h], wk)
            sp = torch.einsum("hd,hpd->hp", q[:, :d_h], pr.kc.double()) + q[:, d_h:] @ pr.kr.double().t()
            sc = torch.cat([sp, q_lat @ c[:n].t() + q[:, d_h:] @ kr[:n].t()], dim=1) * scale
            rl = torch.logsumexp(sc, dim=1)
            w = torch.exp(sc - rl[:, None])
            vals = torch.cat([pr.v.double(), torch.einsum("nc,hdc->hnd", c[:n], wv)], dim=1)
            ro = torch.einsum("hi,hid->hd", w, vals)
            # a score's fp32 roundings: each sum of m products rounds at most m times by e of sums no larger than their magnitude
            size_p = torch.einsum("hd,hpd->hp", q[:, :d_h].abs(), pr.kc.double().abs()) + q[:, d_h:].abs() @ pr.kr.double().abs().t()
            mag = torch.einsum("hd,hdc->hc", q[:, :d_h].abs(), wk.abs())
            size_s = mag @ c[:n].abs().t() + q[:, d_h:].abs() @ kr[:n].abs().t()
            ds = scale * e * torch.cat([((d_h + d_r) / 8 + 4) * size_p, (d_h + (d_c + d_r) / 8 + 4) * size_s], dim=1)
            ds = ds.amax(dim=1) + 4 * e * sc.abs().amax(dim=1)
            # relative error of an exponential, (2 + 1.173 |x|) ulp, once for the key and once for the chunks' rescale
            exps = 2 * e * (4 + 2.4 * (sc.amax(dim=1, keepdim=True) - sc))
            rel = ds[:, None] + exps + (P + n + d_c) * e                     # and the sums over keys and latents
            tol = torch.einsum("hi,hid->hd", w * rel, (vals - ro[:, None]).abs()) + (P + n + d_c) * e * torch.einsum(
                "hi,hid->hd", w, vals.abs()) + 4 * e * ro.abs()
            # (a suffix value goes through c and W_UV: its magnitude there bounds the roundings of the two sums)
            lat = w[:, P:] @ c[:n].abs()
            tol += (n + d_c) * e * torch.einsum("hc,hdc->hd", lat, wv.abs())
            ltol = ds + (w * exps).sum(dim=1) + (P + n) * e + 4 * e * (rl.abs() + 10)
            assert ((o[t].double().view(n_h, d_h) - ro).abs() <= tol).all(), (b, j)
            assert ((lse[t].double() - rl).abs() <= ltol).all(), (b, j)


@pytest.mark.parametrize("s,P,bs,paged", [(V2, 70, 16, True), (V2, 1, 64, True), (V2, 131, 64, False), (WIDE, 37, 16, True)])
def test_fp32_expansion_at_full_widths(mla, s, P, bs, paged):  # noqa: F811
    import torch
    pr = Problem(s, "fp32", P, [1, 70], 1, bs, paged, seed=P)
    want = pr.prefix[:, s["d_c"]:].clone()
    for x in (pr.kc, pr.v, pr.kr):
        x.fill_(7)
    mla.mla_prefix_expand(layer(mla, s, "fp32"), pr.cache(mla), 1, pr.W_UK, pr.W_UV, pr.kc, pr.v, pr.kr)
    assert mla.mla_get_device_error() == mla.MLA_OK
    assert pr.kr.equal(want)
    c = pr.prefix[:, :s["d_c"]].double()
    for got, W in ((pr.kc, pr.W_UK), (pr.v, pr.W_UV)):
        w = W.double().view(s["n_h"], s["d_h"], s["d_c"])
        ref, mag = torch.einsum("pc,hdc->hpd", c, w), torch.einsum("pc,hdc->hpd", c.abs(), w.abs())
        # 16 to 30 products per lane and five rounds between lanes
        assert ((got.double() - ref).abs() <= (s["d_c"] / 32 + 6) * 2.0 ** -24 * mag).all()


@pytest.mark.parametrize("P,suffix,n_q,paged", [(192, [70, 200, 71], 70, True), (64, [130], 130, True),
                                                (100, [150, 300], 150, False), (0, [129, 140], 129, True)])
def test_many_new_tokens_per_request(mla, P, suffix, n_q, paged):  # noqa: F811
    """A chunk of every request's own prompt over the shared prefix: causal within the chunk."""
    pr = Problem(V2, "bf16", P, suffix, n_q, 64, paged, seed=n_q)
    o, lse, err = run_shared(mla, pr)
    assert err == mla.MLA_OK
    check(pr, o, lse)


@pytest.mark.parametrize("dtype,tokens,bs", [("bf16", 1000, 64), ("bf16", 200, 128), ("fp32", 77, 16)])
def test_a_prefix_whose_last_page_is_not_full(mla, dtype, tokens, bs):  # noqa: F811
    """Its whole pages are shared and expanded; the tokens after them are the
    beginning of every request's own suffix, cached in a page of its own."""
    import torch
    from tests.gpu_util import ATOL, RTOL
    s = V2 if dtype == "bf16" else dict(n_h=4, d_h=32, d_c=64, d_r=16)
    p = layer(mla, s, dtype)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dt)
    n_h, d_h, d_c, D = s["n_h"], s["d_h"], s["d_c"], s["d_c"] + s["d_r"]
    W_UK, W_UV = normal(n_h * d_h, d_c, std=d_c ** -0.5), normal(n_h * d_h, d_c, std=d_c ** -0.5)
    i32 = dict(dtype=torch.int32, device="cuda")
    B, pages = 5, tokens // bs
    P, rest = pages * bs, tokens % bs
    width, nb = pages + 3, pages + 2 * B
    data = torch.full((nb, bs, D), float("nan"), dtype=dt, device="cuda")
    pool = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    shared, free = pool[:pages].clone(), pool[pages:].contiguous()
    cache = mla.Cache(data, torch.full((B, width), -1, **i32))
    prefix = normal(tokens, D)

    def planned(c, ctx, new, T, free, shared=None):
        n = ctx.numel()
        out = [torch.empty(n, **i32), torch.empty(n + 1, **i32), torch.empty(T, **i32), torch.empty(T, **i32),
               torch.empty(T, dtype=torch.int64, device="cuda"), torch.empty(1, **i32)]
        mla.mla_batch_plan(c, ctx, new, free, *out, shared_blocks=shared)
        return out
    one = mla.Cache(data, torch.full((1, width), -1, **i32))
    plan = planned(one, torch.zeros(1, **i32), torch.full((1,), P, **i32), P, shared)
    mla.mla_cache_write(p, prefix[:P].contiguous(), plan[4], one)
    kc = torch.empty((n_h, P, d_h), dtype=dt, device="cuda")
    v, kr = torch.empty_like(kc), torch.empty((P, s["d_r"]), dtype=dt, device="cuda")
    mla.mla_prefix_expand(p, one, 0, W_UK, W_UV, kc, v, kr)
    # the rest of the prefix and one new token per request, all written by slots
    plan = planned(cache, torch.full((B,), P, **i32), torch.full((B,), rest + 1, **i32), B * (rest + 1), free, shared)
    own = normal(B, 1, D)
    mla.mla_cache_write(p, torch.cat([prefix[P:].expand(B, rest, D), own], dim=1).contiguous().view(-1, D), plan[4], cache)
    assert mla.mla_get_device_error() == mla.MLA_OK and plan[0].tolist() == [tokens + 1] * B
    qa = normal(B, n_h, d_h + s["d_r"])
    o, lse = torch.empty((B, n_h * d_h), dtype=dt, device="cuda"), torch.empty((B, n_h), device="cuda")
    mla.mla_decode_shared(p, qa, kc, v, kr, cache, plan[0], 1, W_UK, W_UV, o, lse)
    assert mla.mla_get_device_error() == mla.MLA_OK
    wk, wv = W_UK.double().view(n_h, d_h, d_c), W_UV.double().view(n_h, d_h, d_c)
    for b in range(B):
        rows = torch.cat([prefix, own[b]]).double()
        k = torch.cat([torch.einsum("nc,hdc->hnd", rows[:, :d_c], wk), rows[None, :, d_c:].expand(n_h, -1, -1)], dim=2)
        sc = torch.einsum("hd,hnd->hn", qa[b].double(), k) / math.sqrt(d_h + s["d_r"])
        ro = torch.einsum("hn,nc,hdc->hd", torch.softmax(sc, dim=1), rows[:, :d_c], wv).reshape(-1)
        rl = torch.logsumexp(sc, dim=1)
        assert ((o[b].double() - ro).abs() <= ATOL + RTOL * ro.abs()).all()
        assert ((lse[b].double() - rl).abs() <= ATOL + RTOL * rl.abs()).all()
