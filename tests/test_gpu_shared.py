"""GPU parity of the shared-prefix calls: mla_prefix_expand (a cached prefix
decompressed once) and mla_decode_shared (order A over the expanded prefix and
order B over each sequence's own positions, as one softmax) against the
definition in 64 bits, and a run of them together with the calls around them.

Tolerances. Every rounding to bf16 is off by at most u = eps / 2 = 2^-8 of the
value. The final rounding and the rounding of the suffix readout are bounded by
u times the value; the roundings that are summed over many terms (P, the latent
readout, the absorbed query) are independent, each with a standard deviation of
at most u / sqrt(3) of its value, and are bounded by six standard deviations of
their sum, formed per output element in 64 bits (6 sigma: 2e-9 per element).
The lse is fp32: the first order of the absorbed query's rounding is corrected,
its second order remains. fp32 sums and exponentials add at most 2e-5."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

V2 = dict(n_h=128, d_h=128, d_c=512, d_r=64)
TINY = dict(n_h=4, d_h=32, d_c=64, d_r=16)
ODD = dict(n_h=3, d_h=40, d_c=70, d_r=6)


@pytest.fixture(scope="module")
def mla():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mla_latent_kv_33_b200 import mla as m
    return m


def layer(mla, s, dtype, scale=0.0):
    return mla.dims(256 if s is not V2 else 5120, s["n_h"], s["d_h"], s["d_c"], 96 if s is not V2 else 1536, s["d_r"],
                    10000.0, scale, dtype)


class Problem:
    """A batch over one prefix: random latents, weights and queries, a paged (or
    contiguous) cache with NaN in every slot that holds no token."""

    def __init__(self, s, dtype, P, suffix, n_q, bs=64, paged=True, seed=0, q_std=1.0, spare_pages=1):
        import torch
        self.s, self.P, self.n_q, self.bs, self.paged = s, P, n_q, bs, paged
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + 17)
        n_h, d_h, d_c, d_r = s["n_h"], s["d_h"], s["d_c"], s["d_r"]

        def normal(shape, std=1.0):
            return (torch.randn(shape, generator=g, device="cuda") * std).to(dt)
        self.lens = [P + x for x in suffix]
        B, D = len(suffix), d_c + d_r
        self.B, self.T = B, B * n_q
        self.W_UK, self.W_UV = normal((n_h * d_h, d_c), d_c ** -0.5), normal((n_h * d_h, d_c), d_c ** -0.5)
        self.qa = normal((self.T, n_h, d_h + d_r), q_std)
        self.prefix = normal((P, D))
        self.suffix = [normal((x, D)) for x in suffix]
        width = max(-(-L // bs) for L in self.lens) + spare_pages
        if paged:
            # the prefix's whole pages are shared; a page it only starts is each sequence's own
            ns = P // bs
            perm = torch.randperm(ns + B * (width - ns), generator=g, device="cuda").to(torch.int32)
            self.data = torch.full((perm.numel(), bs, D), float("nan"), dtype=dt, device="cuda")
            self.table = torch.empty((B, width), dtype=torch.int32, device="cuda")
            self.table[:, :ns] = perm[:ns]
            self.table[:, ns:] = perm[ns:].view(B, width - ns)
        else:
            self.data = torch.full((B, width * bs, D), float("nan"), dtype=dt, device="cuda")
            self.table = None
        for b, L in enumerate(self.lens):
            self.rows(b, torch.arange(L, device="cuda"), torch.cat([self.prefix, self.suffix[b]]))
        self.kc = torch.empty((n_h, P, d_h), dtype=dt, device="cuda")
        self.v, self.kr = torch.empty_like(self.kc), torch.empty((P, d_r), dtype=dt, device="cuda")
        c = self.prefix[:, :d_c].double()
        if P:
            self.kc.copy_(torch.einsum("pc,hdc->hpd", c, self.W_UK.double().view(n_h, d_h, d_c)))
            self.v.copy_(torch.einsum("pc,hdc->hpd", c, self.W_UV.double().view(n_h, d_h, d_c)))
            self.kr.copy_(self.prefix[:, d_c:])
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def rows(self, b, pos, values):
        if self.paged:
            at = self.table[b, pos // self.bs].long() * self.bs + pos % self.bs
        else:
            at = b * self.data.shape[1] + pos
        self.data.view(-1, self.data.shape[-1])[at] = values

    def cache(self, mla):
        return mla.Cache(self.data, self.table)


def reference(pr, scale):
    """(o, lse) in 64 bits and the tolerance of each element (module docstring)."""
    import torch
    s, P, n_q = pr.s, pr.P, pr.n_q
    n_h, d_h, d_c = s["n_h"], s["d_h"], s["d_c"]
    wk, wv = pr.W_UK.double().view(n_h, d_h, d_c), pr.W_UV.double().view(n_h, d_h, d_c)
    kp, vp, rp = pr.kc.double(), pr.v.double(), pr.kr.double()
    tc = s is V2 and pr.qa.dtype == torch.bfloat16
    u = torch.finfo(pr.qa.dtype).eps / 2
    six = 6 * u / math.sqrt(3)
    o = torch.empty((pr.T, n_h, d_h), dtype=torch.float64, device="cuda")
    tol, lse = torch.empty_like(o), torch.empty((pr.T, n_h), dtype=torch.float64, device="cuda")
    ltol = torch.full_like(lse, 2e-5)
    for b, L in enumerate(pr.lens):
        rows = pr.suffix[b].double()
        c, kr = rows[:, :d_c], rows[:, d_c:]
        for j in range(n_q):
            t, n = b * n_q + j, L - P - n_q + 1 + j
            q = pr.qa[t].double()
            q_lat = torch.einsum("hd,hdc->hc", q[:, :d_h], wk)
            sp = torch.einsum("hd,hpd->hp", q[:, :d_h], kp) + q[:, d_h:] @ rp.t()
            ss = q_lat @ c[:n].t() + q[:, d_h:] @ kr[:n].t()
            sc = torch.cat([sp, ss], dim=1) * scale
            lse[t] = torch.logsumexp(sc, dim=1)
            w = torch.exp(sc - lse[t][:, None])
            wp, ws = w[:, :P], w[:, P:]
            lat = ws @ c[:n]                                   # this row's share of the latent readout
            o_s = torch.einsum("hc,hdc->hd", lat, wv)
            o[t] = torch.einsum("hp,hpd->hd", wp, vp) + o_s
            tol[t] = 2e-5 * (1 + o[t].abs()) + u * o[t].abs()
            if tc:
                vs = torch.einsum("nc,hdc->hnd", c[:n], wv)
                tol[t] += u * o_s.abs()                                                        # W_UV readout
                tol[t] += six * torch.einsum("hc,hdc->hd", lat ** 2, wv ** 2).sqrt()           # latent readout
                tol[t] += six * (torch.einsum("hp,hpd->hd", wp ** 2, vp ** 2)                  # P, prefix
                                 + torch.einsum("hn,hnd->hd", ws ** 2, vs ** 2)).sqrt()        # P, suffix
                # the absorbed query: ds_i = scale sum_j dq_j c_ij moves o by sum_i w_i ds_i (v_i - o)
                cov = torch.einsum("hn,nc,hnd->hcd", ws, c[:n], vs) - lat[:, :, None] * o[t][:, None]
                tol[t] += six * scale * torch.einsum("hc,hcd->hd", q_lat ** 2, cov ** 2).sqrt()
                # lse: the first order of ds is added back (with the rounded latent readout); its square is left
                ds = six * scale * ((q_lat ** 2) @ (c[:n] ** 2).t()).amax(dim=1).sqrt()
                ltol[t] += ds ** 2 / 2 + u * ds
    return o.view(pr.T, -1), lse, tol.view(pr.T, -1), ltol


def run_shared(mla, pr, scale=0.0, dtype="bf16", want_lse=True, **kw):
    import torch
    p = layer(mla, pr.s, dtype, scale)
    HD = pr.s["n_h"] * pr.s["d_h"]
    o = torch.full((pr.T + 1, HD), 7.0, dtype=pr.qa.dtype, device="cuda")  # one canary row behind each output
    lse = torch.full((pr.T + 1, pr.s["n_h"]), 7.0, device="cuda")
    before = pr.data.clone()
    mla.mla_decode_shared(p, pr.qa, pr.kc, pr.v, pr.kr, pr.cache(mla), pr.seq_lens, pr.n_q, pr.W_UK, pr.W_UV,
                          o[:-1], lse[:-1] if want_lse else None, **kw)
    err = mla.mla_get_device_error()
    assert (o[-1] == 7).all() and (lse[-1] == 7).all()
    assert torch.equal(pr.data.view(torch.uint8), before.view(torch.uint8))
    return o[:-1], lse[:-1], err


def check(pr, o, lse, scale=None):
    s = scale or 1.0 / math.sqrt(pr.s["d_h"] + pr.s["d_r"])
    ro, rl, tol, ltol = reference(pr, s)
    for what, got, ref, t in (("o", o, ro, tol), ("lse", lse, rl, ltol)):
        err = (got.double() - ref).abs()
        bad = ~(err <= t)
        assert not bad.any(), (what, int(bad.sum()), bad.numel(), float((err / t).nan_to_num(nan=1e9).max()))


CASES = {  # geometry, dtype, P, suffix lengths (new tokens included), n_q, block size, paged
    "one_row_no_prefix": (V2, "bf16", 0, [1], 1, 64, True),
    "one_row_one_block": (V2, "bf16", 64, [1], 1, 64, True),
    "three_rows_one_tile": (V2, "bf16", 128, [1, 64, 65], 1, 64, True),
    "odd_half_tile": (V2, "bf16", 192, [63, 129, 2, 256, 257], 1, 128, True),
    "b33_p640": (V2, "bf16", 640, [1 + 7 * i for i in range(33)], 1, 64, True),
    "b128_p320": (V2, "bf16", 320, [1 + i % 90 for i in range(128)], 1, 64, True),
    "b129_second_row_block": (V2, "bf16", 448, [1 + (5 * i) % 70 for i in range(129)], 1, 64, True),
    "nq2_rows_across_blocks": (V2, "bf16", 256, [2 + (3 * i) % 40 for i in range(70)], 2, 64, True),
    "nq3_no_prefix": (V2, "bf16", 0, [3, 5, 300], 3, 64, True),
    "nq5_b80_three_row_blocks": (V2, "bf16", 128, [5 + i for i in range(80)], 5, 64, True),
    "b2_p4160_many_pieces": (V2, "bf16", 4160, [600, 1], 1, 64, True),
    "contiguous_p100": (V2, "bf16", 100, [1, 33, 400], 1, 64, False),
    "contiguous_nq2_p129": (V2, "bf16", 129, [2, 70], 2, 64, False),
    "tiny_fp32": (TINY, "fp32", 700, [1, 5, 90], 1, 16, True),
    "tiny_fp32_nq4_p0": (TINY, "fp32", 0, [4, 40], 4, 16, True),
    "tiny_bf16_p257": (TINY, "bf16", 257, [300, 1], 1, 16, True),
    "odd_dims_fp32_contiguous": (ODD, "fp32", 31, [2, 30], 2, 5, False),
    "odd_dims_fp32_pages_of_5": (ODD, "fp32", 33, [3, 300], 3, 5, True),
}


@pytest.mark.parametrize("case", list(CASES))
def test_shared_decode_matches_its_definition(mla, case):
    s, dtype, P, suffix, n_q, bs, paged = CASES[case]
    pr = Problem(s, dtype, P, suffix, n_q, bs, paged, seed=len(case))
    o, lse, err = run_shared(mla, pr, dtype=dtype)
    assert err == mla.MLA_OK
    check(pr, o, lse)


def test_large_scores_force_the_accumulator_rescale(mla):
    """Queries six times wider: scores of standard deviation 6, so that running
    maxima grow by more than 2^8 between tiles."""
    pr = Problem(V2, "bf16", 1344, [40, 1, 300, 7, 90], 1, seed=3, q_std=6.0)
    o, lse, err = run_shared(mla, pr)
    assert err == mla.MLA_OK
    check(pr, o, lse)


def test_given_scale_and_no_lse(mla):
    pr = Problem(V2, "bf16", 192, [9, 70], 1, seed=4)
    o, lse, err = run_shared(mla, pr, scale=0.02)
    assert err == mla.MLA_OK
    check(pr, o, lse, scale=float(np.float32(0.02)))
    o2, untouched, err = run_shared(mla, pr, scale=0.02, want_lse=False)
    assert err == mla.MLA_OK and (untouched == 7).all() and o2.equal(o)


@pytest.mark.parametrize("case", ["b33_p640", "nq2_rows_across_blocks", "tiny_fp32"])
def test_prefix_pages_of_the_table_are_not_read(mla, case):
    s, dtype, P, suffix, n_q, bs, paged = CASES[case]
    pr = Problem(s, dtype, P, suffix, n_q, bs, paged, seed=5)
    ref = run_shared(mla, pr, dtype=dtype)
    pr.table[:, :P // bs] = -5
    got = run_shared(mla, pr, dtype=dtype)
    assert got[2] == ref[2] == mla.MLA_OK
    assert got[0].equal(ref[0]) and got[1].equal(ref[1])


@pytest.mark.parametrize("s,dtype", [(V2, "bf16"), (TINY, "fp32")])
def test_bad_lengths_leave_their_rows_unwritten(mla, s, dtype):
    import torch
    pr = Problem(s, dtype, 128, [3, 40, 9, 70, 5], 2, 64, seed=6)
    good = run_shared(mla, pr, dtype=dtype)
    assert good[2] == mla.MLA_OK
    cap = pr.table.shape[1] * 64
    pr.seq_lens.copy_(torch.tensor([128 + 1, 168, cap + 1, 198, -2 ** 31], dtype=torch.int32))
    o, lse, err = run_shared(mla, pr, dtype=dtype)
    assert err == mla.MLA_ERR_DEVICE_DATA
    for b in range(5):
        rows = slice(2 * b, 2 * b + 2)
        if b in (1, 3):
            assert torch.allclose(o[rows].float(), good[0][rows].float(), atol=1e-2, rtol=1e-2)
        else:
            assert (o[rows] == 7).all() and (lse[rows] == 7).all()
    assert mla.mla_get_device_error() == mla.MLA_OK


def test_bad_suffix_page_is_reported(mla):
    pr = Problem(V2, "bf16", 128, [70, 3], 1, seed=8)
    pr.table[0, 3] = pr.data.shape[0]
    _, _, err = run_shared(mla, pr)
    assert err == mla.MLA_ERR_DEVICE_DATA


@pytest.mark.parametrize("overlap", [False, True])
def test_two_streams_graphs_and_repeats_are_bit_equal(mla, overlap):
    """Same inputs, several ways of calling: eager, eager again, captured and
    replayed, and two calls at once on two streams with a workspace each."""
    import torch
    prs = [Problem(V2, "bf16", 448, [1 + 9 * i for i in range(20)], 1, seed=9),
           Problem(V2, "bf16", 960, [2 + 5 * i for i in range(11)], 2, seed=10)]
    p = layer(mla, V2, "bf16")
    was = mla.get_launch_overlap()
    mla.set_launch_overlap(overlap)
    try:
        first = [run_shared(mla, pr)[:2] for pr in prs]
        again = [run_shared(mla, pr)[:2] for pr in prs]
        outs, graphs, ws, caches = [], [], [], []
        for pr in prs:
            outs.append((torch.zeros((pr.T, 16384), dtype=torch.bfloat16, device="cuda"),
                         torch.zeros((pr.T, 128), device="cuda")))
            ws.append(torch.empty(mla.workspace_size(p, mla.OP_DECODE_SHARED, pr.B, pr.n_q, pr.P), dtype=torch.uint8,
                                  device="cuda"))
            caches.append(pr.cache(mla))

        def call(i, stream=None):
            pr = prs[i]
            mla.mla_decode_shared(p, pr.qa, pr.kc, pr.v, pr.kr, caches[i], pr.seq_lens, pr.n_q, pr.W_UK, pr.W_UV,
                                  *outs[i], ws=ws[i], stream=stream)
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for _ in range(3):
            for i, st in enumerate(streams):
                call(i, st)
        torch.cuda.synchronize()
        for i in range(2):
            assert all(a.equal(b) and a.equal(c) for a, b, c in zip(first[i], again[i], outs[i]))
        for i in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                call(i)
            graphs.append(g)
        for i in range(2):
            outs[i][0].zero_()
        for g in graphs + graphs:
            g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert all(a.equal(b) for a, b in zip(first[i], outs[i]))
        assert mla.mla_get_device_error() == mla.MLA_OK
    finally:
        mla.set_launch_overlap(was)


def test_own_workspace_on_a_side_stream(mla):
    """Without a workspace argument the call makes its own, which the allocator
    must not hand out again while the side stream still uses it."""
    import torch
    pr = Problem(V2, "bf16", 1920, [200 + i for i in range(40)], 1, seed=14)
    want, _, err = run_shared(mla, pr)
    assert err == mla.MLA_OK
    p, c, side = layer(mla, V2, "bf16"), pr.cache(mla), torch.cuda.Stream()
    nbytes = mla.workspace_size(p, mla.OP_DECODE_SHARED, pr.B, 1, pr.P)
    outs = [torch.zeros((pr.T, 16384), dtype=torch.bfloat16, device="cuda") for _ in range(6)]
    torch.cuda.synchronize()
    for o in outs:
        mla.mla_decode_shared(p, pr.qa, pr.kc, pr.v, pr.kr, c, pr.seq_lens, 1, pr.W_UK, pr.W_UV, o, stream=side)
        torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")  # would land in a freed workspace
    torch.cuda.synchronize()
    assert all(o.equal(want) for o in outs)


def test_outputs_that_are_only_16_byte_aligned(mla):
    import torch
    pr = Problem(V2, "bf16", 320, [30, 700, 1], 1, seed=15)
    p, c = layer(mla, V2, "bf16"), pr.cache(mla)

    def off16(x):  # same shape, its first element 16 bytes past a 256-byte boundary
        n = 16 // x.element_size()
        return torch.zeros(x.numel() + n, dtype=x.dtype, device="cuda")[n:].view(x.shape)
    kc, v, kr = off16(pr.kc), off16(pr.v), off16(pr.kr)
    ref = [torch.zeros_like(x) for x in (pr.kc, pr.v, pr.kr)]
    mla.mla_prefix_expand(p, c, 0, pr.W_UK, pr.W_UV, *ref)
    mla.mla_prefix_expand(p, c, 0, pr.W_UK, pr.W_UV, kc, v, kr)
    assert kc.equal(ref[0]) and v.equal(ref[1]) and kr.equal(ref[2])
    want, want_lse, err = run_shared(mla, pr)
    o = off16(want)
    ws = torch.empty(mla.workspace_size(p, mla.OP_DECODE_SHARED, 3, 1, 320) + 16, dtype=torch.uint8, device="cuda")[16:]
    mla.mla_decode_shared(p, off16(pr.qa).copy_(pr.qa), off16(kc).copy_(pr.kc), off16(v).copy_(pr.v),
                          off16(kr).copy_(pr.kr), c, pr.seq_lens, 1, off16(pr.W_UK).copy_(pr.W_UK),
                          off16(pr.W_UV).copy_(pr.W_UV), o, ws=ws)
    assert err == mla.mla_get_device_error() == mla.MLA_OK and o.equal(want)
    # the ordinary decode's latent readout, split rows and whole ones
    q = torch.randn((3, 128, 576), device="cuda").to(torch.bfloat16)
    a = torch.zeros((3, 128, 512), dtype=torch.bfloat16, device="cuda")
    b = off16(a)
    for splits in (0, 1, 3):
        mla.mla_decode(p, q, c, pr.seq_lens, 1, a, num_splits=splits)
        mla.mla_decode(p, q, c, pr.seq_lens, 1, b, num_splits=splits)
        assert mla.mla_get_device_error() == mla.MLA_OK and a.equal(b)


# ---------------------------------------------------------------- expansion --

EXPANDS = {  # geometry, dtype, P, block size, paged
    "one_token": (V2, "bf16", 1, 64, True),
    "p63": (V2, "bf16", 63, 64, True),
    "p64": (V2, "bf16", 64, 64, True),
    "p130_bs128": (V2, "bf16", 130, 128, True),
    "p257": (V2, "bf16", 257, 64, True),
    "p1000": (V2, "bf16", 1000, 64, True),
    "contiguous_p300": (V2, "bf16", 300, 64, False),
    "tiny_fp32_p17": (TINY, "fp32", 17, 16, True),
    "tiny_bf16_p33": (TINY, "bf16", 33, 16, True),
    "odd_fp32_p6": (ODD, "fp32", 6, 5, False),
}


@pytest.mark.parametrize("case", list(EXPANDS))
def test_expansion_matches_its_definition(mla, case):
    import torch
    s, dtype, P, bs, paged = EXPANDS[case]
    pr = Problem(s, dtype, P, [1, 70, 2], 1, bs, paged, seed=len(case))
    n_h, d_h, d_c = s["n_h"], s["d_h"], s["d_c"]

    def padded(x):  # a canary behind the output
        return torch.full((x.numel() + 8,), 7.0, dtype=x.dtype, device="cuda")
    outs = [padded(x) for x in (pr.kc, pr.v, pr.kr)]
    kc, v, kr = (o[:-8].view(x.shape) for o, x in zip(outs, (pr.kc, pr.v, pr.kr)))
    mla.mla_prefix_expand(layer(mla, s, dtype), pr.cache(mla), 1, pr.W_UK, pr.W_UV, kc, v, kr)
    assert mla.mla_get_device_error() == mla.MLA_OK
    assert all((o[-8:] == 7).all() for o in outs)
    assert kr.equal(pr.prefix[:, d_c:])
    c = pr.prefix[:, :d_c].double()
    u = torch.finfo(kc.dtype).eps / 2
    for got, W in ((kc, pr.W_UK), (v, pr.W_UV)):
        w = W.double().view(n_h, d_h, d_c)
        ref, mag = torch.einsum("pc,hdc->hpd", c, w), torch.einsum("pc,hdc->hpd", c.abs(), w.abs())
        # one rounding, and fp32 sums of d_c products (each partial sum rounded by at most 2^-24 of its size)
        assert ((got.double() - ref).abs() <= u * ref.abs() * (1 + 1e-3) + d_c * 2.0 ** -24 * mag).all()


def test_expansion_of_a_bad_page_is_reported_and_zero(mla):
    pr = Problem(V2, "bf16", 300, [5, 9], 1, seed=12)
    pr.table[0, 1] = -1
    mla.mla_prefix_expand(layer(mla, V2, "bf16"), pr.cache(mla), 0, pr.W_UK, pr.W_UV, pr.kc, pr.v, pr.kr)
    assert mla.mla_get_device_error() == mla.MLA_ERR_DEVICE_DATA
    assert (pr.kc[:, 64:128] == 0).all() and (pr.v[:, 64:128] == 0).all() and (pr.kr[64:128] == 0).all()
    assert (pr.kc[:, 128:] != 0).any(dim=2).all()


# -------------------------------------------------------- a step, all of it --

@pytest.mark.parametrize("B,n_q,pages,bs", [(9, 1, 5, 64), (70, 2, 3, 128)])
def test_serving_steps_with_a_shared_prefix(mla, B, n_q, pages, bs):
    """Two steps as a serving program makes them: plan, append, per-head
    queries, shared decode; the prefix written by slots and expanded once. The
    result equals the ordinary decode and W_UV readout over the same tables."""
    import torch
    from tests.gpu_util import ATOL, RTOL
    p = mla.dims(512, 128, 128, 512, 192, 64)
    g = torch.Generator(device="cuda")
    g.manual_seed(B)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)
    W = {k: normal(m, n, std=n ** -0.5) for k, (m, n) in dict(
        W_DKV=(512, 512), W_KR=(64, 512), W_DQ=(192, 512), W_UQ=(16384, 192), W_QR=(8192, 192), W_UK=(16384, 512),
        W_UV=(16384, 512)).items()}
    P, width = pages * bs, pages + 4
    num_blocks = pages + B * 3
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.full((B, width), -1, **i32)
    data = torch.full((num_blocks, bs, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    cache = mla.Cache(data, table)
    pool = torch.randperm(num_blocks, generator=g, device="cuda").to(torch.int32)
    shared, free = pool[:pages].clone(), pool[pages:]
    kc = torch.empty((128, P, 128), dtype=torch.bfloat16, device="cuda")
    v, kr = torch.empty_like(kc), torch.empty((P, 64), dtype=torch.bfloat16, device="cuda")
    # the prefix, as a request of its own: rows from elsewhere, written by slot, expanded
    one = mla.Cache(data, torch.full((1, width), -1, **i32))
    plan = [torch.empty(n, **i32) for n in (1, 2, P, P)] + [torch.empty(P, dtype=torch.int64, device="cuda"),
                                                            torch.empty(1, **i32)]
    mla.mla_batch_plan(one, torch.zeros(1, **i32), torch.full((1,), P, **i32), shared, *plan)
    mla.mla_cache_write(p, normal(P, 576), plan[4], one)
    mla.mla_prefix_expand(p, one, 0, W["W_UK"], W["W_UV"], kc, v, kr)
    ctx, T = torch.full((B,), P, **i32), B * n_q
    new = torch.full((B,), n_q, **i32)
    for step in range(2):
        seq_lens, row_start, used = torch.empty(B, **i32), torch.empty(B + 1, **i32), torch.empty(1, **i32)
        seq_idx, pos = torch.empty(T, **i32), torch.empty(T, **i32)
        slots = torch.empty(T, dtype=torch.int64, device="cuda")
        mla.mla_batch_plan(cache, ctx, new, free, seq_lens, row_start, seq_idx, pos, slots, used, shared_blocks=shared)
        h = normal(T, 512)
        mla.mla_cache_append(p, h, W["W_DKV"], W["W_KR"], seq_idx, pos, cache)
        qa = torch.empty((T, 128, 192), dtype=torch.bfloat16, device="cuda")
        mla.mla_query_heads(p, h, W["W_DQ"], W["W_UQ"], W["W_QR"], pos, qa)
        o = torch.empty((T, 16384), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((T, 128), device="cuda")
        mla.mla_decode_shared(p, qa, kc, v, kr, cache, seq_lens, n_q, W["W_UK"], W["W_UV"], o, lse)
        assert mla.mla_get_device_error() == mla.MLA_OK
        assert seq_lens.tolist() == [P + n_q * (step + 1)] * B and row_start[-1] == T
        # the ordinary path over the same tables
        q = torch.empty((T, 128, 576), dtype=torch.bfloat16, device="cuda")
        mla.mla_absorb_q(p, h, W["W_DQ"], W["W_UQ"], W["W_QR"], W["W_UK"], pos, q)
        o_lat, lse2 = torch.empty((T, 128, 512), dtype=torch.bfloat16, device="cuda"), torch.empty_like(lse)
        mla.mla_decode(p, q, cache, seq_lens, n_q, o_lat, lse2)
        o2 = torch.empty_like(o)
        mla.mla_out_proj(p, o_lat, W["W_UV"], o2)
        assert mla.mla_get_device_error() == mla.MLA_OK
        # each path is within the tolerance of the exact result
        err = (o.double() - o2.double()).abs()
        assert (err <= 2 * (ATOL + RTOL * o2.double().abs())).all()
        assert ((lse - lse2).abs() <= 2 * (ATOL + RTOL * lse2.abs())).all()
        ctx, free = seq_lens.clone(), free[int(used):].contiguous()
