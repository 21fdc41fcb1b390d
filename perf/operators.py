"""Measured cases of the shared-prefix serving operators.

One decode step of a batch whose requests all start with the same long prefix
(a system prompt, a document, few-shot examples) takes four operators next to
the projections:

  plan    mla_batch_plan: block tables, slot maps, sequence ids, positions and
          lengths, built on the GPU from the requests' lengths.
  write   mla_cache_write: ready latent rows ([c_KV | k_R]) scattered into the
          paged cache by a slot map.
  expand  mla_prefix_expand: the prefix decompressed once into per-head keys
          K_C = W_UK c_KV, values V = W_UV c_KV and the shared k_R.
  shared  mla_decode_shared: attention of every new token over the expanded
          prefix (read once for the whole batch) and over its own suffix of
          the latent cache, as one softmax.

Each case is run in a plain form (elementary torch operations, 32-bit, rounded
once) or, with ``own`` set, through the framework's calls. ``exact`` gives the
same outputs from the definition in 64 bits.
"""
import math

import torch

own = False

# DeepSeek-V2/V3 head geometry, and the small fp32 layer of the workload table
GEOMETRY = {
    "v2": dict(n_h=128, d_h=128, d_c=512, d_r=64),
    "tiny": dict(n_h=4, d_h=32, d_c=64, d_r=16),
}
D_MODEL = {"v2": (5120, 1536), "tiny": (256, 96)}  # (d, d_cq): named by the dims, not read here
DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # the table update of one decode step: 64 requests, contexts U[1024, 8192], one token each
        dict(name="plan_step_b64", op="plan", B=64, ctx_lo=1024, ctx_hi=8192, chunk=1, prompts=0, block_size=64,
             shared=16, pad=0),
        # a mixed step: 1024 requests, half of them with a prompt chunk of up to 128 tokens, padded row buffers
        dict(name="plan_mixed_b1024", op="plan", B=1024, ctx_lo=0, ctx_hi=4096, chunk=128, prompts=512,
             block_size=128, shared=4, pad=100),
        # the new rows of a decode step that were computed elsewhere
        dict(name="write_step_t64", op="write", geo="v2", dtype="bf16", T=64, blocks=16, block_size=64, pad=0),
        # a transferred prompt: 12289 rows, some of them padding
        dict(name="write_prompt_t12289", op="write", geo="v2", dtype="bf16", T=12289, blocks=512, block_size=64,
             pad=97),
        # a short system prompt whose last page is not full
        dict(name="expand_p1000", op="expand", geo="v2", dtype="bf16", P=1000, block_size=64),
        # a long document
        dict(name="expand_p8192", op="expand", geo="v2", dtype="bf16", P=8192, block_size=64),
        # latency: a few requests over a short prompt
        dict(name="shared_b4_p512", op="shared", geo="v2", dtype="bf16", B=4, n_q=1, P=512, suf_lo=1, suf_hi=64,
             block_size=64),
        # an ordinary serving batch
        dict(name="shared_b64_p4096", op="shared", geo="v2", dtype="bf16", B=64, n_q=1, P=4096, suf_lo=1,
             suf_hi=1024, block_size=64),
        # a larger batch over a longer prompt
        dict(name="shared_b128_p8192", op="shared", geo="v2", dtype="bf16", B=128, n_q=1, P=8192, suf_lo=1,
             suf_hi=1024, block_size=64),
        # the largest: 256 requests over one long document
        dict(name="shared_b256_p16384", op="shared", geo="v2", dtype="bf16", B=256, n_q=1, P=16384, suf_lo=1,
             suf_hi=512, block_size=64),
        # two new tokens per request (speculative step), prefix not a multiple of the key tile
        dict(name="shared_b100_nq2_p2112", op="shared", geo="v2", dtype="bf16", B=100, n_q=2, P=2112, suf_lo=2,
             suf_hi=500, block_size=128),
        # fp32 storage, small layer
        dict(name="shared_fp32_b8_p700", op="shared", geo="tiny", dtype="fp32", B=8, n_q=1, P=700, suf_lo=1,
             suf_hi=90, block_size=16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "write", "expand", "shared", "shared"])
    if op == "plan":
        B = _log_int(rng, 1, 1024)
        chunk = _log_int(rng, 1, 511)
        ctx_lo = rng.choice([0, 1, 64, 512])
        return dict(op=op, B=B, ctx_lo=ctx_lo, ctx_hi=ctx_lo + _log_int(rng, 1, 8192), chunk=chunk,
                    prompts=rng.randint(0, B) if B * chunk <= 1 << 17 else 0, block_size=rng.choice([16, 64, 128]),
                    shared=rng.choice([0, 0, 1, 4, 16]), pad=rng.choice([0, 0, 1, 77]))
    if op == "write":
        geo, dtype = rng.choice([("v2", "bf16"), ("v2", "bf16"), ("v2", "fp32"), ("tiny", "bf16"), ("tiny", "fp32")])
        T = _log_int(rng, 1, 12289 if dtype == "bf16" else 6001)
        block_size = rng.choice([16, 64, 128])
        return dict(op=op, geo=geo, dtype=dtype, T=T, blocks=(T + rng.randint(0, T) + block_size) // block_size,
                    block_size=block_size, pad=rng.choice([0, 0, 1, 33]) if T > 64 else 0)
    if op == "expand":
        if rng.random() < 0.2:
            return dict(op=op, geo="tiny", dtype=rng.choice(["fp32", "bf16"]), P=_log_int(rng, 1, 2000), block_size=16)
        return dict(op=op, geo="v2", dtype="bf16", P=_log_int(rng, 1, 8192), block_size=rng.choice([64, 128]))
    n_q = rng.choice([1, 1, 1, 2, 3])
    if rng.random() < 0.15:
        return dict(op=op, geo="tiny", dtype=rng.choice(["fp32", "bf16"]), B=_log_int(rng, 1, 16), n_q=n_q,
                    P=rng.randint(0, 900), suf_lo=n_q, suf_hi=n_q + rng.randint(0, 100), block_size=16)
    B = _log_int(rng, 1, 256 // n_q)
    # the prefix ends on a 64-token block; the cost of the largest listed case bounds it
    P = 64 * _log_int(rng, 1, max(1, min(256, 256 * 16384 // (64 * B * n_q))))
    block_size = rng.choice([64, 128])
    suf_hi = n_q + _log_int(rng, 1, max(1, min(2048, 65536 // (B * n_q))))
    return dict(op=op, geo="v2", dtype="bf16", B=B, n_q=n_q, P=P, suf_lo=n_q, suf_hi=suf_hi, block_size=block_size)


# ------------------------------------------------------------------ inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(0x51A7ED + 7919 * int(seed))
    return g


def _normal(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _dims(case):
    """The framework's description of the layer (framework runs only)."""
    from mla_latent_kv_33_b200 import mla
    d, d_cq = D_MODEL[case["geo"]]
    s = GEOMETRY[case["geo"]]
    return mla.dims(d, s["n_h"], s["d_h"], s["d_c"], d_cq, s["d_r"], 10000.0, 0.0, case["dtype"])


def _plan_lengths(case, g):
    B, bs = case["B"], case["block_size"]
    lo = max(case["ctx_lo"], case["shared"] * bs)
    ctx = torch.randint(lo, max(lo, case["ctx_hi"]) + 1, (B,), generator=g, device="cuda")
    new = torch.ones(B, dtype=torch.int64, device="cuda")
    if case["prompts"]:
        who = torch.randperm(B, generator=g, device="cuda")[:case["prompts"]]
        new[who] = torch.randint(0, case["chunk"] + 1, (case["prompts"],), generator=g, device="cuda")
    return ctx, new


def _prepare_plan(case, seed):
    g = _gen(seed)
    B, bs, shared = case["B"], case["block_size"], case["shared"]
    ctx, new = _plan_lengths(case, g)
    width = (max(case["ctx_hi"], shared * bs) + case["chunk"]) // bs + 2
    held = (ctx + bs - 1) // bs  # entries a request already has, the shared ones among them
    # row buffers and free list are sized once, for the fullest step of this shape
    T = B - case["prompts"] + case["prompts"] * case["chunk"] + case["pad"]
    spare = B - case["prompts"] + case["prompts"] * (case["chunk"] // bs + 1)
    pool = torch.randperm(shared + int((held - shared).sum()) + spare, generator=g, device="cuda").to(torch.int32)
    num_blocks = pool.numel()
    table = torch.full((B, width), -7, dtype=torch.int32, device="cuda")
    col = torch.arange(width, device="cuda")
    own_part = (col[None] >= shared) & (col[None] < held[:, None])
    table[own_part] = pool[shared:shared + int(own_part.sum())]
    z = dict(dtype=torch.int32, device="cuda")
    st = dict(op="plan", bs=bs, num_blocks=num_blocks, ctx=ctx.int(), new=new.int(),
              shared=pool[:shared].clone(), free=pool[num_blocks - spare:].clone(), table=table,
              seq_lens=torch.zeros(B, **z), row_start=torch.zeros(B + 1, **z), seq_idx=torch.zeros(T, **z),
              positions=torch.zeros(T, **z), slots=torch.zeros(T, dtype=torch.int64, device="cuda"),
              used=torch.zeros(1, **z))
    if own:
        from mla_latent_kv_33_b200 import mla
        # the plan needs the cache's page geometry and table; the pages themselves are not touched
        st["cache"] = mla.Cache(torch.empty((num_blocks, bs, 1), dtype=torch.bfloat16, device="cuda"), table)
    return st


def _prepare_write(case, seed):
    g = _gen(seed)
    s, dt = GEOMETRY[case["geo"]], DTYPE[case["dtype"]]
    D = s["d_c"] + s["d_r"]
    N = case["blocks"] * case["block_size"]
    slots = torch.randperm(N, generator=g, device="cuda")[:case["T"]].clone()
    if case["pad"]:
        slots[torch.randperm(case["T"], generator=g, device="cuda")[:case["pad"]]] = -1
    st = dict(op="write", rows=_normal(g, (case["T"], D), 1.0, dt), slots=slots,
              data=_normal(g, (case["blocks"], case["block_size"], D), 1.0, dt))
    if own:
        from mla_latent_kv_33_b200 import mla
        table = torch.arange(case["blocks"], dtype=torch.int32, device="cuda")[None].contiguous()
        st["p"], st["cache"] = _dims(case), mla.Cache(st["data"], table)
    return st


def _paged(g, case, s, dt, lens, shared_rows):
    """A paged pool and its table: every sequence starts with the blocks that hold
    shared_rows [P][D] (whole blocks of them are shared; the rows of a last, partial
    block are copied into each sequence's own block), followed by N(0, 1) rows up to
    its length. Slots that hold no token are NaN."""
    D, bs, B = s["d_c"] + s["d_r"], case["block_size"], len(lens)
    P = shared_rows.shape[0]
    nshared = P // bs
    width = max((max(lens) + bs - 1) // bs, 1)
    own_blocks = [(L + bs - 1) // bs - nshared for L in lens]
    total = nshared + sum(own_blocks)
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    data = torch.full((total, bs, D), float("nan"), dtype=dt, device="cuda")
    table[:, :nshared] = perm[:nshared]
    data[perm[:nshared].long()] = shared_rows[:nshared * bs].view(nshared, bs, D)
    at = nshared
    flat = data.view(-1, D)
    off = torch.arange(bs, device="cuda")
    for b, L in enumerate(lens):
        blk = perm[at:at + own_blocks[b]]
        table[b, nshared:nshared + own_blocks[b]] = blk
        at += own_blocks[b]
        rows = (blk.long()[:, None] * bs + off).view(-1)[:L - nshared * bs]
        tail = P - nshared * bs
        if rows.numel():
            fresh = _normal(g, (rows.numel(), D), 1.0, dt)
            fresh[:tail] = shared_rows[nshared * bs:]
            flat[rows] = fresh
    return data, table


def _prepare_expand(case, seed):
    g = _gen(seed)
    s, dt = GEOMETRY[case["geo"]], DTYPE[case["dtype"]]
    P = case["P"]
    HD = s["n_h"] * s["d_h"]
    W_UK = _normal(g, (HD, s["d_c"]), s["d_c"] ** -0.5, dt)
    W_UV = _normal(g, (HD, s["d_c"]), s["d_c"] ** -0.5, dt)
    none = torch.empty((0, s["d_c"] + s["d_r"]), dtype=dt, device="cuda")
    data, table = _paged(g, case, s, dt, [max(1, P // 3), P], none)  # the prefix is sequence 1
    st = dict(op="expand", s=s, P=P, bs=case["block_size"], data=data, table=table, W_UK=W_UK, W_UV=W_UV,
              kc=torch.empty((s["n_h"], P, s["d_h"]), dtype=dt, device="cuda"),
              v=torch.empty((s["n_h"], P, s["d_h"]), dtype=dt, device="cuda"),
              kr=torch.empty((P, s["d_r"]), dtype=dt, device="cuda"))
    if own:
        from mla_latent_kv_33_b200 import mla
        st["p"], st["cache"] = _dims(case), mla.Cache(data, table)
    return st


def _prepare_shared(case, seed):
    g = _gen(seed)
    s, dt = GEOMETRY[case["geo"]], DTYPE[case["dtype"]]
    n_h, d_h, d_c, d_r = s["n_h"], s["d_h"], s["d_c"], s["d_r"]
    B, n_q, P = case["B"], case["n_q"], case["P"]
    T = B * n_q
    W_UK = _normal(g, (n_h * d_h, d_c), d_c ** -0.5, dt)
    W_UV = _normal(g, (n_h * d_h, d_c), d_c ** -0.5, dt)
    suf = torch.randint(case["suf_lo"], case["suf_hi"] + 1, (B,), generator=g, device="cuda").tolist()
    lens = [P + x for x in suf]
    prefix = _normal(g, (P, d_c + d_r), 1.0, dt)
    data, table = _paged(g, case, s, dt, lens, prefix)
    # the prefix as the expansion lays it out: per-head keys and values, one RoPE key
    c = prefix[:, :d_c].float()
    kc = torch.matmul(c, W_UK.float().view(n_h, d_h, d_c).transpose(1, 2)).to(dt)
    v = torch.matmul(c, W_UV.float().view(n_h, d_h, d_c).transpose(1, 2)).to(dt)
    st = dict(op="shared", s=s, n_q=n_q, P=P, bs=case["block_size"], lens=lens, data=data, table=table, W_UK=W_UK,
              W_UV=W_UV, kc=kc, v=v, kr=prefix[:, d_c:].contiguous(),
              seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
              qa=_normal(g, (T, n_h, d_h + d_r), 1.0, dt),
              o=torch.empty((T, n_h * d_h), dtype=dt, device="cuda"),
              lse=torch.empty((T, n_h), dtype=torch.float32, device="cuda"))
    if own:
        from mla_latent_kv_33_b200 import mla
        st["p"], st["cache"] = _dims(case), mla.Cache(data, table)
        need = mla.workspace_size(st["p"], mla.OP_DECODE_SHARED, B, n_q, P)
        st["ws"] = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    return st


def prepare(case, seed):
    return {"plan": _prepare_plan, "write": _prepare_write, "expand": _prepare_expand,
            "shared": _prepare_shared}[case["op"]](case, seed)


# --------------------------------------------------------- one pass, plain --

def _plain_plan(st):
    bs, table, T = st["bs"], st["table"], st["seq_idx"].numel()
    B, width = table.shape
    ctx, new = st["ctx"].long(), st["new"].long()
    seq = ctx + new
    held = (ctx + bs - 1) // bs
    need = (seq + bs - 1) // bs - held
    first = torch.cumsum(need, 0) - need
    start = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0)])
    col = torch.arange(width, device=table.device)[None]
    k = col - held[:, None]
    fresh = (k >= 0) & (k < need[:, None])
    pick = st["free"][(first[:, None] + k).clamp(0, st["free"].numel() - 1)]
    nshared = st["shared"].numel()
    upd = torch.where(fresh, pick, table)
    if nshared:
        upd[:, :nshared] = st["shared"]
    table.copy_(upd)
    t = torch.arange(T, device=table.device)
    b = torch.searchsorted(start[1:].contiguous(), t, right=True).clamp(max=B - 1)
    pad = t >= start[-1]
    pos = torch.where(pad, 0, ctx[b] + t - start[b])
    slot = table[b, (pos // bs).clamp(max=width - 1)].long() * bs + pos % bs
    return dict(table=table, seq_lens=seq.int(), row_start=start.int(), seq_idx=torch.where(pad, -1, b).int(),
                positions=pos.int(), slots=torch.where(pad, -1, slot), used=need.sum().int().view(1))


def _plain_write(st):
    rows, slots = st["rows"], st["slots"]
    flat = st["data"].view(-1, rows.shape[1])
    # padding rows repeat the row of the largest slot, so that no row count reaches the host
    i = slots.argmax()
    pad = slots < 0
    flat.index_copy_(0, torch.where(pad, slots[i], slots), torch.where(pad[:, None], rows[i], rows))
    return st["data"]


def _rows_of(st, b, lo, hi):
    """Cache rows of positions lo .. hi - 1 of sequence b, in 32 bits."""
    pos = torch.arange(lo, hi, device="cuda")
    blk = st["table"][b, pos // st["bs"]].long()
    return st["data"].view(-1, st["data"].shape[-1])[blk * st["bs"] + pos % st["bs"]].float()


def _plain_expand(st):
    s = st["s"]
    rows = _rows_of(st, 1, 0, st["P"])
    c, dt = rows[:, :s["d_c"]], st["W_UK"].dtype
    heads = (s["n_h"], s["d_h"], s["d_c"])
    return (torch.matmul(c, st["W_UK"].float().view(heads).transpose(1, 2)).to(dt),
            torch.matmul(c, st["W_UV"].float().view(heads).transpose(1, 2)).to(dt), rows[:, s["d_c"]:].to(dt))


def _plain_shared(st):
    s, n_q, P = st["s"], st["n_q"], st["P"]
    n_h, d_h, d_c, d_r = s["n_h"], s["d_h"], s["d_c"], s["d_r"]
    qa = st["qa"].float()
    T, dt = qa.shape[0], st["qa"].dtype
    scale = 1.0 / math.sqrt(d_h + d_r)
    W_UK, W_UV = st["W_UK"].float().view(n_h, d_h, d_c), st["W_UV"].float().view(n_h, d_h, d_c)
    # prefix: per-head keys and values, all token rows at once
    q = qa.transpose(0, 1)  # [n_h][T][d_h + d_r]
    sp = torch.matmul(q[:, :, :d_h], st["kc"].float().transpose(1, 2))
    sp += torch.matmul(q[:, :, d_h:], st["kr"].float().t())
    sp *= scale
    m_p = sp.amax(dim=2) if P else torch.full((n_h, T), -math.inf, device="cuda")
    # suffix: absorbed queries against each sequence's latent rows
    q_lat = torch.matmul(q[:, :, :d_h], W_UK)
    qf = torch.cat([q_lat, q[:, :, d_h:]], dim=2)  # [n_h][T][d_c + d_r]
    m_s, l_s = torch.empty((n_h, T), device="cuda"), torch.empty((n_h, T), device="cuda")
    o_s = torch.empty((n_h, T, d_c), device="cuda")
    for b, L in enumerate(st["lens"]):
        rows = _rows_of(st, b, P, L)
        t = slice(b * n_q, (b + 1) * n_q)
        ss = torch.matmul(qf[:, t], rows.t()) * scale  # [n_h][n_q][L - P]
        if n_q > 1:  # new token j sits at position L - n_q + j
            j = torch.arange(n_q, device="cuda")[:, None]
            ss = ss.masked_fill(torch.arange(P, L, device="cuda")[None] > L - n_q + j, -math.inf)
        m = ss.amax(dim=2)
        e = torch.exp(ss - m[:, :, None])
        m_s[:, t], l_s[:, t] = m, e.sum(dim=2)
        o_s[:, t] = torch.matmul(e, rows[:, :d_c])
    m = torch.maximum(m_p, m_s)
    a_s = torch.exp(m_s - m)
    l = l_s * a_s
    o = torch.matmul(o_s * a_s[:, :, None], W_UV.transpose(1, 2))
    if P:
        sp -= m[:, :, None]
        e = sp.exp_()
        l = l + e.sum(dim=2)
        o = o + torch.matmul(e, st["v"].float())
    o = o / l[:, :, None]
    return o.transpose(0, 1).reshape(T, n_h * d_h).to(dt), (m + torch.log(l)).t().contiguous()


# ----------------------------------------------------- one pass, framework --

def _own_plan(st):
    from mla_latent_kv_33_b200 import mla
    mla.mla_batch_plan(st["cache"], st["ctx"], st["new"], st["free"], st["seq_lens"], st["row_start"], st["seq_idx"],
                       st["positions"], st["slots"], st["used"], shared_blocks=st["shared"])
    return {k: st[k] for k in ("table", "seq_lens", "row_start", "seq_idx", "positions", "slots", "used")}


def _own_write(st):
    from mla_latent_kv_33_b200 import mla
    mla.mla_cache_write(st["p"], st["rows"], st["slots"], st["cache"])
    return st["data"]


def _own_expand(st):
    from mla_latent_kv_33_b200 import mla
    mla.mla_prefix_expand(st["p"], st["cache"], 1, st["W_UK"], st["W_UV"], st["kc"], st["v"], st["kr"])
    return st["kc"], st["v"], st["kr"]


def _own_shared(st):
    from mla_latent_kv_33_b200 import mla
    mla.mla_decode_shared(st["p"], st["qa"], st["kc"], st["v"], st["kr"], st["cache"], st["seq_lens"], st["n_q"],
                          st["W_UK"], st["W_UV"], st["o"], st["lse"], ws=st["ws"])
    return st["o"], st["lse"]


def run(state):
    forms = dict(plan=_own_plan, write=_own_write, expand=_own_expand, shared=_own_shared) if own else \
        dict(plan=_plain_plan, write=_plain_write, expand=_plain_expand, shared=_plain_shared)
    return forms[state["op"]](state)


# -------------------------------------------------------------------- work --

def work(case):
    """Bytes and operations of one pass: inputs read once, outputs written once
    (averages where the lengths are drawn)."""
    if case["op"] == "plan":
        B, bs = case["B"], case["block_size"]
        rows = (B - case["prompts"]) + case["prompts"] * case["chunk"] / 2
        T = B - case["prompts"] + case["prompts"] * case["chunk"] + case["pad"]
        fresh = rows / bs  # blocks taken from the free list: read, and written into the table
        return dict(bytes=4 * B * 4 + B * case["shared"] * 4 + 8 * fresh + T * 16, flops=0)
    s = GEOMETRY[case["geo"]]
    n_h, d_h, d_c, d_r = s["n_h"], s["d_h"], s["d_c"], s["d_r"]
    D, es = d_c + d_r, 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "write":
        return dict(bytes=(case["T"] - case["pad"]) * 2 * D * es + case["T"] * 8, flops=0)
    weights = 2 * n_h * d_h * d_c * es
    if case["op"] == "expand":
        P = case["P"]
        return dict(bytes=P * D * es + weights + P * (2 * n_h * d_h + d_r) * es, flops=4 * P * n_h * d_h * d_c)
    T, P = case["B"] * case["n_q"], case["P"]
    suf = (case["suf_lo"] + case["suf_hi"]) / 2
    size = P * (2 * n_h * d_h + d_r) * es + case["B"] * suf * D * es + weights
    size += T * n_h * (2 * d_h + d_r) * es + T * n_h * 4
    flops = T * n_h * (2 * P * (2 * d_h + d_r) + 2 * suf * (2 * d_c + d_r) + 4 * d_h * d_c)
    return dict(bytes=size, flops=flops)


# ------------------------------------------------------------------- exact --

def _exact_plan(st):
    bs, nshared, T = st["bs"], st["shared"].numel(), st["seq_idx"].numel()
    ctx, new, free = st["ctx"].tolist(), st["new"].tolist(), st["free"].tolist()
    table = [row[:] for row in st["table"].tolist()]
    head = st["shared"].tolist()
    seq_idx, positions, slots, start, taken = [], [], [], [0], 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        table[b][:nshared] = head
        for blk in range(-(-c // bs), -(-(c + n) // bs)):
            table[b][blk] = free[taken]
            taken += 1
        for pos in range(c, c + n):
            seq_idx.append(b)
            positions.append(pos)
            slots.append(table[b][pos // bs] * bs + pos % bs)
        start.append(start[-1] + n)
    pad = T - len(seq_idx)

    def ints(x, dtype=torch.int32):
        return torch.tensor(x, dtype=dtype, device="cuda")
    return dict(table=ints(table), seq_lens=ints([c + n for c, n in zip(ctx, new)]), row_start=ints(start),
                seq_idx=ints(seq_idx + [-1] * pad), positions=ints(positions + [0] * pad),
                slots=ints(slots + [-1] * pad, torch.int64), used=ints([taken]))


def _exact_write(st):
    out = st["data"].clone().view(-1, st["rows"].shape[1])
    for t, slot in enumerate(st["slots"].tolist()):
        if slot >= 0:
            out[slot] = st["rows"][t]
    return out.view(st["data"].shape)


def _latents(st, b, lo, hi):
    """Rows lo .. hi - 1 of sequence b in 64 bits, page by page."""
    bs, out = st["bs"], []
    for i in range(lo // bs, -(-hi // bs)):
        page = st["data"][int(st["table"][b, i])].double()
        out.append(page[max(lo - i * bs, 0):min(hi - i * bs, bs)])
    return torch.cat(out)


def _exact_expand(st):
    s = st["s"]
    rows = _latents(st, 1, 0, st["P"])
    c = rows[:, :s["d_c"]].t()
    kc = torch.stack([(w.double() @ c).t() for w in st["W_UK"].split(s["d_h"])])
    v = torch.stack([(w.double() @ c).t() for w in st["W_UV"].split(s["d_h"])])
    return kc, v, rows[:, s["d_c"]:]


def _exact_shared(st):
    """Order A throughout: the suffix rows are decompressed per head and joined
    to the prefix's keys and values; one softmax over all of them."""
    s, n_q, P = st["s"], st["n_q"], st["P"]
    n_h, d_h, d_c, d_r = s["n_h"], s["d_h"], s["d_c"], s["d_r"]
    kp, vp, rp = st["kc"].double(), st["v"].double(), st["kr"].double()
    wk, wv = st["W_UK"].double(), st["W_UV"].double()
    out, lse = [], []
    for b, L in enumerate(st["lens"]):
        rows = _latents(st, b, P, L)
        ks = (rows[:, :d_c] @ wk.t()).view(L - P, n_h, d_h).transpose(0, 1)
        vs = (rows[:, :d_c] @ wv.t()).view(L - P, n_h, d_h).transpose(0, 1)
        for j in range(n_q):
            q = st["qa"][b * n_q + j].double()
            qc, qr = q[:, :d_h, None], q[:, d_h:]
            seen = L - P - n_q + j + 1
            score = torch.cat([(kp @ qc)[:, :, 0] + qr @ rp.t(),
                               ((ks @ qc)[:, :, 0] + qr @ rows[:, d_c:].t())[:, :seen]], dim=1) / math.sqrt(d_h + d_r)
            z = torch.logsumexp(score, dim=1)
            w = torch.exp(score - z[:, None])[:, None]
            out.append((w[:, :, :P] @ vp + w[:, :, P:] @ vs[:, :seen]).reshape(-1))
            lse.append(z)
    return torch.stack(out), torch.stack(lse)


def exact(case, seed):
    st = prepare(case, seed)
    return {"plan": _exact_plan, "write": _exact_write, "expand": _exact_expand, "shared": _exact_shared}[st["op"]](st)
