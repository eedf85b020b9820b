"""What the operators around the 8-bit K/V cache are measured on.

Four operators of one serving step with K and V held as e4m3 codes and one
fp32 scale for each (page, KV head):

``advance``  the batch's index arrays from the requests' token counts: page
             allocation and release, q_start, context lengths, slot map
``insert``   per-head QK RMSNorm, partial rotary embedding and the insert of the
             new K and V rows into the 8-bit cache, block scales kept up to date
``decode``   attention over the selected blocks, few queries a sequence
``prefill``  the same attention for many queries a sequence

With ``own`` false, ``run`` computes the plain forms in elementary torch
operations; with ``own`` true it makes the library's calls.
"""
import math

import torch

own = False

BLOCK, DIM, HEADS = 128, 128, 16          # tokens a page, head dim, query heads a KV head
E4M3_MAX = 448.0
ROTARY, THETA, EPS = 64, 10000.0, 1e-6
MAX_PAGES = 16384                         # pages in a state's pool at most (1 GiB of K for 4 heads)


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one user's chat, one token at a time: latency
        dict(name="decode 1x32k", op="decode", seqs=1, ctx_lo=32768, ctx_hi=32768, nq_lo=1, nq_hi=1, kv=4, topk=16),
        # the repository's decode batch
        dict(name="decode 64x128k", op="decode", seqs=64, ctx_lo=131072, ctx_hi=131072, nq_lo=1, nq_hi=1, kv=4, topk=16),
        # the repository's ragged verify batch: 4 draft tokens a sequence
        dict(name="verify 32x4 ragged", op="decode", seqs=32, ctx_lo=4096, ctx_hi=1048576, nq_lo=4, nq_hi=4, kv=4, topk=16),
        # the repository's tiny prefill: one KV head
        dict(name="prefill 2k one group", op="prefill", seqs=1, ctx_lo=2048, ctx_hi=2048, nq_lo=2048, nq_hi=2048, kv=1, topk=4),
        # several requests' odd-sized chunks in one call
        dict(name="prefill mixed chunks", op="prefill", seqs=5, ctx_lo=1001, ctx_hi=40001, nq_lo=129, nq_hi=1001, kv=4, topk=16),
        # the last chunk of the repository's 128K chunked prefill
        dict(name="prefill 128k last chunk", op="prefill", seqs=1, ctx_lo=131072, ctx_hi=131072, nq_lo=16384, nq_hi=16384, kv=4, topk=16),
        # the new rows of a decode step
        dict(name="insert 64 rows", op="insert", seqs=64, ctx_lo=1000, ctx_hi=131072, nq_lo=1, nq_hi=1, kv=4),
        # the new rows of a mixed step: short chunks, pages begun and continued
        dict(name="insert ragged rows", op="insert", seqs=33, ctx_lo=301, ctx_hi=65537, nq_lo=1, nq_hi=300, kv=4),
        # the new rows of a prefill chunk
        dict(name="insert 16384 rows", op="insert", seqs=1, ctx_lo=131072, ctx_hi=131072, nq_lo=16384, nq_hi=16384, kv=4),
        # one sequence, one token
        dict(name="advance one", op="advance", seqs=1, ctx_lo=5000, ctx_hi=5000, new_hi=1, ends=0),
        # a decode step in which some requests end and some drafts are taken back
        dict(name="advance 256", op="advance", seqs=256, ctx_lo=100, ctx_hi=131072, new_hi=4, ends=3),
        # many prompts admitted at once
        dict(name="advance 1024 prompts", op="advance", seqs=1024, ctx_lo=1, ctx_hi=4096, new_hi=1000, ends=7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "insert", "insert", "advance"])
    if op == "decode":
        nq = rng.choice([1, 1, 2, 3, 4, 8])
        lo, hi = sorted(_log(rng, 8, 262144) for _ in range(2))
        return dict(op=op, seqs=_log(rng, 1, 256 // nq), ctx_lo=lo, ctx_hi=hi, nq_lo=1, nq_hi=min(nq, lo), kv=rng.choice([1, 2, 4]),
                    topk=rng.choice([1, 4, 15, 16, 32, 64]))
    if op == "prefill":
        seqs = _log(rng, 1, 16)
        lo, hi = sorted(_log(rng, 9, 65536) for _ in range(2))
        nq = min(lo, _log(rng, 9, 4096 // seqs))
        return dict(op=op, seqs=seqs, ctx_lo=lo, ctx_hi=hi, nq_lo=rng.randint(1, nq), nq_hi=nq, kv=rng.choice([1, 2, 4]),
                    topk=rng.choice([1, 4, 15, 16, 32]))
    if op == "insert":
        seqs = _log(rng, 1, 128)
        lo, hi = sorted(_log(rng, 1, 131072) for _ in range(2))
        nq = min(lo, _log(rng, 1, 16384 // seqs))
        return dict(op=op, seqs=seqs, ctx_lo=lo, ctx_hi=hi, nq_lo=rng.randint(1, nq), nq_hi=nq, kv=rng.choice([1, 2, 4]))
    seqs = _log(rng, 1, 2048)
    lo, hi = sorted(_log(rng, 1, 65536) for _ in range(2))
    return dict(op=op, seqs=seqs, ctx_lo=lo, ctx_hi=hi, new_hi=_log(rng, 1, min(8192, 524288 // seqs)), ends=rng.randint(0, 9))


def _lengths(case):
    """(context, new rows) of each sequence: spread over the case's ranges, the same for every seed."""
    n, lo, hi = case["seqs"], case["ctx_lo"], case["ctx_hi"]
    ctx = [int(round(lo * (hi / lo) ** (i / max(1, n - 1)))) for i in range(n)]
    ctx = [ctx[(i * 7) % n] if n % 7 else ctx[i] for i in range(n)]
    if case["op"] == "advance":
        return ctx, None
    a, b = case["nq_lo"], case["nq_hi"]
    return ctx, [min(c, a + (i * 7919) % (b - a + 1)) for i, c in enumerate(ctx)]


def _deltas(case):
    """Signed token counts of an advance: mostly new tokens, some requests ended, some tokens taken back."""
    ctx, _ = _lengths(case)
    out = []
    for i, c in enumerate(ctx):
        r = (i * 31 + 11) % 100
        out.append(-c if r < case["ends"] else -min(c, 1 + i % 3) if r < 2 * case["ends"] else 1 + (i * 7919) % case["new_hi"])
    return ctx, out


def _blocks(tokens):
    return (tokens + BLOCK - 1) // BLOCK


# ---------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _codes(g, *shape):
    return (torch.randn(*shape, generator=g, device="cuda") * 100).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _batch_inputs(case, g, distinct):
    """q_start, ctx_len and a page table over a shuffled pool; `distinct`: no page twice."""
    ctx, nq = _lengths(case)
    starts = [0]
    for n in nq:
        starts.append(starts[-1] + n)
    width = max(_blocks(c) for c in ctx)
    need = sum(_blocks(c) for c in ctx)
    pages = need + 3 if distinct else min(need + 3, MAX_PAGES)
    # a sequence's pages follow one another in a shuffled order; beyond the pool's size sequences share pages, as prefixes do
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor([0] + [_blocks(c) for c in ctx[:-1]], device="cuda").cumsum(0)
    table = perm[(first[:, None] + torch.arange(width, device="cuda")[None, :]) % pages]
    used = torch.arange(width, device="cuda")[None, :] < _ints([_blocks(c) for c in ctx])[:, None]
    table = torch.where(used, table, torch.full_like(table, -1)).contiguous()
    return dict(ctx=ctx, nq=nq, rows=starts[-1], pages=pages, q_start=_ints(starts), ctx_len=_ints(ctx), page_table=table)


def _attention_inputs(case, g):
    b = _batch_inputs(case, g, False)
    rows, kv, topk, pages = b["rows"], case["kv"], case["topk"], b["pages"]
    b["q"] = (1.5 * torch.randn(rows, HEADS * kv, DIM, generator=g, device="cuda")).to(torch.bfloat16)
    b["k"], b["v"] = _codes(g, pages, kv, BLOCK, DIM), _codes(g, pages, kv, BLOCK, DIM)
    b["k_scale"] = torch.exp2(-7.2 + torch.rand(pages, kv, generator=g, device="cuda"))
    b["v_scale"] = torch.exp2(-7.2 + torch.rand(pages, kv, generator=g, device="cuda"))
    # the selection as the indexer leaves it: the own block and topk - 1 earlier ones, some of them liked by many rows
    seq, pos = _row_places(b)
    cur, width = pos // BLOCK, b["page_table"].shape[1]
    liked = torch.rand(kv, width, generator=g, device="cuda") * 0.5
    score = torch.rand(rows, kv, width, generator=g, device="cuda") + liked[None]
    at = torch.arange(width, device="cuda")
    score = torch.where(at[None, None, :] < cur[:, None, None], score, torch.where(at[None, None, :] == cur[:, None, None], 9.0, -1.0))
    best, ids = score.topk(min(topk, width), dim=-1)
    ids = torch.where(best >= 0, ids, width).sort(dim=-1).values
    sel = torch.full((rows, kv, topk), -1, dtype=torch.int32, device="cuda")
    sel[:, :, :ids.shape[-1]] = torch.where(ids < width, ids, -1).to(torch.int32)
    b["block_idx"] = sel
    return b


def _insert_inputs(case, g):
    b = _batch_inputs(case, g, True)
    rows, kv, pages = b["rows"], case["kv"], b["pages"]
    if pages > MAX_PAGES // 8:             # the untouched pages of a long context: one page stands for them all
        touched = torch.zeros_like(b["page_table"], dtype=torch.bool)
        seq, pos = _row_places(b)
        touched[seq, pos // BLOCK] = True
        ids = torch.full_like(b["page_table"], -1)
        pages = int(touched.sum()) + 1
        ids[touched] = 1 + torch.randperm(pages - 1, generator=g, device="cuda").to(torch.int32)
        b["page_table"] = torch.where(touched, ids, torch.where(b["page_table"] >= 0, 0, -1).to(torch.int32)).contiguous()
        b["pages"] = pages
    b["q"] = torch.randn(rows, HEADS * kv, DIM, generator=g, device="cuda").to(torch.bfloat16)
    for n in ("k_new", "v_new"):           # tokens of differing magnitude, so that block scales grow
        size = torch.exp2(2 * torch.rand(rows, kv, 1, generator=g, device="cuda") - 1)
        b[n] = (size * torch.randn(rows, kv, DIM, generator=g, device="cuda")).to(torch.bfloat16)
    for n in ("q_norm_w", "k_norm_w"):
        b[n] = (1 + 0.2 * torch.randn(DIM, generator=g, device="cuda")).to(torch.bfloat16)
    b["k"], b["v"] = _codes(g, pages, kv, BLOCK, DIM), _codes(g, pages, kv, BLOCK, DIM)
    for n in ("k_scale", "v_scale"):
        b[n] = torch.exp2(torch.randint(-9, -6, (pages, kv), generator=g, device="cuda").float())
    return b


def _advance_inputs(case, g):
    ctx, delta = _deltas(case)
    n = len(ctx)
    have, after = [_blocks(c) for c in ctx], [_blocks(c + d) for c, d in zip(ctx, delta)]
    width = max(max(have), max(after))
    need = sum(max(0, b - a) for a, b in zip(have, after))
    held = sum(have)
    pages = held + need + 5
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    used = torch.arange(width, device="cuda")[None, :] < _ints(have)[:, None]
    table[used] = perm[:held]
    head = int(torch.randint(0, pages, (1,), generator=g, device="cuda"))
    ring = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    free = pages - held
    ring[(head + torch.arange(free, device="cuda")) % pages] = perm[held:]
    rows = sum(d for d in delta if d > 0)
    return dict(pages=pages, rows=rows, delta=_ints(delta), ctx_len=_ints(ctx), page_table=table, ring=ring,
                pool=_ints([head, free, 0, 0]))


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = _advance_inputs(case, g) if op == "advance" else _insert_inputs(case, g) if op == "insert" else _attention_inputs(case, g)
    s["op"] = op
    if own:                                # the handles, result buffers and workspace that a serving loop keeps
        import block_sparse_long_13_b200 as msa
        empty = lambda *shape, dtype: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
        if op == "advance":
            n = s["delta"].numel()
            s["out"] = dict(ctx_len=empty(n, dtype=torch.int32), pool=empty(4, dtype=torch.int32), q_start=empty(n + 1, dtype=torch.int32),
                            slot_map=empty(max(1, s["rows"]), dtype=torch.int32))
            return s
        kv = case["kv"]
        s["cfg"] = msa.Config(num_q_heads=HEADS * kv, num_kv_heads=kv, idx_heads=2 * kv, topk=case.get("topk", 16))
        s["batch"] = msa.Batch(q_start=s["q_start"], ctx_len=s["ctx_len"], page_table=s["page_table"], total_q=s["rows"],
                               max_q_per_seq=max(s["nq"]), num_pages=s["pages"])
        if op == "insert":
            s["q_out"] = torch.empty_like(s["q"])
        else:
            size = (msa.decode_fp8_workspace_bytes if op == "decode" else msa.prefill_fp8_workspace_bytes)(s["cfg"], s["batch"])
            s["out"], s["lse"] = torch.empty_like(s["q"]), empty(s["rows"], HEADS * kv, dtype=torch.float32)
            s["workspace"] = empty(max(1, size), dtype=torch.uint8)
    return s


# ---------------------------------------------------------------- plain forms
def _row_places(s):
    """Sequence and position of each query row."""
    starts = s["q_start"].long()
    row = torch.arange(s["rows"], device=starts.device)
    seq = torch.searchsorted(starts, row, right=True) - 1
    return seq, s["ctx_len"].long()[seq] - starts[seq + 1] + row


def _plain_attention(s):
    q, sel = s["q"], s["block_idx"].long()
    rows, kv, topk = sel.shape
    seq, pos = _row_places(s)
    out = torch.empty_like(q)
    lse = torch.empty(rows, q.shape[1], dtype=torch.float32, device=q.device)
    group = torch.arange(kv, device=q.device)[None, :, None]
    offset = torch.arange(BLOCK, device=q.device)
    step = max(1, (1 << 29) // (kv * topk * BLOCK * DIM))     # rows whose keys, in 32 bits, fit in 2 GiB
    for a in range(0, rows, step):
        z = min(rows, a + step)
        n, b = z - a, sel[a:z]
        page = s["page_table"].long()[seq[a:z, None, None], b.clamp(min=0)].clamp(min=0)
        keys = s["k"][page, group].view(torch.float8_e4m3fn).float() * s["k_scale"][page, group][..., None, None]
        qf = q[a:z].view(n, kv, HEADS, DIM).float()
        logit = (qf @ keys.view(n, kv, topk * BLOCK, DIM).transpose(-1, -2)) * (1.0 / math.sqrt(DIM))
        del keys
        hidden = (b[..., None] < 0) | (b[..., None] * BLOCK + offset > pos[a:z, None, None, None])
        logit = logit.masked_fill(hidden.view(n, kv, 1, topk * BLOCK), float("-inf"))
        top = logit.amax(-1, keepdim=True)
        top = torch.where(top > float("-inf"), top, 0.0)
        p = torch.exp(logit - top)
        total = p.sum(-1, keepdim=True)
        values = s["v"][page, group].view(torch.float8_e4m3fn).float() * s["v_scale"][page, group][..., None, None]
        values = values.masked_fill(hidden[..., None], 0.0).view(n, kv, topk * BLOCK, DIM)
        o = torch.where(total > 0, (p @ values) / total, 0.0)
        out[a:z] = o.view(n, kv * HEADS, DIM).to(out.dtype)
        lse[a:z] = (top + torch.log(total)).view(n, kv * HEADS)
    return {"out": out, "lse": lse}


def _norm_rope(x, weight, pos):
    """Per-head RMSNorm, then the rotary embedding of channel pairs (i, i + ROTARY / 2); 32 bits, angles in 64."""
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    half = ROTARY // 2
    inv = torch.pow(torch.tensor(THETA, dtype=torch.float64, device=x.device),
                    -2.0 * torch.arange(half, dtype=torch.float64, device=x.device) / ROTARY)
    angle = pos.double()[:, None] * inv
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    a, b = y[..., :half], y[..., half:ROTARY]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., ROTARY:]], dim=-1)


def _insert_codes(cache, scale, x, page, slot):
    """x's rows into their pages as codes: a page's scale is the least power of two that holds its largest new value,
    or the old one where that is enough or larger and the page was not begun by this call; older rows of a page whose
    scale grew are rounded again."""
    pages, kv = scale.shape
    amax = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)                       # [rows][kv]
    top = torch.zeros(pages, kv, device=x.device).index_reduce_(0, page, amax, "amax")
    first = torch.full((pages,), BLOCK, device=x.device, dtype=torch.int64).index_reduce_(0, page, slot, "amin")
    touched = (first < BLOCK)[:, None]
    part, exponent = torch.frexp(top)                                                  # part in [0.5, 1); 448 = 0.875 * 2^9
    fit = torch.where(top > 0, torch.ldexp(torch.ones_like(top), torch.where(part > 0.875, exponent - 8, exponent - 9).clamp(min=-126)), 2.0 ** -126)
    grown = touched & ((first == 0)[:, None] | (top > E4M3_MAX * scale))
    new = torch.where(grown, fit, scale)
    again = torch.nonzero(grown & (first > 0)[:, None])                                # older rows to round again
    old = cache[again[:, 0], again[:, 1]].view(torch.float8_e4m3fn).float() * (scale / new)[again[:, 0], again[:, 1], None, None]
    older = torch.arange(BLOCK, device=x.device)[None, :] < first[again[:, 0], None]
    kept = cache[again[:, 0], again[:, 1]]
    cache[again[:, 0], again[:, 1]] = torch.where(older[..., None], old.to(torch.float8_e4m3fn).view(torch.uint8), kept)
    code = (x / new[page][..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    cache[page[:, None], torch.arange(kv, device=x.device)[None, :], slot[:, None]] = code.view(torch.uint8)
    scale.copy_(new)


def _insert_outputs(s, q):
    # codes as the e4m3 values they are, in units of their block's scale
    return {"q": q, "k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn), "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _plain_insert(s):
    seq, pos = _row_places(s)
    page, slot = s["page_table"].long()[seq, pos // BLOCK], pos % BLOCK
    q = _norm_rope(s["q"], s["q_norm_w"], pos).to(torch.bfloat16)
    _insert_codes(s["k"], s["k_scale"], _norm_rope(s["k_new"], s["k_norm_w"], pos), page, slot)
    _insert_codes(s["v"], s["v_scale"], s["v_new"].float(), page, slot)
    return _insert_outputs(s, q)


def _plain_advance(s):
    delta, ctx, table, ring, pool = s["delta"].long(), s["ctx_len"].long(), s["page_table"], s["ring"], s["pool"].long()
    n, width = table.shape
    pages = ring.numel()
    after = ctx + delta
    have, want = (ctx + BLOCK - 1) // BLOCK, (after + BLOCK - 1) // BLOCK
    grow, back = (want - have).clamp(min=0), (have - want).clamp(min=0)
    taken, given = grow.cumsum(0), back.cumsum(0)                                      # inclusive
    need, free = taken[-1], given[-1]
    block = torch.arange(width, device=delta.device)[None, :]
    fresh, done = (block >= have[:, None]) & (block < want[:, None]), (block >= want[:, None]) & (block < have[:, None])
    # freed pages go to the ring's tail, new ones come from its head, both in order of (sequence, block)
    place = (pool[0] + pool[1] + (given - back)[:, None] + block - want[:, None]) % pages
    ring[place[done]] = table[done]
    place = (pool[0] + (taken - grow)[:, None] + block - have[:, None]) % pages
    table[fresh] = ring[place[fresh]]
    rows = delta.clamp(min=0)
    q_start = torch.cat([torch.zeros_like(rows[:1]), rows.cumsum(0)])
    row = torch.arange(s["rows"], device=delta.device)
    seq = torch.searchsorted(q_start, row, right=True) - 1
    pos = after[seq] - q_start[seq + 1] + row
    slot = table.long()[seq, pos // BLOCK] * BLOCK + pos % BLOCK
    state = torch.stack([(pool[0] + need) % pages, pool[1] - need + free, torch.zeros_like(need), q_start[-1]])
    whole = lambda t: t.to(torch.int32)  # noqa: E731
    return {"ctx_len": whole(after), "pool": whole(state), "q_start": whole(q_start), "slot_map": whole(slot), "page_table": table, "ring": ring}


# ---------------------------------------------------------------- one pass
def run(state):
    s = state
    op = s["op"]
    if not own:
        return _plain_advance(s) if op == "advance" else _plain_insert(s) if op == "insert" else _plain_attention(s)
    import block_sparse_long_13_b200 as msa
    if op == "advance":
        o = s["out"]
        msa.advance_batch(s["delta"], s["ctx_len"], s["page_table"], s["ring"], s["pool"], o["ctx_len"], o["pool"], o["q_start"], o["slot_map"])
        return {**o, "slot_map": o["slot_map"][:s["rows"]], "page_table": s["page_table"], "ring": s["ring"]}
    if op == "insert":
        msa.qknorm_rope_insert_fp8(s["cfg"], s["batch"], s["q"], s["k_new"], s["v_new"], s["q_norm_w"], s["k_norm_w"], s["q_out"], s["k"], s["v"],
                                   s["k_scale"], s["v_scale"], rotary_dim=ROTARY, rope_theta=THETA, eps=EPS)
        return _insert_outputs(s, s["q_out"])
    call = msa.attn_decode_fp8 if op == "decode" else msa.attn_prefill_fp8
    call(s["cfg"], s["batch"], s["q"], s["k"], s["v"], s["k_scale"], s["v_scale"], s["block_idx"], s["out"], s["lse"], s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "advance":
        ctx, delta = _deltas(case)
        moved = sum(abs(_blocks(c + d) - _blocks(c)) for c, d in zip(ctx, delta))
        rows = sum(d for d in delta if d > 0)
        return {"bytes": 4 * (4 * len(ctx) + 1 + rows + 2 * moved + 8), "flops": 0}
    ctx, nq = _lengths(case)
    rows, kv = sum(nq), case["kv"]
    if op == "insert":
        row = 2 * HEADS * kv * DIM * 2 + 2 * kv * DIM * (2 + 1)       # q in and out, new k and v in as bf16, out as codes
        return {"bytes": rows * row + 4 * DIM, "flops": 0}
    topk = case["topk"]
    tiles = keys = 0.0
    for c, n in zip(ctx, nq):
        have = _blocks(c)
        mean = min(topk, max(1.0, (c - n / 2) / BLOCK))               # blocks a row selects
        tiles += kv * have * (1 - (1 - min(1.0, mean / have)) ** n)   # distinct ones over the sequence's rows
        keys += sum(min(topk - 1, p // BLOCK) * BLOCK + p % BLOCK + 1 for p in range(c - n, c)) * kv * HEADS
    bytes_ = tiles * (2 * BLOCK * DIM + 8) + rows * (2 * HEADS * kv * DIM * 2 + 4 * HEADS * kv + 4 * kv * topk)
    return {"bytes": bytes_, "flops": 4 * DIM * keys}


# ---------------------------------------------------------------- the definition in 64 bits
def _table():
    """The value of each e4m3 code (sign, 4 exponent bits of bias 7, 3 mantissa bits; 0x7f and 0xff are NaN)."""
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.nan if (e, m) == (15, 7) else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v.append(-x if c & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _exact_attention(s):
    value = _table()
    q, sel = s["q"].double(), s["block_idx"].long()
    rows, kv, topk = sel.shape
    at = [(i, c - n + j) for i, (c, n) in enumerate(zip(s["ctx"], s["nq"])) for j in range(n)]
    at = torch.tensor(at, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(rows, q.shape[1], dtype=torch.float64, device="cuda")
    step = max(1, (1 << 28) // (topk * BLOCK * DIM))
    for g in range(kv):
        heads = slice(g * HEADS, (g + 1) * HEADS)
        k, v = s["k"][:, g], s["v"][:, g]
        ks, vs = s["k_scale"][:, g].double(), s["v_scale"][:, g].double()
        for a in range(0, rows, step):
            w = slice(a, min(rows, a + step))
            b, seq, pos = sel[w, g], at[w, 0], at[w, 1]
            page = s["page_table"].long()[seq[:, None], b.clamp(min=0)].clamp(min=0)
            place = (b[:, :, None] * BLOCK + torch.arange(BLOCK, device="cuda")).reshape(len(b), -1)
            seen = (place >= 0) & (place <= pos[:, None]) & (b >= 0).repeat_interleave(BLOCK, 1)
            kd = (value[k[page].long()] * ks[page][:, :, None, None]).reshape(len(b), -1, DIM)
            x = torch.bmm(q[w, heads], kd.mT) / math.sqrt(DIM)
            del kd
            x = torch.where(seen[:, None, :], x, -math.inf)
            lse[w, heads] = torch.logsumexp(x, -1)
            p = torch.exp(x - torch.where(torch.isinf(lse[w, heads]), 0.0, lse[w, heads])[..., None])
            vd = (value[v[page].long()] * vs[page][:, :, None, None]).reshape(len(b), -1, DIM)
            out[w, heads] = torch.bmm(p, torch.where(seen[..., None], vd, 0.0))
    return {"out": out, "lse": lse}


def _exact_insert(s):
    """Results before their last rounding: a code's value in units of its block's scale, unrounded."""
    value = _table()
    kv = s["k_scale"].shape[1]
    at = [(i, c - n + j) for i, (c, n) in enumerate(zip(s["ctx"], s["nq"])) for j in range(n)]
    at = torch.tensor(at, device="cuda")
    seq, pos = at[:, 0], at[:, 1]
    page, slot = s["page_table"].long()[seq, pos // BLOCK], pos % BLOCK

    def turned(x, w):
        x = x.double()
        x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / DIM + EPS) * w.double()
        i = torch.arange(ROTARY // 2, dtype=torch.float64, device="cuda")
        z = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"), pos.double()[:, None] / THETA ** (2 * i / ROTARY))
        pair = torch.complex(x[..., :ROTARY // 2], x[..., ROTARY // 2:ROTARY]) * z[:, None]
        return torch.cat([pair.real, pair.imag, x[..., ROTARY:]], -1)

    got = {"q": turned(s["q"], s["q_norm_w"])}
    for n, x in (("k", turned(s["k_new"], s["k_norm_w"])), ("v", s["v_new"].double())):
        codes, scale = value[s[n].long()], s[n + "_scale"].double().clone()
        last = torch.full((len(scale),), -1, device="cuda", dtype=torch.int64)
        begun = torch.full((len(scale),), False, device="cuda")
        begun[page[slot == 0]] = True
        top = torch.zeros_like(scale)
        for j in range(kv):
            top[:, j].scatter_reduce_(0, page, x[:, j].abs().amax(-1), "amax")
        last.scatter_reduce_(0, page, slot, "amax")
        powers = torch.tensor([2.0 ** e for e in range(-60, 60)], dtype=torch.float64, device="cuda")
        fit = powers[torch.searchsorted(E4M3_MAX * powers, top)]                         # the first that holds top
        new = torch.where((last >= 0)[:, None] & (begun[:, None] | (top > E4M3_MAX * scale)), fit, scale)
        mine = torch.zeros(len(scale), BLOCK, dtype=torch.bool, device="cuda")
        mine[page, slot] = True
        behind = torch.arange(BLOCK, device="cuda")[None] > last[:, None]                # rows behind the last one stay
        keep = (behind | begun[:, None] | (last < 0)[:, None])[:, None, :, None]
        codes = torch.where(keep, codes, codes * (scale / new)[:, :, None, None])
        codes[page, :, slot] = x / new[page][..., None]
        got[n], got[n + "_scale"] = codes, new
    return got


def exact(case, seed):
    if case["op"] == "advance":            # whole numbers only
        return None
    s = prepare(case, seed)
    return _exact_insert(s) if case["op"] == "insert" else _exact_attention(s)
