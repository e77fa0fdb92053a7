"""Measured cases of the operators of a serving step around a caller-owned paged cache: the
step's plan (row ranges, pages, slots) from request lengths, the append with rotation by
positions of several axes, attention whose scores are capped, biased by distance or masked by
window, document and prefix, and the draw of the next token with every row's own parameters.

The rows of a batch are packed: rows [row_start[s], row_start[s + 1]) belong to sequence s, row
i of it stands at position p = ctx_len[s] + i.  Query head h reads kv head h // (heads / kv heads).

plan       a sequence brings new_len[s] rows after seq_len[s] cached positions; a negative
           new_len ends it, and its pages go on top of the stack of free pages, sequence by
           sequence.  The pages of new blocks of positions come from the top of the stack, in
           the order (sequence, block).  Rows of nobody get position and slot -1.
append     cached row p of sequence s takes k, rotated, and v; pair j of a row is turned by the
           angle of position positions[axis[j]][row]; an axis of -1 leaves the pair alone.
attention  x_t = cap tanh(q . k_t / sqrt(head_dim) / cap) - slope[h] |p - t| over the positions
           max(first[row], p + 1 - window) <= t < max(p + 1, prefix[s]); out = softmax(x) v, and
           0 where a row sees nothing.
sample     tokens in the order (logit descending, index ascending); the first top_k; of those the
           shortest prefix whose probability reaches top_p; of those the ones with at least min_p
           times the largest probability.  The draw runs over what is left in index order: the
           first token whose running mass exceeds uniform * mass.  A temperature of 0 takes the
           first token of the order.

``run`` is one pass: with ``own`` the calls of the library, without it the same operators in
elementary torch operations.  ``exact`` is the definition in 64 bits, one sequence and head, or
one row, at a time.
"""
import math
import random

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_HEADS = [(9, 3, 64), (32, 8, 64), (32, 8, 128), (8, 1, 128), (16, 16, 64), (12, 4, 80), (10, 2, 96), (4, 2, 16),
          (15, 5, 72), (6, 6, 128)]


# ------------------------------------------------------------------ cases

def _attention(**kw):
    d = dict(op="paged", dtype="bf16", heads=32, kv_heads=8, head_dim=128, page=64, nseq=1, new=1, ctx=0, even=False,
             idle=0, pad=0, cap=0.0, slopes=False, window=0, docs=0, prefix=0)
    d.update(kw)
    return d


def listed():
    return [
        # A decode step of a large batch: one row a sequence, a page taken now and then.
        dict(name="plan_decode_batch", op="plan", page=64, nseq=256, new=1, ctx=8000, ended=0, pad=0, lens=1),
        # A step that takes in ragged prompts while other requests end and give their pages back.
        dict(name="plan_prompts", op="plan", page=16, nseq=96, new=1024, ctx=4000, ended=7, pad=301, lens=2),
        # One decode step of a batch whose text goes on behind images: three axes, contiguous sections.
        dict(name="axes_decode_batch", op="append", dtype="bf16", cache="bf16", heads=32, kv_heads=8, head_dim=128,
             page=64, nseq=128, new=1, ctx=8000, even=False, idle=0, pad=0, axes=3, pattern="sections", lens=3),
        # Prompts of images and text, from an fp32 projection into a bf16 cache, rows left over behind them.
        dict(name="axes_prompts", op="append", dtype="f32", cache="bf16", heads=32, kv_heads=8, head_dim=64,
             page=64, nseq=16, new=1024, ctx=0, even=False, idle=0, pad=37, axes=3, pattern="turns", lens=4),
        # The next token of one chat of a few hundred tokens, capped scores: a launch's latency.
        _attention(name="scored_one_token", heads=9, kv_heads=3, head_dim=64, page=16, ctx=261, even=True, cap=50.0, lens=5),
        # A serving batch's step through a layer with a sliding window: the pages before it are gone.
        _attention(name="scored_window_batch", nseq=64, ctx=16000, cap=50.0, window=4096, lens=6),
        # A long-context step of a model without rotation: distances in the scores.
        _attention(name="scored_distance_long", head_dim=64, nseq=4, ctx=32768, even=True, slopes=True, lens=7),
        # Chunks of long documents through a windowed layer with capped scores.
        _attention(name="scored_window_chunk", page=128, nseq=3, new=512, ctx=16000, pad=11, cap=50.0, window=4096, lens=8),
        # Packed training-like rows served as one prompt: documents behind one another, capped scores.
        _attention(name="scored_documents", op="prompt", page=0, nseq=2, new=6000, pad=19, cap=30.0, docs=1500, lens=9),
        # An fp32 engine's prompts whose instructions see each other both ways, distances in the scores.
        _attention(name="scored_prefix_f32", op="prompt", dtype="f32", heads=9, kv_heads=3, head_dim=64, page=0, nseq=7,
                   new=701, pad=5, slopes=True, prefix=300, lens=10),
        # The next token of one chat.
        dict(name="sample_one", op="sample", dtype="f32", rows=1, vocab=49152, mix=False, temperature=0.8, top_k=0,
             top_p=0.95, min_p=0.0, pad=0, lens=11),
        # A serving batch's tokens: every request with its own parameters.
        dict(name="sample_batch", op="sample", dtype="f32", rows=256, vocab=128256, mix=True, temperature=1.0, top_k=50,
             top_p=0.9, min_p=0.05, pad=0, lens=12),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "prompt", "paged", "paged", "sample"])
    lens = rng.randrange(1 << 20)
    pad = rng.choice([0, 0, rng.randrange(1, 64)])
    if op == "sample":
        rows = _spread(rng, 1, 256)
        vocab = _spread(rng, 300, min(256000, 30000000 // rows))
        return dict(op=op, dtype=rng.choice(["f32", "f32", "bf16"]), rows=rows, vocab=vocab, mix=rng.random() < 0.5,
                    temperature=rng.choice([0.0, 0.3, 0.7, 1.0, 1.4]), top_k=rng.choice([0, 0, 1, _spread(rng, 2, 1000)]),
                    top_p=rng.choice([1.0, 0.5, 0.9, 0.95, 0.99]), min_p=rng.choice([0.0, 0.0, 0.02, 0.1]),
                    pad=rng.choice([0, 0, 3, 64]), lens=lens)
    if op == "plan":
        nseq = _spread(rng, 1, 1000)
        return dict(op=op, page=rng.choice([16, 32, 64, 128, 256]), nseq=nseq,
                    new=rng.choice([1, _spread(rng, 2, max(2, min(4096, 60000 // nseq)))]), ctx=_spread(rng, 1, 16000),
                    ended=rng.choice([0, 3, 10]), pad=pad, lens=lens)
    heads, kv_heads, head_dim = rng.choice(_HEADS)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    page = rng.choice([16, 32, 64, 128, 256])
    even, idle = rng.random() < 0.3, rng.choice([0, 0, 3, 5])
    if op == "append":
        nseq = _spread(rng, 1, 256)
        return dict(op=op, dtype=dtype, cache=rng.choice(["bf16", dtype]), heads=heads, kv_heads=kv_heads,
                    head_dim=head_dim, page=page, nseq=nseq, new=rng.choice([1, _spread(rng, 2, max(2, 16000 // nseq))]),
                    ctx=rng.choice([0, _spread(rng, 1, 8000)]), even=even, idle=idle, pad=pad, axes=rng.choice([2, 3, 4]),
                    pattern=rng.choice(["sections", "turns", "part"]), lens=lens)
    kw = dict(cap=rng.choice([0.0, 0.0, 5.0, 30.0, 50.0]), slopes=rng.random() < 0.4,
              window=rng.choice([0, 0, 1, _spread(rng, 2, 4096)]), docs=rng.choice([0, 0, _spread(rng, 2, 1500)]))
    kw["prefix"] = 0 if kw["docs"] else rng.choice([0, _spread(rng, 1, 600)])
    if op == "prompt":
        nseq = _spread(rng, 1, 24)
        new = _spread(rng, 1, (6000 if nseq <= 2 else 2500 if nseq <= 4 else 1024) if dtype == "bf16" else 512)
        page = ctx = 0
    else:
        nseq = _spread(rng, 1, 48)
        new = rng.choice([1, 1, _spread(rng, 2, 512 if nseq <= 3 else 48)])
        ctx = _spread(rng, 1, (16000 if nseq <= 4 else 6000) if dtype == "bf16" else 2000)
    return _attention(op=op, dtype=dtype, heads=heads, kv_heads=kv_heads, head_dim=head_dim, page=page, nseq=nseq,
                      new=new, ctx=ctx, even=even, idle=idle, pad=pad, lens=lens, **kw)


def _lengths(case):
    """(new rows, cached positions) of every sequence.  The first has the largest of both; with
    `idle`, every idle-th sequence has no new row; with `ended`, every ended-th one ends."""
    r = random.Random(case["lens"])
    new, ctx = [], []
    for s in range(case["nseq"]):
        full = case.get("even") or s == 0
        n = case["new"] if full else r.randint(1, case["new"])
        c = case["ctx"] if full else r.randint(0, case["ctx"])
        if case.get("idle") and s % case["idle"] == case["idle"] - 1:
            n = 0
        if case.get("ended") and s % case["ended"] == case["ended"] - 1:
            n = -1
        new.append(n)
        ctx.append(c)
    return new, ctx


def _masks(case):
    """What the masks are made of: the first position that every row sees (None without
    documents) and every sequence's prefix.  Documents are of 1 to `docs` positions; the last
    position of every fourth one is a separator that sees nothing."""
    new, ctx = _lengths(case)
    r = random.Random(case["lens"] + 1)
    prefix = [min(n + c, r.randint(0, case["prefix"])) if case["prefix"] else 0 for n, c in zip(new, ctx)]
    if not case["docs"]:
        return None, prefix
    first = []
    for n, c in zip(new, ctx):
        at, of = 0, np.zeros(n + c, dtype=np.int64)
        while at < n + c:
            end = min(n + c, at + r.randint(1, case["docs"]))
            of[at:end] = at
            if r.random() < 0.25:
                of[end - 1] = end
            at = end
        first.append(of[c:])
    return first, prefix


def _spans(case):
    """(from, to) of the positions that every row sees, a pair of arrays a sequence."""
    new, ctx = _lengths(case)
    first, prefix = _masks(case)
    out = []
    for s, (n, c) in enumerate(zip(new, ctx)):
        p = np.arange(c, c + n)
        lo = np.maximum(0, p + 1 - case["window"]) if case["window"] else np.zeros(n, dtype=np.int64)
        if first is not None:
            lo = np.maximum(lo, first[s])
        out.append((lo, np.maximum(p + 1, prefix[s])))
    return out


def work(case):
    if case["op"] == "sample":
        cells = case["rows"] * case["vocab"]
        return {"bytes": cells * (4 if case["dtype"] == "f32" else 2) + 24 * case["rows"], "flops": 4 * cells}
    new, ctx = _lengths(case)
    if case["op"] == "plan":
        P, rows = case["page"], sum(max(n, 0) for n in new) + case["pad"]
        pages = sum((c + P - 1) // P if n < 0 else (n + c + P - 1) // P - (c + P - 1) // P for n, c in zip(new, ctx))
        # lengths in; row ranges and lengths out; a page id read and written; position and slot a row
        return {"bytes": 20 * len(new) + 8 * pages + 12 * rows, "flops": 4 * rows}
    H, KV, hd = case["heads"], case["kv_heads"], case["head_dim"]
    rows, e = sum(new), 4 if case["dtype"] == "f32" else 2
    if case["op"] == "append":
        ec = 4 if case["cache"] == "f32" else 2
        # q, k, v, the positions and the rotation in; the rotated q and the cache rows out
        rope = max(n + c for n, c in zip(new, ctx)) if case["nseq"] > 1 else rows
        return {"bytes": rows * hd * ((H + 2 * KV) * (e + ec)) + 4 * rows * case["axes"] + min(rows, rope) * hd * 4,
                "flops": 3 * rows * hd * (H + KV)}
    pairs = cached = 0
    for lo, hi in _spans(case):
        seen = hi > lo
        pairs += int((hi - lo)[seen].sum())
        cached += int(hi[seen].max() - lo[seen].min()) if seen.any() else 0
    return {"bytes": 2 * rows * H * hd * e + 2 * cached * KV * hd * e, "flops": 4 * pairs * H * hd}


# ------------------------------------------------------------------ inputs

def _ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    return {"sample": _prepare_sample, "plan": _prepare_plan}.get(case["op"], _prepare_rows)(case, g)


def _prepare_sample(case, g):
    R, V = case["rows"], case["vocab"]
    # a language model's logits: a broad bulk, and in each row a few tokens that stand out
    buf = torch.randn(R, V + case["pad"], device="cuda", generator=g).mul_(2.5)
    top = torch.randint(V, (R, 8), device="cuda", generator=g)
    buf.scatter_add_(1, top, torch.rand(R, 8, device="cuda", generator=g) * 9.0)
    r = random.Random(case["lens"])

    def each(name, choices):
        return [r.choice(choices) if case["mix"] and i else case[name] for i in range(R)]

    T, k = each("temperature", [0.0, 0.6, 0.8, 1.0, 1.2]), each("top_k", [0, 0, 1, 20, 64, 400])
    p, m = each("top_p", [1.0, 0.8, 0.9, 0.95]), each("min_p", [0.0, 0.0, 0.02, 0.1])
    return dict(op="sample", logits=buf.to(_TYPES[case["dtype"]])[:, :V], temperature=_ints(T, torch.float32),
                top_k=_ints(k), top_p=_ints(p, torch.float32), min_p=_ints(m, torch.float32),
                uniforms=torch.rand(R, device="cuda", generator=g), ids=torch.zeros(R, dtype=torch.int32, device="cuda"))


def _prepare_plan(case, g):
    new, ctx = _lengths(case)
    P, rows = case["page"], sum(max(n, 0) for n in new) + case["pad"]
    held = [(c + P - 1) // P for c in ctx]
    need = [0 if n < 0 else (n + c + P - 1) // P - h for n, c, h in zip(new, ctx, held)]
    pool = sum(held) + sum(need) + 50
    ids = torch.randperm(pool, device="cuda", generator=g).to(torch.int32)
    width = max(h + n for h, n in zip(held, need)) + 1
    where, at = np.full((len(new), width), -1, dtype=np.int64), 0
    for s, h in enumerate(held):
        where[s, :h] = np.arange(at, at + h)
        at += h
    where = torch.from_numpy(where).cuda()
    stack = torch.full((pool,), -1, dtype=torch.int32, device="cuda")
    stack[:pool - at] = ids[at:]
    S = len(new)
    return dict(op="plan", page=P, new_len=_ints(new), seq_len=_ints(ctx),
                page_table=torch.where(where >= 0, ids[where.clamp(min=0)], -1).to(torch.int32).contiguous(),
                free_pages=stack, free_count=_ints([pool - at]), row_start=_ints([0] * (S + 1)), ctx_len=_ints([0] * S),
                positions=_ints([0] * rows), slots=_ints([0] * rows, torch.int64), seq_len_out=_ints([0] * S),
                free_count_out=_ints([0]), status=_ints([0]))


def _axis_map(case):
    """The axis of every pair: in contiguous sections (the first axis has the smallest), in turns,
    or in turns with the last quarter of the pairs not rotated."""
    half, n = case["head_dim"] // 2, case["axes"]
    if case["pattern"] == "sections":
        cut = [half * (2 * a + 1) // (2 * n) for a in range(n)]
        return [max(a for a in range(n) if a == 0 or j >= cut[a]) for j in range(half)]
    whole = half - half // 4 if case["pattern"] == "part" else half
    return [j % n if j < whole else -1 for j in range(half)]


def _prepare_rows(case, g):
    dev = torch.device("cuda")
    new, ctx = _lengths(case)
    H, KV, hd, S, page = case["heads"], case["kv_heads"], case["head_dim"], case["nseq"], case["page"]
    used = sum(new)
    rows = max(used + case["pad"], 1)
    t = _TYPES[case["dtype"]]
    ct = _TYPES[case.get("cache", case["dtype"])]

    def normal(*shape, dtype=t, scale=1.0):
        x = torch.randn(*shape, device=dev, dtype=torch.float32 if dtype == torch.float32 else torch.bfloat16, generator=g)
        return x.mul_(scale).to(dtype)

    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    st = dict(op=case["op"], used=used, new_max=max(new), len_max=max(n + c for n, c in zip(new, ctx)), ws=None,
              row_start=_ints(starts), ctx_len=_ints(ctx), status=_ints([0]),
              # trained queries point somewhere: scores spread by a few units
              q=normal(rows, H, hd, scale=2.0), out=torch.zeros(rows, H, hd, dtype=ct, device=dev))
    if case["op"] != "paged":
        st["k"], st["v"] = normal(rows, KV, hd), normal(rows, KV, hd)
    if case["op"] != "prompt":
        # every sequence holds the pages that its positions reach, scattered over a pool that
        # earlier sequences have filled; those before a window have been given back
        gone = [0] * S
        if case.get("window"):
            gone = [int(lo[0]) // page if len(lo) else 0 for lo, _ in _spans(case)]
        need = [(n + c + page - 1) // page for n, c in zip(new, ctx)]
        pool = sum(need) - sum(gone) + 7
        order = torch.randperm(pool, device=dev, generator=g).to(torch.int32)
        slot, at = np.full((S, max(max(need), 1)), -1, dtype=np.int64), 0
        for s, m in enumerate(need):
            slot[s, gone[s]:m] = np.arange(at, at + m - gone[s])
            at += m - gone[s]
        slot = torch.from_numpy(slot).to(dev)
        st["page_table"] = torch.where(slot >= 0, order[slot.clamp(min=0)], -1).to(torch.int32).contiguous()
        st["k_cache"], st["v_cache"] = normal(pool, KV, page, hd, dtype=ct), normal(pool, KV, page, hd, dtype=ct)
    if case["op"] == "append":
        # the rotation's (cos, sin) by position and pair, theta 500,000
        i = torch.arange(hd // 2, device=dev, dtype=torch.float64)
        angle = torch.arange(st["len_max"], device=dev, dtype=torch.float64)[:, None] * 500000.0 ** (-2.0 * i / hd)
        st["rope"] = torch.stack([angle.cos(), angle.sin()], dim=-1).float().contiguous()
        # text counts all axes up together; an image's rows and columns count on from its start
        r = random.Random(case["lens"] + 2)
        pos = np.zeros((case["axes"], rows), dtype=np.int64)
        for s, (n, c) in enumerate(zip(new, ctx)):
            i, at = 0, r.randint(0, c)
            while i < n:
                m = min(n - i, r.randint(1, 200))
                x, w = np.arange(m), r.randint(1, 24)
                image = r.random() < 0.5
                for a in range(case["axes"]):
                    turn = (x * 0, x // w, x % w, x % 2)[a] if image else x
                    pos[a, starts[s] + i:starts[s] + i + m] = at + turn
                at = int(pos[:, starts[s] + i:starts[s] + i + m].max()) + 1
                i += m
        st["axis"] = _axis_map(case)
        st["positions"] = torch.from_numpy(pos).to(dev, torch.int32)
        return st
    first, prefix = _masks(case)
    st["scores"] = dict(cap=case["cap"], window=case["window"], slopes=None, first=None, prefix_len=None)
    if case["slopes"]:
        st["scores"]["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device=dev)
    if case["prefix"]:
        st["scores"]["prefix_len"] = _ints(prefix)
    if first is not None:
        flat = np.concatenate(first + [np.zeros(rows - used, dtype=np.int64)])
        st["scores"]["first"] = torch.from_numpy(flat).to(dev, torch.int32)
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    if own:
        return _run_own(st)
    if st["op"] == "sample":
        return _plain_sample(st)
    if st["op"] == "plan":
        return _plain_plan(st)
    if st["op"] == "append":
        return _plain_append(st)
    if st["op"] == "paged":
        return _plain_attention(st, _pages(st, st["k_cache"]), _pages(st, st["v_cache"]), st["ctx_len"].long())
    at = st["row_start"][:-1, None].long() + torch.arange(st["new_max"], device=st["q"].device)
    at = at.clamp(max=st["k"].shape[0] - 1)
    return _plain_attention(st, st["k"].float()[at], st["v"].float()[at], torch.zeros_like(st["ctx_len"]).long())


_PLANNED = ("row_start", "ctx_len", "positions", "slots", "page_table", "seq_len_out", "free_count_out", "free_pages")


def _run_own(st):
    import llama_decode_kv_gb300 as slm
    if st["op"] == "sample":
        slm.sample_rows(st["logits"], st["temperature"], st["top_k"], st["top_p"], st["min_p"], st["uniforms"], st["ids"])
        return {"ids": st["ids"]}
    if st["op"] == "plan":
        slm.rows_plan(st["new_len"], st["seq_len"], st["page_table"], st["page"], st["free_pages"], st["free_count"],
                      st["row_start"], st["ctx_len"], st["positions"], st["slots"], st["seq_len_out"],
                      st["free_count_out"], st["status"])
        return {k: st[k] for k in _PLANNED}
    if st["op"] == "append":
        slm.kv_append_axes(st["k"], st["v"], st["k_cache"], st["v_cache"], st["page_table"], st["row_start"],
                           st["ctx_len"], st["status"], st["rope"], st["axis"], st["positions"], q=st["q"],
                           q_out=st["out"])
        return {"k_cache": st["k_cache"], "v_cache": st["v_cache"], "q": st["out"]}
    if st["ws"] is None:  # a program keeps one workspace for its shapes
        rows, H, hd = st["q"].shape
        KV = st["k"].shape[1] if st["op"] == "prompt" else st["k_cache"].shape[1]
        st["ws"] = torch.empty(slm.attention_rows_workspace_bytes(st["q"].dtype, rows, st["row_start"].numel() - 1, H, KV, hd),
                               dtype=torch.uint8, device=st["q"].device)
    if st["op"] == "paged":
        slm.attention_paged_scored(st["q"], st["k_cache"], st["v_cache"], st["page_table"], st["row_start"],
                                   st["ctx_len"], st["out"], st["ws"], st["status"], **st["scores"])
    else:
        slm.attention_prompt_scored(st["q"], st["k"], st["v"], st["row_start"], st["out"], st["ws"], st["status"],
                                    **st["scores"])
    return {"out": st["out"]}


def _plain_sample(st):
    # in 64 bits: the draw ends next to the border of two tokens' masses
    x = st["logits"].float()
    R, V = x.shape
    best = x.argmax(dim=1)  # the lowest index of the largest logits
    T = st["temperature"][:, None]
    val, order = torch.sort(x, dim=1, descending=True, stable=True)
    w = ((val.double() - val[:, :1].double()) / torch.where(T > 0, T, 1.0).double()).exp()
    rank = torch.arange(V, device=x.device)[None]
    k = st["top_k"][:, None]
    w = torch.where((k <= 0) | (rank < k), w, 0.0)
    run_sum = w.cumsum(dim=1)
    p = st["top_p"][:, None].double()
    before = run_sum - w
    keep = (p >= 1) | (before < p * run_sum[:, -1:])
    keep &= w >= st["min_p"][:, None].double()
    w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0.0))
    c = w.cumsum(dim=1)
    hit = (c > st["uniforms"][:, None].double() * c[:, -1:]).to(torch.int8)
    ids = torch.where(T[:, 0] > 0, hit.argmax(dim=1), best)
    return {"ids": ids.to(torch.int32)}


def _plain_plan(st):
    P, new, ctx = st["page"], st["new_len"].long(), st["seq_len"].long()
    table, dev = st["page_table"], st["new_len"].device
    ends, n = new < 0, new.clamp(min=0)
    held = (ctx + P - 1) // P
    need = torch.where(ends, 0, (ctx + n + P - 1) // P - held)
    back = torch.where(ends, held, 0)
    F = st["free_count"].long()
    block = torch.arange(table.shape[1], device=dev)
    # the ended sequences' pages, then the new ones from the top of the stack
    s, b = torch.nonzero(block[None] < back[:, None], as_tuple=True)
    st["free_pages"][F + torch.arange(s.numel(), device=dev)] = table[s, b]
    s, b = torch.nonzero((block[None] >= held[:, None]) & (block[None] < (held + need)[:, None]), as_tuple=True)
    table[s, b] = st["free_pages"][F + back.sum() - 1 - torch.arange(s.numel(), device=dev)]
    start = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), n.cumsum(0)])
    r = torch.arange(st["positions"].numel(), device=dev)
    owner = torch.searchsorted(start[1:], r, right=True)
    mine = owner < new.numel()
    owner = owner.clamp(max=new.numel() - 1)
    pos = torch.where(mine, ctx[owner] + r - start[owner], 0)
    slot = table[owner, pos // P].long() * P + pos % P
    return {"row_start": start.int(), "ctx_len": torch.where(ends, 0, ctx).int(), "positions": torch.where(mine, pos, -1).int(),
            "slots": torch.where(mine, slot, -1), "page_table": table,
            "seq_len_out": torch.where(ends, 0, ctx + n).int(),
            "free_count_out": (F + back.sum() - need.sum()).int(), "free_pages": st["free_pages"]}


def _owners(st):
    """(sequence, number within it) of every row that belongs to a sequence."""
    r = torch.arange(st["used"], device=st["q"].device)
    s = torch.searchsorted(st["row_start"][1:].long(), r, right=True)
    return s, r - st["row_start"].long()[s]


def _rotate(x, cs):
    """Rotate the pairs (i, i + head_dim / 2) of x [rows][heads][head_dim]."""
    a, b = x.float().chunk(2, dim=-1)
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    return torch.cat([a * c - b * s, a * s + b * c], dim=-1)


def _plain_append(st):
    s, n = _owners(st)
    pos = st["ctx_len"].long()[s] + n
    page = st["k_cache"].shape[2]
    pages, slots = st["page_table"].long()[s, pos // page], pos % page
    axis = torch.tensor(st["axis"], device=pos.device)
    turn = st["positions"][:, :st["used"]].long()[axis.clamp(min=0)].t()  # [rows][pairs]
    cs = st["rope"][turn, torch.arange(axis.numel(), device=pos.device)]
    cs = torch.where((axis >= 0)[None, :, None], cs, torch.tensor([1.0, 0.0], device=pos.device))
    st["k_cache"][pages, :, slots] = _rotate(st["k"][:st["used"]], cs).to(st["k_cache"].dtype)
    st["v_cache"][pages, :, slots] = st["v"][:st["used"]].to(st["v_cache"].dtype)
    out = torch.zeros_like(st["out"])
    out[:st["used"]] = _rotate(st["q"][:st["used"]], cs).to(out.dtype)
    return {"k_cache": st["k_cache"], "v_cache": st["v_cache"], "q": out}


def _pages(st, cache):
    """[sequences][positions][kv heads][head_dim] of a paged cache, in 32 bits."""
    S = st["page_table"].shape[0]
    x = cache[st["page_table"].long().clamp(min=0)].permute(0, 1, 3, 2, 4)
    return x.reshape(S, -1, cache.shape[1], cache.shape[3])[:, :st["len_max"]].float()


def _plain_attention(st, k, v, ctx):
    S, L, KV, hd = k.shape
    H, N = st["q"].shape[1], st["new_max"]
    G, sc = H // KV, st["scores"]
    step = torch.arange(N, device=k.device)
    rows = (st["row_start"][:-1, None].long() + step).clamp(max=st["q"].shape[0] - 1)
    q = st["q"].float()[rows].view(S, N, KV, G, hd).permute(0, 2, 3, 1, 4).reshape(S, KV, G * N, hd)
    x = (q @ k.permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(hd)).view(S, KV, G, N, L)
    if sc["cap"]:
        x = x.div_(sc["cap"]).tanh_().mul_(sc["cap"])
    t = torch.arange(L, device=k.device)
    p = (ctx[:, None] + step)[:, :, None]  # [sequences][new][1]
    if sc["slopes"] is not None:
        far = (p - t).abs().float()[:, None, None]
        x = x.addcmul_(sc["slopes"].view(1, KV, G, 1, 1), far, value=-1.0)
    end = p + 1 if sc["prefix_len"] is None else torch.maximum(p + 1, sc["prefix_len"].long()[:, None, None])
    seen = t < end
    if sc["window"]:
        seen = seen & (t > p - sc["window"])
    if sc["first"] is not None:
        seen = seen & (t >= sc["first"].long()[rows][:, :, None])
    seen = seen[:, None, None]
    x = x.masked_fill_(~seen, -math.inf)
    top = x.amax(dim=-1, keepdim=True)
    x = x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    o = x.view(S, KV, G * N, L) @ v.permute(0, 2, 1, 3)
    total = x.sum(dim=-1).view(S, KV, G * N, 1)
    o = (o / torch.where(total > 0, total, 1.0)).view(S, KV, G, N, hd).permute(0, 3, 1, 2, 4).reshape(S, N, H, hd)
    s, n = _owners(st)
    out = torch.zeros_like(st["out"])
    out[:st["used"]] = o[s, n].to(out.dtype)
    return {"out": out}


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"sample": _exact_sample, "plan": _exact_plan, "append": _exact_append}.get(case["op"], _exact_attention)(case, st)


def _exact_sample(case, st):
    logits = st["logits"].float().cpu().numpy()
    T, k, p, m, u = (st[n].cpu().numpy() for n in ("temperature", "top_k", "top_p", "min_p", "uniforms"))
    ids = []
    for r in range(case["rows"]):
        x = logits[r].astype(np.float64)
        if not T[r] > 0:
            ids.append(int(np.flatnonzero(x == x.max())[0]))
            continue
        order = np.lexsort((np.arange(x.size), -x))
        if 0 < k[r] < x.size:
            order = order[:k[r]]
        w = np.exp((x[order] - x[order[0]]) / np.float64(T[r]))
        if p[r] < 1:
            enough = np.flatnonzero(np.cumsum(w) >= np.float64(p[r]) * w.sum())
            n = int(enough[0]) + 1 if enough.size else order.size
            order, w = order[:n], w[:n]
        order, w = order[w >= np.float64(m[r])], w[w >= np.float64(m[r])]
        by_index = np.argsort(order)
        c = np.cumsum(w[by_index])
        ids.append(int(order[by_index][np.flatnonzero(c > np.float64(u[r]) * c[-1])[0]]))
    return {"ids": torch.tensor(ids, dtype=torch.int32, device="cuda")}


def _exact_plan(case, st):
    new, ctx = _lengths(case)
    P, table = case["page"], st["page_table"].tolist()
    stack = st["free_pages"].tolist()
    n_free = int(st["free_count"])
    for s, n in enumerate(new):
        if n < 0:
            for b in range((ctx[s] + P - 1) // P):
                stack[n_free] = table[s][b]
                n_free += 1
    start, pos, slots, after = [0], [], [], []
    for s, n in enumerate(new):
        for i in range(max(n, 0)):
            at = ctx[s] + i
            if at % P == 0:
                n_free -= 1
                table[s][at // P] = stack[n_free]
            pos.append(at)
            slots.append(table[s][at // P] * P + at % P)
        start.append(len(pos))
        after.append(0 if n < 0 else ctx[s] + n)
    nobody = [-1] * case["pad"]
    return {"row_start": _ints(start), "ctx_len": _ints([0 if n < 0 else c for n, c in zip(new, ctx)]),
            "positions": _ints(pos + nobody), "slots": _ints(slots + nobody, torch.int64), "page_table": _ints(table),
            "seq_len_out": _ints(after), "free_count_out": _ints([n_free]), "free_pages": _ints(stack)}


def _exact_append(case, st):
    new, ctx = _lengths(case)
    half, page = case["head_dim"] // 2, case["page"]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    kc, vc = st["k_cache"].double(), st["v_cache"].double()
    table = st["page_table"].tolist()
    first = 0
    for s in range(case["nseq"]):
        n, c = new[s], ctx[s]
        if n == 0:
            continue
        turn = torch.ones(n, 1, half, dtype=torch.complex128, device="cuda")
        for j, a in enumerate(st["axis"]):
            if a >= 0:
                angle = st["rope"][st["positions"][a, first:first + n].long(), j].double()
                turn[:, 0, j] = torch.complex(angle[:, 0].contiguous(), angle[:, 1].contiguous())
        for src in ("q", "k"):
            x = st[src][first:first + n].double()
            y = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * turn
            y = torch.cat([y.real, y.imag], dim=-1)
            if src == "q":
                out[first:first + n] = y
        p = c
        while p < c + n:  # page by page
            m = min(page - p % page, c + n - p)
            i, j = p - c, p % page
            kc[table[s][p // page], :, j:j + m] = y[i:i + m].transpose(0, 1)
            vc[table[s][p // page], :, j:j + m] = st["v"][first + i:first + i + m].double().transpose(0, 1)
            p += m
        first += n
    return {"k_cache": kc, "v_cache": vc, "q": out}


def _exact_attention(case, st):
    new, ctx = _lengths(case)
    H, KV, hd, page = case["heads"], case["kv_heads"], case["head_dim"], case["page"]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    row0 = 0
    for s, (lo, hi) in enumerate(_spans(case)):
        n, c = new[s], ctx[s]
        seen = hi > lo
        if not seen.any():
            row0 += n
            continue
        a0, a1 = int(lo[seen].min()), int(hi[seen].max())  # nothing else is looked at
        t = torch.arange(a0, a1, device="cuda")
        lo_t, hi_t = (torch.from_numpy(x).cuda()[:, None] for x in (lo, hi))
        hidden = (t < lo_t) | (t >= hi_t)
        p = torch.arange(c, c + n, device="cuda")[:, None]
        live = torch.from_numpy(seen).cuda()
        for g in range(KV):
            if case["op"] == "paged":
                ids = st["page_table"][s].long()[t // page]
                k, v = (st[w][ids, g, t % page].double() for w in ("k_cache", "v_cache"))
            else:
                k, v = (st[w][row0 + a0:row0 + a1, g].double() for w in ("k", "v"))
            for h in range(g * (H // KV), (g + 1) * (H // KV)):
                x = st["q"][row0:row0 + n, h].double() @ k.t() / math.sqrt(hd)
                if case["cap"]:
                    x = case["cap"] * torch.tanh(x / case["cap"])
                if case["slopes"]:
                    x = x - st["scores"]["slopes"][h].double() * (p - t).abs()
                w = torch.softmax(x[live].masked_fill_(hidden[live], -math.inf), dim=-1)
                out[row0:row0 + n, h][live] = w @ v
        row0 += n
    return {"out": out}
