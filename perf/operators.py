"""Measured cases of the packed-row cache operators: appending keys and values to a paged
cache with the position rotation on the way, attention of new rows (a chunk of a prompt, or
one token) over a paged cache, and causal attention over whole packed prompts.

The rows of a batch are packed: rows [row_start[s], row_start[s + 1]) belong to sequence s.
A sequence has ctx_len[s] positions cached before its new rows; row i of it stands at
position ctx_len[s] + i.  Query head h reads kv head h // (heads / kv heads).

``run`` is one pass: with ``own`` the calls of the library, without it the same operators in
elementary torch operations, in 32 bits, rounded once at the end.  ``exact`` is the
definition in 64 bits, one sequence and kv head at a time.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # The next token of one chat, SmolLM2-135M heads: a launch's latency.
        dict(name="append_one_token", op="append", dtype="f32", cache="bf16", heads=9, kv_heads=3, head_dim=64,
             page=16, nseq=1, new=1, ctx=261, even=True, idle=0, pad=0, lens=1),
        # One decode step of a large batch with contexts of all lengths.
        dict(name="append_decode_batch", op="append", dtype="bf16", cache="bf16", heads=32, kv_heads=8, head_dim=128,
             page=64, nseq=256, new=1, ctx=8000, even=False, idle=0, pad=0, lens=2),
        # The prompts of a batch, straight from an fp32 projection into a bf16 cache, with
        # rows of a fixed-size buffer left over behind the last prompt.
        dict(name="append_prompts", op="append", dtype="f32", cache="bf16", heads=32, kv_heads=8, head_dim=64,
             page=64, nseq=16, new=1024, ctx=0, even=False, idle=0, pad=37, lens=3),
        # SmolLM2's 16 prompts of 512 tokens: short prompts, three query heads to a kv head.
        dict(name="prompt_batch16", op="prompt", dtype="bf16", cache="bf16", heads=9, kv_heads=3, head_dim=64,
             page=0, nseq=16, new=512, ctx=0, even=True, idle=0, pad=0, lens=4),
        # One Llama-3.2-1B prompt of 2,048 tokens.
        dict(name="prompt_2048", op="prompt", dtype="bf16", cache="bf16", heads=32, kv_heads=8, head_dim=64,
             page=0, nseq=1, new=2048, ctx=0, even=True, idle=0, pad=0, lens=5),
        # Long documents of different lengths with 128-wide heads: the tensor cores' case.
        dict(name="prompt_long", op="prompt", dtype="bf16", cache="bf16", heads=32, kv_heads=8, head_dim=128,
             page=0, nseq=2, new=8192, ctx=0, even=False, idle=0, pad=19, lens=6),
        # Ragged short prompts of an fp32 engine.
        dict(name="prompt_f32_ragged", op="prompt", dtype="f32", cache="f32", heads=9, kv_heads=3, head_dim=64,
             page=0, nseq=7, new=701, ctx=0, even=False, idle=0, pad=5, lens=7),
        # The next token of one chat of a few hundred tokens.
        dict(name="paged_one_token", op="paged", dtype="bf16", cache="bf16", heads=9, kv_heads=3, head_dim=64,
             page=16, nseq=1, new=1, ctx=261, even=True, idle=0, pad=0, lens=8),
        # Llama-3.2-1B's long-context step: 4 sequences of 32,768 cached positions.
        dict(name="paged_long_context", op="paged", dtype="bf16", cache="bf16", heads=32, kv_heads=8, head_dim=64,
             page=64, nseq=4, new=1, ctx=32768, even=True, idle=0, pad=0, lens=9),
        # A serving batch's step: 64 sequences with contexts of all lengths.
        dict(name="paged_decode_batch", op="paged", dtype="bf16", cache="bf16", heads=32, kv_heads=8, head_dim=128,
             page=64, nseq=64, new=1, ctx=8000, even=False, idle=0, pad=0, lens=10),
        # Chunked prefill of three long prompts, ragged chunks of up to 512 tokens.
        dict(name="paged_chunk", op="paged", dtype="bf16", cache="bf16", heads=32, kv_heads=8, head_dim=128,
             page=128, nseq=3, new=512, ctx=16000, even=False, idle=0, pad=11, lens=11),
        # An fp32 engine's mixed batch: short chunks and single tokens, one slot idle.
        dict(name="paged_f32_mixed", op="paged", dtype="f32", cache="f32", heads=9, kv_heads=3, head_dim=64,
             page=64, nseq=12, new=33, ctx=1000, even=False, idle=5, pad=3, lens=12),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "prompt", "paged", "paged"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    heads, kv_heads, head_dim = rng.choice([(9, 3, 64), (32, 8, 64), (32, 8, 128), (8, 1, 128), (16, 16, 64),
                                            (12, 4, 80), (10, 2, 96), (4, 2, 16), (15, 5, 72), (6, 6, 128)])
    page = rng.choice([16, 32, 64, 128, 256])
    even = rng.random() < 0.3
    lens = rng.randrange(1 << 20)
    pad = rng.choice([0, 0, rng.randrange(1, 64)])
    idle = rng.choice([0, 0, 3, 5])
    if op == "append":
        cache = rng.choice(["bf16", dtype])
        nseq = _spread(rng, 1, 256)
        new = rng.choice([1, _spread(rng, 2, max(2, 16384 // nseq))])
        ctx = rng.choice([0, _spread(rng, 1, 8000)])
    elif op == "prompt":
        cache, page, ctx = dtype, 0, 0
        nseq = _spread(rng, 1, 24)
        new = _spread(rng, 1, (8192 if nseq == 1 else 4096 if nseq <= 4 else 1024) if dtype == "bf16" else 512)
    else:
        cache = dtype
        nseq = _spread(rng, 1, 48)
        new = rng.choice([1, 1, _spread(rng, 2, 512 if nseq <= 4 else 48)])
        ctx = _spread(rng, 1, (30000 if nseq <= 4 else 6000) if dtype == "bf16" else 2000)
    return dict(op=op, dtype=dtype, cache=cache, heads=heads, kv_heads=kv_heads, head_dim=head_dim, page=page,
                nseq=nseq, new=new, ctx=ctx, even=even, idle=idle, pad=pad, lens=lens)


def _lengths(case):
    """(new rows, cached positions) of every sequence.  The first has the largest of both;
    with `idle`, every idle-th sequence has no new row."""
    r = random.Random(case["lens"])
    new, ctx = [], []
    for s in range(case["nseq"]):
        full = case["even"] or s == 0
        n = case["new"] if full else r.randint(1, case["new"])
        c = case["ctx"] if full else r.randint(0, case["ctx"])
        if case["idle"] and s % case["idle"] == case["idle"] - 1:
            n = 0
        new.append(n)
        ctx.append(c)
    return new, ctx


def work(case):
    new, ctx = _lengths(case)
    rows, H, KV, hd = sum(new), case["heads"], case["kv_heads"], case["head_dim"]
    e, ec = (4 if case[k] == "f32" else 2 for k in ("dtype", "cache"))
    if case["op"] == "append":
        # q, k, v and the rotation in; the rotated q and the cache rows out
        rope = max(n + c for n, c in zip(new, ctx)) if case["nseq"] > 1 else rows
        return {"bytes": rows * hd * ((H + 2 * KV) * (e + ec)) + min(rows, rope) * hd * 4,
                "flops": 3 * rows * hd * (H + KV)}
    pairs = sum(n * c + n * (n + 1) // 2 for n, c in zip(new, ctx))
    cached = sum(n + c for n, c in zip(new, ctx) if n)
    return {"bytes": 2 * rows * H * hd * e + 2 * cached * KV * hd * ec, "flops": 4 * pairs * H * hd}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    new, ctx = _lengths(case)
    H, KV, hd, S, page = case["heads"], case["kv_heads"], case["head_dim"], case["nseq"], case["page"]
    used = sum(new)
    rows = used + case["pad"]
    t, ct = _TYPES[case["dtype"]], _TYPES[case["cache"]]

    def normal(*shape, dtype=t, scale=1.0):
        x = torch.randn(*shape, device=dev, dtype=torch.float32 if dtype == torch.float32 else torch.bfloat16, generator=g)
        return x.mul_(scale).to(dtype)

    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    st = dict(op=case["op"], used=used, new_max=max(new), len_max=max(n + c for n, c in zip(new, ctx)), ws=None,
              row_start=torch.tensor(starts, dtype=torch.int32, device=dev),
              ctx_len=torch.tensor(ctx, dtype=torch.int32, device=dev),
              status=torch.zeros(1, dtype=torch.int32, device=dev),
              # trained queries point somewhere: scores spread by a few units
              q=normal(max(rows, 1), H, hd, scale=2.0), out=torch.zeros(max(rows, 1), H, hd, dtype=ct, device=dev))
    if case["op"] != "paged":
        st["k"], st["v"] = normal(max(rows, 1), KV, hd), normal(max(rows, 1), KV, hd)
    if case["op"] != "prompt":
        # every sequence holds the pages its positions reach, scattered over a pool that
        # earlier sequences have filled
        need = [(n + c + page - 1) // page for n, c in zip(new, ctx)]
        pool = sum(need) + 7
        order = torch.randperm(pool, device=dev, generator=g).to(torch.int32)
        slot, at = [[-1] * max(max(need), 1) for _ in range(S)], 0
        for s, m in enumerate(need):
            slot[s][:m] = range(at, at + m)
            at += m
        slot = torch.tensor(slot, dtype=torch.int64, device=dev)
        st["page_table"] = torch.where(slot >= 0, order[slot.clamp(min=0)], torch.full_like(slot, -1, dtype=torch.int32)).contiguous()
        st["k_cache"], st["v_cache"] = normal(pool, KV, page, hd, dtype=ct), normal(pool, KV, page, hd, dtype=ct)
    if case["op"] == "append":
        # the rotation's (cos, sin) by position, theta 500,000
        i = torch.arange(hd // 2, device=dev, dtype=torch.float64)
        angle = torch.arange(st["len_max"], device=dev, dtype=torch.float64)[:, None] * 500000.0 ** (-2.0 * i / hd)
        st["rope"] = torch.stack([angle.cos(), angle.sin()], dim=-1).float().contiguous()
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    if own:
        return _run_own(st)
    if st["op"] == "append":
        return _plain_append(st)
    if st["op"] == "paged":
        return _plain_attention(st, _pages(st, st["k_cache"]), _pages(st, st["v_cache"]), st["ctx_len"].long())
    at = st["row_start"][:-1, None].long() + torch.arange(st["new_max"], device=st["q"].device)
    at = at.clamp(max=st["k"].shape[0] - 1)
    return _plain_attention(st, st["k"].float()[at], st["v"].float()[at], torch.zeros_like(st["ctx_len"]).long())


def _run_own(st):
    import llama_decode_kv_gb300 as slm
    if st["op"] == "append":
        slm.kv_append(st["k"], st["v"], st["k_cache"], st["v_cache"], st["page_table"], st["row_start"], st["ctx_len"],
                      st["status"], rope=st["rope"], q=st["q"], q_out=st["out"])
        return {"k_cache": st["k_cache"], "v_cache": st["v_cache"], "q": st["out"]}
    if st["ws"] is None:  # a program keeps one workspace for its shapes
        rows, H, hd = st["q"].shape
        KV = st["k"].shape[1] if st["op"] == "prompt" else st["k_cache"].shape[1]
        st["ws"] = torch.empty(slm.attention_rows_workspace_bytes(st["q"].dtype, rows, st["row_start"].numel() - 1, H, KV, hd),
                               dtype=torch.uint8, device=st["q"].device)
    if st["op"] == "paged":
        slm.attention_paged(st["q"], st["k_cache"], st["v_cache"], st["page_table"], st["row_start"], st["ctx_len"],
                            st["out"], st["ws"], st["status"])
    else:
        slm.attention_prompt(st["q"], st["k"], st["v"], st["row_start"], st["out"], st["ws"], st["status"])
    return {"out": st["out"]}


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
    cs = st["rope"][pos]
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
    G = H // KV
    step = torch.arange(N, device=k.device)
    rows = (st["row_start"][:-1, None].long() + step).clamp(max=st["q"].shape[0] - 1)
    q = st["q"].float()[rows].view(S, N, KV, G, hd).permute(0, 2, 3, 1, 4).reshape(S, KV, G * N, hd)
    x = (q @ k.permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(hd)).view(S, KV, G, N, L)
    seen = torch.arange(L, device=k.device) <= (ctx[:, None] + step)[:, :, None]
    x = torch.where(seen[:, None, None], x, -math.inf)
    x = (x - x.amax(dim=-1, keepdim=True)).exp_()
    o = (x.view(S, KV, G * N, L) @ v.permute(0, 2, 1, 3)) / x.sum(dim=-1).view(S, KV, G * N, 1)
    o = o.view(S, KV, G, N, hd).permute(0, 3, 1, 2, 4).reshape(S, N, H, hd)
    s, n = _owners(st)
    out = torch.zeros_like(st["out"])
    out[:st["used"]] = o[s, n].to(out.dtype)
    return {"out": out}


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    new, ctx = _lengths(case)
    H, KV, hd = case["heads"], case["kv_heads"], case["head_dim"]
    G, page, half = H // KV, case["page"], hd // 2
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=st["q"].device)
    if case["op"] == "append":
        kc, vc = st["k_cache"].double(), st["v_cache"].double()
        table = st["page_table"].tolist()
        first = 0
        for s in range(case["nseq"]):
            n, c = new[s], ctx[s]
            if n == 0:
                continue
            angle = st["rope"][c:c + n].double()
            turn = torch.complex(angle[..., 0], angle[..., 1])[:, None]
            for src, dst in ((st["q"], None), (st["k"], kc)):
                x = src[first:first + n].double()
                y = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * turn
                y = torch.cat([y.real, y.imag], dim=-1)
                if dst is None:
                    out[first:first + n] = y
                else:
                    rotated = y
            p = c
            while p < c + n:  # page by page
                m = min(page - p % page, c + n - p)
                i, j = p - c, p % page
                kc[table[s][p // page], :, j:j + m] = rotated[i:i + m].transpose(0, 1)
                vc[table[s][p // page], :, j:j + m] = st["v"][first + i:first + i + m].double().transpose(0, 1)
                p += m
            first += n
        return {"k_cache": kc, "v_cache": vc, "q": out}
    first = 0
    for s in range(case["nseq"]):
        n, c = new[s], ctx[s]
        if n == 0:
            continue
        hidden = torch.ones(n, c + n, dtype=torch.bool, device=out.device).triu(c + 1)
        if case["op"] == "paged":
            ids = st["page_table"][s, :(c + n + page - 1) // page].long()
        for g in range(KV):
            if case["op"] == "paged":
                k = st["k_cache"][ids, g].reshape(-1, hd)[:c + n].double()
                v = st["v_cache"][ids, g].reshape(-1, hd)[:c + n].double()
            else:
                k, v = (st[w][first:first + n, g].double() for w in ("k", "v"))
            for h in range(g * G, g * G + G):
                a = st["q"][first:first + n, h].double() @ k.t() / math.sqrt(hd)
                out[first:first + n, h] = torch.softmax(a.masked_fill_(hidden, -math.inf), dim=-1) @ v
        first += n
    return {"out": out}
