"""Scored attention of packed rows on the GPU -- slm_attention_paged_scored and
slm_attention_prompt_scored: capped scores, distances, windows, documents, prefixes -- against the
definition in 64 bits.

Tolerances (u = 2^-24, h = 2^-8, half a step of bf16): q . k is off by ds as in test_gpu_rows.  A cap's
tanh has a slope of at most 1, so ds stays, and is off by 2^-20 of itself (its polynomial: 2^-20.4; tanhf:
less), a distance's term by its rounding and the position difference's, 3 u |slope d|; scores are then
rounded twice more, in the natural and the log2 domain: with X the largest |x| and B the largest
|slope d| that the row sees, a score is off by e = ds + 2^-20 X + 4 u (X + B).  A weight is off by the factor
1 +- (e + 8 u), the output by 2 (e + 8 u) vmax, the sums over L positions add L 2^-22 vmax; bf16 calls
round the weights (h A, with A the weighted mean of |v|) and the result (h |out|)."""
import math

import pytest

from test_gpu_rows import BF16, F32, H16, U, Batch, slm  # noqa: F401  (slm: the fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def spans(b, m):
    """(from, to) of every sequence's rows under the masks m."""
    out = []
    for s, (n, c) in enumerate(zip(b.new, b.ctx)):
        p = torch.arange(c, c + n)
        lo = torch.zeros(n, dtype=torch.long)
        if m.get("window"):
            lo = torch.maximum(lo, p + 1 - m["window"])
        if m.get("first") is not None:
            lo = torch.maximum(lo, torch.tensor(m["first"][s], dtype=torch.long))
        hi = p + 1
        if m.get("prefix") is not None:
            hi = torch.clamp(hi, min=min(max(m["prefix"][s], 0), n + c))
        out.append((lo, hi))
    return out


def documents(b, seed, most, separators=True):
    """first[] of every sequence: documents of 1 to `most` positions; some end in a row that sees nothing."""
    import random
    r = random.Random(seed)
    first = []
    for n, c in zip(b.new, b.ctx):
        of, at = [], 0
        while at < n + c:
            end = min(n + c, at + r.randint(1, most))
            of += [at] * (end - at)
            if separators and r.random() < 0.3:
                of[-1] = end
            at = end
        first.append(of[c:])
    return first


def arguments(b, m):
    """The keyword arguments of a call."""
    kw = {k: m[k] for k in ("scale", "cap", "window") if k in m}
    if m.get("slopes"):
        kw["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / b.H) for h in range(b.H)], device="cuda")
    if m.get("prefix") is not None:
        kw["prefix_len"] = torch.tensor(m["prefix"], dtype=torch.int32, device="cuda")
    if m.get("first") is not None:
        flat = [7 << 20] * b.rows
        for s, f in enumerate(m["first"]):
            flat[b.starts[s]:b.starts[s] + len(f)] = f
        kw["first"] = torch.tensor(flat, dtype=torch.int32, device="cuda")
    return kw


def check(b, out, keys, values, m, kw, dtype):
    worst = 0.0
    for s, (lo, hi) in enumerate(spans(b, m)):
        n, c = b.new[s], b.ctx[s]
        if n == 0:
            continue
        rows = slice(b.starts[s], b.starts[s] + n)
        L = n + c
        p, t = torch.arange(c, L, device="cuda")[:, None], torch.arange(L, device="cuda")[None]
        hide = (t < lo.cuda()[:, None]) | (t >= hi.cuda()[:, None])
        blind = (lo >= hi).cuda()
        assert bool((out[rows][blind] == 0).all()), "rows that see nothing"
        scale = m.get("scale") or 1 / math.sqrt(b.hd)
        k64 = torch.where(torch.isfinite(keys[s]), keys[s], 0).double()
        v64 = torch.where(torch.isfinite(values[s]), values[s], 0).double()
        seen = ~hide[~blind]
        vmax = float(v64[seen.any(0)].abs().max()) if seen.numel() and bool(seen.any()) else 0.0
        for h in range(b.H):
            q = b.q[rows, h].double()[~blind]
            if q.shape[0] == 0:
                continue
            kk, vv, hd = k64[:, h // (b.H // b.KV)], v64[:, h // (b.H // b.KV)], hide[~blind]
            x = scale * (q @ kk.t())
            ds = (q.abs() @ kk.abs().t()).masked_fill(hd, 0).amax(-1, keepdim=True) * scale * 2.0 ** -22 * (b.hd + 8)
            if m.get("cap"):
                x = m["cap"] * torch.tanh(x / m["cap"])
            X, B = x.abs().masked_fill(hd, 0).amax(-1, keepdim=True), 0.0
            if m.get("slopes"):
                bias = kw["slopes"][h].double() * (p - t).abs()[~blind]
                B = bias.abs().masked_fill(hd, 0).amax(-1, keepdim=True)
                x = x - bias
            w = torch.softmax(x.masked_fill(hd, -math.inf), dim=-1)
            want, mean = w @ vv, w @ vv.abs()
            e = ds + 2.0 ** -20 * X + 4 * U * (X + B)
            tol = 2 * (e + 8 * U) * vmax + L * 2.0 ** -22 * vmax
            tol = tol + (H16 * (mean + want.abs()) if dtype == BF16 else U * want.abs())
            d = (out[rows, h].double()[~blind] - want).abs()
            assert bool((d <= tol).all()), (s, h, float((d / tol).nan_to_num(nan=9e9).max()))
            worst = max(worst, float((d / tol).max()))
    nobody = list(range(b.starts[0])) + list(range(b.starts[-1], b.rows))
    assert bool((out[nobody] == 7.0).all()), "rows of nobody were written"
    assert int(b.status.item()) == 0
    return worst


HEADS = [(BF16, 9, 3, 64), (BF16, 32, 8, 128), (BF16, 8, 1, 128), (BF16, 4, 2, 16), (BF16, 12, 4, 80), (BF16, 64, 1, 64),
         (BF16, 4, 2, 160), (F32, 9, 3, 64), (F32, 4, 2, 128), (F32, 2, 1, 256), (F32, 6, 6, 72)]
CHUNKS = ([200, 1, 30, 0, 257, 64], [10, 300, 0, 50, 700, 1000])
STEPS = ([1, 1, 1, 0, 1, 1], [0, 5, 300, 9, 1500, 127])
MASKS = ["plain", "cap", "small_cap", "slopes", "window1", "window", "docs", "prefix", "all", "all_prefix"]


def masks(b, name):
    if name == "plain":
        return dict(scale=0.3)
    if name == "cap":
        return dict(cap=30.0)
    if name == "small_cap":  # most products are beyond it
        return dict(cap=0.7)
    if name == "slopes":
        return dict(slopes=True)
    if name == "window1":
        return dict(window=1, cap=5.0)
    if name == "window":
        return dict(window=150)
    if name == "docs":
        return dict(first=documents(b, 3, 90))
    prefix = [((n + c) * (i % 4)) // 3 - 2 for i, (n, c) in enumerate(zip(b.new, b.ctx))]
    if name == "prefix":
        return dict(prefix=prefix, slopes=True)
    if name == "all":
        return dict(first=documents(b, 4, 400), cap=20.0, slopes=True, window=333)
    return dict(prefix=prefix, cap=3.0, slopes=True, window=270)


def paged(slm, b, m, evict=True, **extra):
    """One call over the filled cache, with everything before a sequence's span gone."""
    kw = arguments(b, m)
    keys, values = [k.clone() for k in b.seq_k], [v.clone() for v in b.seq_v]
    b.fill([n + c for n, c in zip(b.new, b.ctx)])
    for s, (lo, hi) in enumerate(spans(b, m)):
        live = lo < hi
        start = int(lo[live].min()) if bool(live.any()) else b.new[s] + b.ctx[s]
        if bool(live.any()) and not bool(live.all()):  # an item may read from its first row's `from` on
            start = min(start, int(lo.min()))
        if not bool(live.any()):
            start = 0 if b.new[s] else start
        if not evict:
            start = 0
        for pos in range(start):
            pg = b.table[s][pos // b.page]
            if pg >= 0:
                b.k_cache[pg, :, pos % b.page] = float("nan")
                b.v_cache[pg, :, pos % b.page] = float("nan")
        for i in range(start // b.page):
            b.page_table[s, i] = -1 if i % 2 else 1 << 30
    out = b.out()
    slm.attention_paged_scored(b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, out, b.workspace(slm),
                               b.status, **kw, **extra)
    return out, keys, values, kw


@pytest.mark.parametrize("name", MASKS)
@pytest.mark.parametrize("dtype,H,KV,hd", HEADS)
def test_paged(slm, dtype, H, KV, hd, name):  # noqa: F811
    for new, ctx in (CHUNKS, STEPS):
        b = Batch(dtype, H, KV, hd, new, ctx, 16, seed=hd + H, lead=2, pad=3)
        m = masks(b, name)
        out, keys, values, kw = paged(slm, b, m)
        check(b, out, keys, values, m, kw, dtype)


@pytest.mark.parametrize("name", MASKS)
@pytest.mark.parametrize("dtype,H,KV,hd", HEADS)
def test_prompt(slm, dtype, H, KV, hd, name):  # noqa: F811
    new = [300, 1, 0, 129, 513, 64]
    b = Batch(dtype, H, KV, hd, new, seed=hd + KV, lead=1, pad=5, fused=True)
    m = masks(b, name)
    kw, out = arguments(b, m), b.out()
    slm.attention_prompt_scored(b.q, b.k, b.v, b.row_start, out, b.workspace(slm), b.status, **kw)
    keys = [b.k[a:a + n] for a, n in zip(b.starts, new)]
    values = [b.v[a:a + n] for a, n in zip(b.starts, new)]
    check(b, out, keys, values, m, kw, dtype)


@pytest.mark.parametrize("name", MASKS)
@pytest.mark.parametrize("H,KV,hd", [(9, 3, 64), (32, 8, 128), (64, 1, 64), (12, 4, 80)])
def test_wide_table(slm, H, KV, hd, name):  # noqa: F811
    """A table for many more positions than there are: the code for long items, and divided ones."""
    b = Batch(BF16, H, KV, hd, *CHUNKS, 16, seed=hd + H, lead=2, pad=3)
    b.page_table = torch.cat([b.page_table, torch.full((len(b.new), 200), -1, dtype=torch.int32, device="cuda")], 1)
    m = masks(b, name)
    out, keys, values, kw = paged(slm, b, m)
    check(b, out, keys, values, m, kw, BF16)


@pytest.mark.parametrize("name", ["plain", "cap", "small_cap", "slopes", "window", "prefix", "all_prefix"])
@pytest.mark.parametrize("H,KV,hd", [(4, 2, 64), (8, 2, 128)])
def test_long_prompt(slm, H, KV, hd, name):  # noqa: F811
    new = [2600, 1700]
    b = Batch(BF16, H, KV, hd, new, seed=hd, pad=5)
    m = masks(b, name)
    kw, out = arguments(b, m), b.out()
    slm.attention_prompt_scored(b.q, b.k, b.v, b.row_start, out, b.workspace(slm), b.status, **kw)
    check(b, out, [b.k[:2600], b.k[2600:4300]], [b.v[:2600], b.v[2600:4300]], m, kw, BF16)


@pytest.mark.parametrize("slope", [-0.3, 1.2, 40.0, -3.0])
@pytest.mark.parametrize("hd", [64, 128])
def test_steep_and_negative_slopes(slm, hd, slope):  # noqa: F811
    """Distances that outweigh the products, or draw a row to its farthest positions."""
    for new, ctx in (([70, 1], [300, 900]), ([1, 1], [5000, 130])):
        b = Batch(BF16, 4, 2, hd, new, ctx, 16, seed=6)
        m = dict(slopes=True)
        b.fill([n + c for n, c in zip(b.new, b.ctx)])
        kw, out = dict(slopes=torch.tensor([slope, 0.0, slope / 7, slope], device="cuda")), b.out()
        slm.attention_paged_scored(b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, out, b.workspace(slm),
                                   b.status, **kw)
        check(b, out, b.seq_k, b.seq_v, m, kw, BF16)


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("dtype,H,KV,hd", [(BF16, 9, 3, 64), (BF16, 32, 8, 128), (F32, 9, 3, 64)])
def test_long(slm, dtype, H, KV, hd, page):  # noqa: F811
    """Windows and documents over contexts that many CTAs share."""
    b = Batch(dtype, H, KV, hd, [1, 1, 40, 700], [9000, 20, 6000, 3000], page, seed=page, pad=1)
    for m in (dict(window=4096, cap=50.0), dict(slopes=True), dict(first=documents(b, 5, 3000), cap=9.0),
              dict(prefix=[0, 7, 6030, 3500], window=5000)):
        out, keys, values, kw = paged(slm, b, m, evict=False)
        check(b, out, keys, values, m, kw, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_plain_masks_agree_with_the_plain_call(slm, dtype):  # noqa: F811
    """Documents as one prompt of many, or as prompts of their own: the same rows."""
    new = [100, 37, 1, 400]
    b = Batch(dtype, 9, 3, 64, new, seed=1)
    apart, together = b.out(), b.out()
    slm.attention_prompt(b.q, b.k, b.v, b.row_start, apart, b.workspace(slm), b.status)
    first = torch.cat([torch.full((n,), a, dtype=torch.int32) for a, n in zip(b.starts, new)]).cuda()
    whole = torch.tensor([0, sum(new)], dtype=torch.int32, device="cuda")
    slm.attention_prompt_scored(b.q, b.k, b.v, whole, together, b.workspace(slm), b.status, first=first)
    tol = 2.0 ** -6 if dtype == BF16 else 2.0 ** -18  # two roundings of weights and results of a few units
    assert float((apart.double() - together.double()).abs().max()) <= tol * 4


def test_refused_mask_is_reported(slm):  # noqa: F811
    """`first` descends: reported, and nothing outside the rows is touched."""
    for dtype, new in ((BF16, [300, 4]), (F32, [300, 4]), (F32, [3, 1])):
        b = Batch(dtype, 9, 3, 64, new, [20, 30], seed=2, pad=4)
        b.fill([n + c for n, c in zip(b.new, b.ctx)])
        first = torch.zeros(b.rows, dtype=torch.int32, device="cuda")
        first[1] = 9
        out = b.out()
        slm.attention_paged_scored(b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, out, b.workspace(slm),
                                   b.status, first=first)
        assert int(b.status.item()) == slm.SLM_ROWS_LENGTH
        assert bool((out[b.starts[-1]:] == 7.0).all())


def test_overlapping_ranges(slm):  # noqa: F811
    """row_start that goes up and down claims more rows than there are: reported, not worked off."""
    for dtype in (BF16, F32):
        b = Batch(dtype, 4, 2, 16, [40] * 6, [0] * 6, seed=2)
        n = b.rows
        starts = torch.tensor([0, n, 0, n, 0, n, 0], dtype=torch.int32, device="cuda")
        out = b.out()
        slm.attention_prompt_scored(b.q, b.k, b.v, starts, out, b.workspace(slm), b.status, window=9)
        assert int(b.status.item()) == slm.SLM_ROWS_LENGTH


@pytest.mark.parametrize("dtype,H,KV,hd", [(BF16, 9, 3, 64), (BF16, 32, 8, 128), (F32, 9, 3, 64)])
def test_captured(slm, dtype, H, KV, hd):  # noqa: F811
    """A captured call on another stream, replayed with other lengths, masks and pages; twice the same bits."""
    b = Batch(dtype, H, KV, hd, [3, 1, 60], [100, 700, 0], 16, seed=8)
    b.fill([n + c for n, c in zip(b.new, b.ctx)])
    m = dict(window=200, cap=20.0, slopes=True, first=documents(b, 9, 50))
    kw, out, ws = arguments(b, m), b.out(), b.workspace(slm)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def call():
        slm.attention_paged_scored(b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, out, ws, b.status, **kw)

    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    g.replay()
    check(b, out, b.seq_k, b.seq_v, m, kw, dtype)
    once = out.clone()
    ws.fill_(0xff)
    g.replay()
    assert bool((once.view(torch.uint8) == out.view(torch.uint8)).all())
    # other lengths and documents in the same buffers: the first sequence brings nothing any more
    c = Batch(dtype, H, KV, hd, [0, 4, 60], [100, 697, 0], 16, seed=8)
    c.q, c.seq_k, c.seq_v, c.status = b.q, b.seq_k, b.seq_v, b.status
    m = dict(m, first=documents(c, 10, 90))
    b.row_start.copy_(c.row_start)
    b.ctx_len.copy_(c.ctx_len)
    kw["first"].copy_(arguments(c, m)["first"])
    out.fill_(7.0)
    g.replay()
    check(c, out, c.seq_k, c.seq_v, m, kw, dtype)


@pytest.mark.parametrize("dtype,hd", [(BF16, 64), (BF16, 128), (F32, 64), (BF16, 192)])
def test_odd_scores(slm, dtype, hd):  # noqa: F811
    """A NaN query makes its row NaN and no other; infinite products meet a cap as +-cap; a huge cap is none."""
    b = Batch(dtype, 4, 2, hd, [130, 1], [0, 200], seed=3)
    b.fill([n + c for n, c in zip(b.new, b.ctx)])
    q = b.q.clone()
    b.q[7, 1] = float("nan")

    def call(**kw):
        out = b.out()
        slm.attention_paged_scored(b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, out, b.workspace(slm),
                                   b.status, **kw)
        return out

    out = call(cap=4.0, window=40)
    assert bool(out[7, 1].isnan().all())
    out[7, 1] = 0
    assert bool(out.isfinite().all())
    b.q = q
    m = dict(cap=1e6)
    out = call(**m)
    check(b, out, b.seq_k, b.seq_v, m, {}, dtype)
    big = (b.q.double() * 1e30).to(dtype)  # products overflow to +-infinity or are +-1e30: weights e^cap or e^-cap
    b.q = big
    out = call(cap=2.0)
    assert bool(out.isfinite().all())


def test_one_workspace_each(slm):  # noqa: F811
    """Two captured calls with workspaces of their own, replayed at once on two streams."""
    b = Batch(BF16, 32, 8, 128, [1] * 8, [5000 + 100 * i for i in range(8)], 64, seed=4)
    b.fill([n + c for n, c in zip(b.new, b.ctx)])
    outs, graphs = [b.out(), b.out()], []
    for out, kw in zip(outs, (dict(cap=30.0), dict(window=1000))):
        ws = b.workspace(slm)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            slm.attention_paged_scored(b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, out, ws, b.status, **kw)
        graphs.append((g, ws, torch.cuda.Stream()))
    for g, _, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    for _ in range(5):
        for g, _, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert bool((w == o).all())
    check(b, outs[0], b.seq_k, b.seq_v, dict(cap=30.0), {}, BF16)


def test_wrong_arguments(slm):  # noqa: F811
    b = Batch(BF16, 4, 2, 64, [5], [0], seed=1)
    out, ws = b.out(), b.workspace(slm)

    def call(**kw):
        slm.attention_prompt_scored(b.q, b.k, b.v, b.row_start, out, ws, b.status, **kw)

    good = torch.zeros(4, device="cuda")
    for kw, why in [(dict(slopes=good[:3]), "slopes"), (dict(slopes=good.double()), "slopes"),
                    (dict(first=torch.zeros(4, dtype=torch.int32, device="cuda")), "first"),
                    (dict(prefix_len=torch.zeros(2, dtype=torch.int32, device="cuda")), "prefix_len"),
                    (dict(first=torch.zeros(5, dtype=torch.int64, device="cuda")), "first")]:
        with pytest.raises(ValueError, match=why):
            call(**kw)
    for kw, why in [(dict(cap=-1.0), "cap"), (dict(cap=math.inf), "cap"), (dict(scale=math.nan), "scale"),
                    (dict(window=-1), "window"), (dict(slopes=torch.zeros(4)), "slopes is not device memory")]:
        with pytest.raises(slm.SlmError, match=why):
            call(**kw)
    assert bool((out == 7.0).all())
