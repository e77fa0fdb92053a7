"""The packed-row operators on the GPU -- slm_kv_append, slm_attention_paged,
slm_attention_prompt -- against their definitions in 64 bits.

Tolerances (u = 2^-24, one fp32 rounding; h = 2^-8, half a step of bf16):
* append: a rotated value is a c - b s: two products and a sum, 2 u (|a c| + |b s|) at most; a
  bf16 result adds its rounding, h |y|.  v, and everything without a rotation, is exact.
* attention: a score is a sum of head_dim exact-in-fp64 products carried in fp32: with up to
  2^-22 lost per addition (the tensor cores align and cut the addends of one step), it is off by
  ds <= 2^-22 (head_dim + 8) max_t sum_d |q_d k_d| / sqrt(head_dim).  A weight is then off by the
  factor 1 +- (ds + 8 u), the output by 2 (ds + 8 u) vmax, and the sums over L positions add
  L 2^-22 vmax at the very most.  bf16 calls round the weights to bf16 (h A, with A the weighted
  mean of |v|) and the result (h |out|).
"""
import ctypes
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U, H16 = 2.0 ** -24, 2.0 ** -8
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def slm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import llama_decode_kv_gb300 as m
    return m


class Batch:
    """A batch of packed rows with everything the three calls take.  Cache slots that hold
    nothing, pages of nobody and rows of nobody are NaN."""

    def __init__(self, dtype, H, KV, hd, new, ctx=None, page=16, cache=None, lead=0, pad=0, seed=0, fused=False,
                 qscale=2.0, spare=3):
        dev = "cuda"
        g = torch.Generator(device=dev).manual_seed(seed + 17)
        self.H, self.KV, self.hd, self.page, self.dtype = H, KV, hd, page, dtype
        self.cache_dtype = cache or dtype
        self.new, self.ctx = list(new), list(ctx if ctx is not None else [0] * len(new))
        S, used = len(self.new), sum(self.new)
        self.rows = lead + used + pad
        starts = [lead]
        for n in self.new:
            starts.append(starts[-1] + n)
        self.starts = starts
        self.row_start = torch.tensor(starts, dtype=torch.int32, device=dev)
        self.ctx_len = torch.tensor(self.ctx, dtype=torch.int32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

        def rnd(*shape):
            return torch.randn(*shape, device=dev, generator=g)

        W = (H + 2 * KV) * hd
        if fused:  # q, k, v are column ranges of one projection's output
            x = rnd(self.rows, W + 16).to(dtype)
            x[:, :H * hd] *= qscale
            parts = x[:, :W].split([H * hd, KV * hd, KV * hd], dim=1)
            self.q, self.k, self.v = (p.unflatten(1, (n, hd)) for p, n in zip(parts, (H, KV, KV)))
        else:
            self.q = (rnd(self.rows, H, hd) * qscale).to(dtype)
            self.k, self.v = rnd(self.rows, KV, hd).to(dtype), rnd(self.rows, KV, hd).to(dtype)
        nobody = list(range(lead)) + list(range(lead + used, self.rows))
        for x in (self.q, self.k, self.v):
            x[nobody] = float("nan")
        need = [(n + c + page - 1) // page for n, c in zip(self.new, self.ctx)]
        pool = sum(need) + spare
        order = torch.randperm(pool, generator=torch.Generator().manual_seed(seed)).tolist()
        tab = [[-1] * max(max(need), 1) for _ in range(S)]
        for s in range(S):
            for i in range(need[s]):
                tab[s][i] = order.pop()
        self.table = tab
        self.page_table = torch.tensor(tab, dtype=torch.int32, device=dev)
        self.k_cache = torch.full((pool, KV, page, hd), float("nan"), device=dev, dtype=self.cache_dtype)
        self.v_cache = self.k_cache.clone()
        # keys and values by sequence, [positions][kv heads][head_dim]
        self.seq_k = [rnd(n + c, KV, hd).to(self.cache_dtype) for n, c in zip(self.new, self.ctx)]
        self.seq_v = [rnd(n + c, KV, hd).to(self.cache_dtype) for n, c in zip(self.new, self.ctx)]

    def fill(self, upto):
        """Put positions [0, upto[s]) of every sequence into the cache."""
        for s, n in enumerate(upto):
            for p0 in range(0, n, self.page):
                m = min(self.page, n - p0)
                pg = self.table[s][p0 // self.page]
                self.k_cache[pg, :, :m] = self.seq_k[s][p0:p0 + m].transpose(0, 1)
                self.v_cache[pg, :, :m] = self.seq_v[s][p0:p0 + m].transpose(0, 1)

    def out(self, dtype=None):
        return torch.full((self.rows, self.H, self.hd), 7.0, device="cuda", dtype=dtype or self.cache_dtype)

    def workspace(self, slm):
        n = slm.attention_rows_workspace_bytes(self.q.dtype, self.rows, len(self.new), self.H, self.KV, self.hd)
        assert n > 0
        return torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")  # NaN everywhere


def attention64(q, k, v, ctx):
    """(out, tolerance terms) of one sequence: q [n][H][hd], k, v [ctx + n][KV][hd]."""
    n, H, hd = q.shape
    G = H // k.shape[1]
    hide = torch.ones(n, k.shape[0], dtype=torch.bool, device=q.device).triu(ctx + 1)
    out = torch.empty(n, H, hd, dtype=torch.float64, device=q.device)
    mean, ds = torch.empty_like(out), torch.empty(n, H, 1, dtype=torch.float64, device=q.device)
    for h in range(H):
        a, kk, vv = q[:, h].double(), k[:, h // G].double(), v[:, h // G].double()
        p = torch.softmax((a @ kk.t() / math.sqrt(hd)).masked_fill(hide, -math.inf), dim=-1)
        out[:, h] = p @ vv
        mean[:, h] = p @ vv.abs()
        ds[:, h] = ((a.abs() @ kk.abs().t()).masked_fill(hide, 0).amax(-1, keepdim=True) / math.sqrt(hd)
                    * (2.0 ** -22 * (hd + 8)))
    return out, mean, ds


def check_attention(b, out, keys, values, dtype):
    err = 0.0
    for s, (n, c) in enumerate(zip(b.new, b.ctx)):
        if n == 0:
            continue
        rows = slice(b.starts[s], b.starts[s] + n)
        want, mean, ds = attention64(b.q[rows], keys[s], values[s], c)
        vmax = float(values[s].double().abs().max())
        tol = 2 * (ds + 8 * U) * vmax + (n + c) * 2.0 ** -22 * vmax
        if dtype == BF16:
            tol = tol + H16 * (mean + want.abs())
        else:
            tol = tol + U * want.abs()
        d = (out[rows].double() - want).abs()
        assert bool((d <= tol).all()), (s, float((d / tol).nan_to_num(nan=9e9).max()))
        err = max(err, float((d / tol).max()))
    nobody = list(range(b.starts[0])) + list(range(b.starts[-1], b.rows))
    assert bool((out[nobody] == 7.0).all()), "rows of nobody were written"
    assert int(b.status.item()) == 0
    return err


# ------------------------------------------------------------------ append

def rope_table(n, hd, theta=10000.0):
    i = torch.arange(hd // 2, dtype=torch.float64, device="cuda")
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * theta ** (-2.0 * i / hd)
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


def check_append(b, kc0, vc0, q_out, rope):
    """The whole cache and q_out against the definition; kc0, vc0: the cache before."""
    kw, vw = kc0.double(), vc0.double()
    ktol = torch.zeros_like(kw)
    half = b.hd // 2
    store = H16 if b.cache_dtype == BF16 else 0.0

    def turn(x, pos):
        x = x.double()
        if rope is None:
            return x, torch.zeros_like(x)
        c, s = (rope[pos].double()[:, None, :, i] for i in (0, 1))
        a, d = x[..., :half], x[..., half:]
        y = torch.cat([a * c - d * s, a * s + d * c], -1)
        t = torch.cat([(a * c).abs() + (d * s).abs(), (a * s).abs() + (d * c).abs()], -1) * 2 * U
        return y, t

    for s, (n, c) in enumerate(zip(b.new, b.ctx)):
        if n == 0:
            continue
        rows, pos = slice(b.starts[s], b.starts[s] + n), torch.arange(c, c + n, device="cuda")
        y, t = turn(b.k[rows], pos)
        pg = torch.tensor(b.table[s], device="cuda")[pos // b.page]
        kw[pg, :, pos % b.page] = y
        ktol[pg, :, pos % b.page] = t + store * y.abs()
        vw[pg, :, pos % b.page] = b.v[rows].to(b.cache_dtype).double()
        if q_out is not None:
            y, t = turn(b.q[rows], pos)
            assert bool(((q_out[rows].double() - y).abs() <= t + store * y.abs()).all()), s
    assert bool((torch.isnan(kw) == torch.isnan(b.k_cache)).all()), "a slot of nobody was written, or one was missed"
    assert bool(((b.k_cache.double() - kw).abs().nan_to_num(0.0) <= ktol.nan_to_num(0.0)).all())
    assert torch.equal(b.v_cache.double().nan_to_num(9e9), vw.nan_to_num(9e9))
    if q_out is not None:
        nobody = list(range(b.starts[0])) + list(range(b.starts[-1], b.rows))
        assert bool((q_out[nobody] == 7.0).all())
    assert int(b.status.item()) == 0


@pytest.mark.parametrize("dtype,cache", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("H,KV,hd,page,new,ctx,lead,pad", [
    (4, 2, 16, 16, [1], [0], 0, 0),
    (9, 3, 64, 16, [1], [261], 0, 0),
    (4, 2, 24, 16, [17, 0, 1, 40], [15, 9, 0, 100], 2, 3),       # 8 mod 16 heads, an idle sequence
    (2, 1, 8, 32, [3, 3], [31, 32], 0, 1),
    (8, 1, 256, 64, [5, 66], [63, 130], 1, 0),
    (6, 6, 128, 128, [0, 0, 130, 0], [0, 5, 127, 0], 0, 0),
])
def test_append(slm, dtype, cache, H, KV, hd, page, new, ctx, lead, pad):
    b = Batch(dtype, H, KV, hd, new, ctx, page, cache, lead, pad, seed=hd + len(new))
    b.fill(b.ctx)
    rope = rope_table(max(n + c for n, c in zip(new, ctx)), hd)
    kc, vc, q_out = b.k_cache.clone(), b.v_cache.clone(), b.out()
    slm.kv_append(b.k, b.v, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, b.status, rope, b.q, q_out)
    check_append(b, kc, vc, q_out, rope)


def test_append_many_rows_fused_projection(slm):
    b = Batch(F32, 9, 3, 64, [700, 1, 0, 900, 1300], [5, 0, 3, 64, 1], 64, BF16, 1, 9, seed=3, fused=True)
    rope = rope_table(1500, 64)
    b.fill(b.ctx)
    kc, vc, q_out = b.k_cache.clone(), b.v_cache.clone(), b.out()
    slm.kv_append(b.k, b.v, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, b.status, rope, b.q, q_out)
    check_append(b, kc, vc, q_out, rope)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_append_without_rotation_without_queries_and_in_place(slm, dtype):
    b = Batch(dtype, 4, 2, 48, [3, 20], [14, 0], 16, seed=1)
    kc, vc = b.k_cache.clone(), b.v_cache.clone()
    slm.kv_append(b.k, b.v, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, b.status)
    check_append(b, kc, vc, None, None)
    rope = rope_table(20, 48)
    q0 = b.q.clone()
    slm.kv_append(b.k, b.v, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, b.status, rope, b.q, b.q)
    got, b.q = b.q, q0
    check_append(b, kc, vc, got, rope)
    # ctx_len None: positions from 0
    b = Batch(dtype, 4, 2, 48, [3, 20], None, 16, seed=2)
    kc, vc = b.k_cache.clone(), b.v_cache.clone()
    slm.kv_append(b.k, b.v, b.k_cache, b.v_cache, b.page_table, b.row_start, None, b.status, rope)
    check_append(b, kc, vc, None, rope)


def test_append_skips_rows_with_bad_pages_and_positions(slm):
    """Bad page ids and positions outside the tables: those rows are not written, the others
    are, and the status says which kind it was."""
    b = Batch(F32, 2, 1, 16, [4, 4], [14, 0], 16, seed=4)
    rope = rope_table(18, 16)
    for bad, bit in ((1000, slm.SLM_ROWS_PAGE), (-1, slm.SLM_ROWS_PAGE)):
        b.page_table[0, 1] = bad  # positions 16, 17 of sequence 0
        b.status.zero_()
        b.k_cache.fill_(float("nan"))
        slm.kv_append(b.k, b.v, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, b.status, rope)
        assert int(b.status.item()) == bit
        assert int((~torch.isnan(b.k_cache[..., 0])).sum()) == 6
    b.page_table[0, 1] = b.table[0][1]
    for ctx0 in (29, -1, 2 ** 31 - 2):  # past the table, negative, past int32
        b.status.zero_()
        b.k_cache.fill_(float("nan"))
        ctx = torch.tensor([ctx0, 0], dtype=torch.int32, device="cuda")
        slm.kv_append(b.k, b.v, b.k_cache, b.v_cache, b.page_table, b.row_start, ctx, b.status)
        assert int(b.status.item()) == slm.SLM_ROWS_LENGTH
        assert int((~torch.isnan(b.k_cache[..., 0])).sum()) == 4 + (3 if ctx0 == 29 else 0)
    for starts in ((0, 10, 5), (0, 4, 9), (-3, 4, 8)):  # descends; past the buffer; before it
        b.status.zero_()
        b.k_cache.fill_(float("nan"))
        rs = torch.tensor(starts, dtype=torch.int32, device="cuda")
        slm.kv_append(b.k, b.v, b.k_cache, b.v_cache, b.page_table, rs, None, b.status)
        assert int(b.status.item()) == slm.SLM_ROWS_LENGTH
    b.status.zero_()  # past the rotation table
    slm.kv_append(b.k, b.v, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, b.status, rope[:17])
    assert int(b.status.item()) == slm.SLM_ROWS_LENGTH


# ------------------------------------------------------------------ attention over the paged cache

PAGED = [  # H, KV, hd, page, new, ctx, lead, pad
    (4, 2, 16, 16, [1], [0], 0, 0),                                   # one key
    (9, 3, 64, 16, [1], [261], 0, 0),
    (9, 3, 64, 16, [1, 1, 0, 1], [63, 64, 500, 127], 1, 2),           # block edges, an idle slot
    (8, 2, 64, 64, [1] * 20, [int(3.7 * i * i) for i in range(20)], 0, 0),
    (8, 1, 128, 256, [1, 1], [5000, 3], 0, 0),
    (32, 8, 64, 128, [130, 1, 7], [257, 1000, 0], 0, 5),              # chunks and tokens mixed
    (12, 4, 80, 32, [45, 3], [90, 31], 0, 0),
    (10, 2, 96, 16, [33, 64, 1], [0, 64, 255], 3, 0),
    (15, 5, 72, 64, [128, 129], [128, 127], 0, 0),
    (6, 6, 128, 16, [65], [63], 0, 0),
    (2, 1, 8, 16, [3, 70], [2, 0], 0, 0),
    (64, 1, 64, 64, [9, 1], [100, 700], 0, 0),                        # the largest group
    (17, 1, 64, 16, [20], [77], 0, 0),
    (4, 2, 256, 32, [20, 1], [40, 300], 0, 0),
    (32, 1, 136, 16, [3, 1], [70, 10], 0, 0),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H,KV,hd,page,new,ctx,lead,pad", PAGED)
def test_attention_paged(slm, dtype, H, KV, hd, page, new, ctx, lead, pad):
    b = Batch(dtype, H, KV, hd, new, ctx, page, None, lead, pad, seed=hd + page + len(new))
    b.fill([n + c for n, c in zip(b.new, b.ctx)])
    out, ws = b.out(), b.workspace(slm)
    args = (b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len)
    slm.attention_paged(*args, out, ws, b.status)
    check_attention(b, out, b.seq_k, b.seq_v, dtype)
    again = b.out()  # the same bits, whatever the workspace held
    slm.attention_paged(*args, again, ws, b.status)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attention_paged_sharp_scores(slm, dtype):
    """Scores in the hundreds, the largest at the first, a middle or the last position: the
    running maximum moves by a lot or never."""
    for seed in range(4):
        b = Batch(dtype, 4, 2, 64, [3, 1, 140], [300, 777, 20], 16, seed=seed, qscale=60.0)
        b.fill([n + c for n, c in zip(b.new, b.ctx)])
        out = b.out()
        slm.attention_paged(b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, out, b.workspace(slm), b.status)
        check_attention(b, out, b.seq_k, b.seq_v, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attention_paged_offsets_beyond_32_bits(slm, dtype):
    """A pool of more than 2^32 bytes and more than 2^31 elements; the sequence's pages are its
    first and its last."""
    KV, page, hd = 2, 64, 64
    pool = (1 << 31) // (KV * page * hd) + 40
    free = torch.cuda.mem_get_info()[0]
    if free < 3 * pool * KV * page * hd * (4 if dtype == F32 else 2):
        pytest.skip("not enough device memory")
    b = Batch(dtype, 4, KV, hd, [2], [188], page, seed=9)
    kc = torch.empty(pool, KV, page, hd, dtype=dtype, device="cuda")
    vc = torch.empty_like(kc)
    ids = [pool - 1, 0, pool - 2]
    b.k_cache, b.v_cache, b.table = kc, vc, [ids]
    b.page_table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    b.fill([190])
    out = b.out()
    slm.attention_paged(b.q, kc, vc, b.page_table, b.row_start, b.ctx_len, out, b.workspace(slm), b.status)
    check_attention(b, out, b.seq_k, b.seq_v, dtype)
    slm.kv_append(b.k, b.v, kc, vc, b.page_table, b.row_start, b.ctx_len, b.status)
    assert torch.equal(kc[pool - 2, :, 60:62], b.k.transpose(0, 1)) and torch.equal(vc[pool - 2, :, 60:62], b.v.transpose(0, 1))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attention_paged_reports_bad_pages_and_lengths(slm, dtype):
    """A bad page or length is reported, harms no other sequence and reads nothing outside."""
    b = Batch(dtype, 4, 2, 32, [5, 3], [30, 40], 16, seed=5)
    b.fill([35, 43])
    b.k_cache[torch.isnan(b.k_cache)] = 0
    b.v_cache[torch.isnan(b.v_cache)] = 0
    ws = b.workspace(slm)
    rows1 = slice(b.starts[1], b.starts[2])
    want = b.out()
    slm.attention_paged(b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, want, ws, b.status)
    assert int(b.status.item()) == 0

    def go(bit, row_start=None, ctx=None, table=None):
        out = b.out()
        b.status.zero_()
        slm.attention_paged(b.q, b.k_cache, b.v_cache, table if table is not None else b.page_table,
                            row_start if row_start is not None else b.row_start, ctx if ctx is not None else b.ctx_len,
                            out, ws, b.status)
        torch.cuda.synchronize()
        assert int(b.status.item()) == bit
        return out

    for bad in (-1, 1 << 30, b.k_cache.shape[0]):
        t = b.page_table.clone()
        t[0, 1] = bad
        got = go(slm.SLM_ROWS_PAGE, table=t)
        d = (got[rows1].double() - want[rows1].double()).abs().max()
        assert float(d) <= (H16 * 8 if dtype == BF16 else 1e-5)  # the split may change with nothing else
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for ctx0 in (-3, 44, 2 ** 31 - 1):
        got = go(slm.SLM_ROWS_LENGTH, ctx=ints(ctx0, 40))
        d = (got[rows1].double() - want[rows1].double()).abs().max()
        assert float(d) <= (H16 * 8 if dtype == BF16 else 1e-5)
    go(slm.SLM_ROWS_LENGTH, row_start=ints(0, 5, 9))
    go(slm.SLM_ROWS_LENGTH, row_start=ints(-2 ** 31, 5, 2 ** 31 - 1))
    go(slm.SLM_ROWS_LENGTH, row_start=ints(6, 2, 8))


def test_attention_refuses_host_memory_and_small_workspaces(slm):
    b = Batch(F32, 4, 2, 32, [5], [30], 16, seed=5)
    b.fill([35])
    out, ws = b.out(), b.workspace(slm)
    args = [b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len]
    for bad in (ws[:-1], ws[1:]):
        with pytest.raises(slm.SlmError, match="workspace"):
            slm.attention_paged(*args, out, bad, b.status)
    for i in range(6):
        host = [a.cpu() if j == i else a for j, a in enumerate(args)]
        with pytest.raises(slm.SlmError, match="not device memory"):
            slm.attention_paged(*host, out, ws, b.status)
    with pytest.raises(slm.SlmError, match="not device memory"):
        slm.kv_append(b.k, b.v, b.k_cache, b.v_cache.cpu(), b.page_table, b.row_start, b.ctx_len, b.status)
    with pytest.raises(slm.SlmError, match="not device memory"):
        slm.attention_prompt(b.q, b.k, b.v.cpu(), b.row_start, out, ws, b.status)
    torch.cuda.synchronize()
    assert bool((out == 7.0).all())


# ------------------------------------------------------------------ prompts

PROMPTS = [  # H, KV, hd, lens, lead, pad
    (4, 2, 16, [1], 0, 0),
    (9, 3, 64, [1, 2, 63, 64, 65, 0, 128, 129], 2, 3),
    (16, 4, 64, [300, 127], 0, 0),
    (8, 2, 128, [513, 255, 1], 0, 7),
    (4, 4, 128, [400], 0, 0),
    (12, 4, 80, [200, 17], 1, 1),
    (10, 2, 96, [150], 0, 0),
    (15, 5, 72, [90, 260], 0, 0),
    (2, 1, 8, [130], 0, 0),
    (64, 1, 64, [37, 5], 0, 0),
    (4, 2, 256, [70, 33], 0, 0),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("H,KV,hd,lens,lead,pad", PROMPTS)
def test_attention_prompt(slm, dtype, fused, H, KV, hd, lens, lead, pad):
    b = Batch(dtype, H, KV, hd, lens, None, 16, None, lead, pad, seed=hd + sum(lens), fused=fused)
    out = b.out()
    slm.attention_prompt(b.q, b.k, b.v, b.row_start, out, b.workspace(slm), b.status)
    parts = [slice(b.starts[s], b.starts[s] + n) for s, n in enumerate(b.new)]
    check_attention(b, out, [b.k[p] for p in parts], [b.v[p] for p in parts], dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attention_prompt_sequences_are_apart(slm, dtype):
    """A sequence of infinities and NaN leaves its neighbours as they are."""
    b = Batch(dtype, 6, 2, 64, [100, 70, 140], None, 16, seed=11)
    ws = b.workspace(slm)
    want, got = b.out(), b.out()
    slm.attention_prompt(b.q, b.k, b.v, b.row_start, want, ws, b.status)
    mid = slice(100, 170)
    b.k[mid], b.v[mid], b.q[mid] = float("inf"), float("nan"), float("-inf")
    slm.attention_prompt(b.q, b.k, b.v, b.row_start, got, ws, b.status)
    assert torch.equal(got[:100], want[:100]) and torch.equal(got[170:], want[170:])
    assert bool(torch.isnan(got[mid]).all())


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prompt_then_chunks_then_tokens(slm, dtype):
    """The three calls as a serving loop makes them: a prompt appended and attended whole, a
    chunk of new tokens on top, then single tokens; every output against the definition over
    the rotated keys that were appended."""
    H, KV, hd, page = 6, 2, 64, 16
    steps = [[130, 40, 1], [50, 3, 70], [1, 1, 1], [1, 0, 1]]
    total = [sum(s[i] for s in steps) for i in range(3)]
    rope = rope_table(max(total), hd)
    base = Batch(dtype, H, KV, hd, total, None, page, seed=21)
    have, keys, vals = [0, 0, 0], [None] * 3, [None] * 3
    for i, new in enumerate(steps):
        b = Batch(dtype, H, KV, hd, new, have, page, seed=30 + i)
        b.k_cache, b.v_cache, b.page_table = base.k_cache, base.v_cache, base.page_table
        qr = torch.empty_like(b.q)
        slm.kv_append(b.k, b.v, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, b.status, rope, b.q, qr)
        for s, n in enumerate(new):  # what the cache has to hold now
            pos = torch.arange(have[s], have[s] + n, device="cuda")
            pg = base.page_table[s].long()[pos // page]
            k_new, v_new = base.k_cache[pg, :, pos % page], base.v_cache[pg, :, pos % page]
            assert torch.equal(v_new, b.v[b.starts[s]:b.starts[s] + n])
            keys[s] = k_new if keys[s] is None else torch.cat([keys[s], k_new])
            vals[s] = v_new if vals[s] is None else torch.cat([vals[s], v_new])
        b.q = qr
        out, ws = b.out(), b.workspace(slm)
        slm.attention_paged(qr, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, out, ws, b.status)
        check_attention(b, out, keys, vals, dtype)
        if i == 0:  # the same rows without the cache
            kr = torch.cat(keys)
            alone = b.out()
            slm.attention_prompt(qr, kr, b.v, b.row_start, alone, ws, b.status)
            check_attention(b, alone, keys, vals, dtype)
        have = [h + n for h, n in zip(have, new)]


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_captured_step_replays_with_new_lengths(slm, dtype):
    """Append and attention captured once as a decode step, replayed while the contexts grow,
    against eager calls."""
    S, H, KV, hd, page = 5, 8, 2, 64, 16
    b = Batch(dtype, H, KV, hd, [1] * S, [60, 3, 290, 15, 127], page, seed=40, spare=0)
    tail = torch.arange(S, dtype=torch.int32, device="cuda")[:, None] + b.k_cache.shape[0]
    pool = torch.zeros(b.k_cache.shape[0] + S, KV, page, hd, dtype=dtype, device="cuda")
    b.fill(b.ctx)
    kc, vc = pool.clone(), pool.clone()
    kc[:-S], vc[:-S] = b.k_cache.nan_to_num(0.0), b.v_cache.nan_to_num(0.0)
    table = torch.where(b.page_table < 0, tail, b.page_table).contiguous()
    rope = rope_table(400, hd)
    qr, out, ws = torch.empty_like(b.q), b.out(), b.workspace(slm)

    def step(kc, vc, out):
        slm.kv_append(b.k, b.v, kc, vc, table, b.row_start, b.ctx_len, b.status, rope, b.q, qr)
        slm.attention_paged(qr, kc, vc, table, b.row_start, b.ctx_len, out, ws, b.status)

    ke, ve = kc.clone(), vc.clone()
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step(kc, vc, out)
    torch.cuda.current_stream().wait_stream(warm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(kc, vc, out)
    kc.copy_(ke)
    vc.copy_(ve)
    g = torch.Generator(device="cuda").manual_seed(1)
    for i in range(4):
        for x in (b.q, b.k, b.v):
            x.copy_(torch.randn(x.shape, device="cuda", generator=g).to(dtype))
        graph.replay()
        got = out.clone()
        eager = b.out()
        step(ke, ve, eager)
        assert torch.equal(got, eager) and torch.equal(kc, ke) and torch.equal(vc, ve)
        b.ctx_len += torch.tensor([1, 1, 2 if i == 0 else 1, 1, 0], dtype=torch.int32, device="cuda")
        if i == 0:
            for c in (kc, vc, ke, ve):
                c[table[2, 291 // page], :, 291 % page] = 0.5
    assert int(b.status.item()) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_two_streams_at_once(slm, dtype):
    """Calls on two streams, a workspace each, give what they give alone."""
    bs = [Batch(dtype, 8, 2, 64, [90, 1, 33], [200, 900, 10 * i], 16, seed=50 + i) for i in range(2)]
    for b in bs:
        b.fill([n + c for n, c in zip(b.new, b.ctx)])
    alone, outs, wss = [], [], [b.workspace(slm) for b in bs]
    run = lambda b, o, w: slm.attention_paged(b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, o, w, b.status)  # noqa: E731
    for b, w in zip(bs, wss):
        alone.append(b.out())
        run(b, alone[-1], w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in bs]
    for _ in range(5):
        outs = [b.out() for b in bs]
        torch.cuda.synchronize()
        for b, o, w, st in zip(bs, outs, wss, streams):
            with torch.cuda.stream(st):
                run(b, o, w)
        torch.cuda.synchronize()
        for o, a in zip(outs, alone):
            assert torch.equal(o, a)


@pytest.mark.parametrize("dtype,H,KV,hd", [(BF16, 6, 2, 64), (BF16, 8, 2, 128), (BF16, 4, 4, 64), (F32, 6, 2, 64)])
def test_ragged_batch(slm, dtype, H, KV, hd):
    """Decode steps, chunks of one and of several tiles and idle slots, of all lengths, in one
    call: items of every kind follow one another in a CTA."""
    S = 41
    new = [(1, 1, 70, 0, 1, 13, 150, 33)[i % 8] for i in range(S)]
    ctx = [(i * 211) % 1500 for i in range(S)]
    b = Batch(dtype, H, KV, hd, new, ctx, 32, None, 1, 2, seed=70 + hd)
    b.fill([n + c for n, c in zip(b.new, b.ctx)])
    out, ws = b.out(), b.workspace(slm)
    slm.attention_paged(b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, out, ws, b.status)
    check_attention(b, out, b.seq_k, b.seq_v, dtype)
    again = b.out()
    slm.attention_paged(b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, again, ws, b.status)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("hd,gap", [(64, 8), (64, 16), (80, 8), (16, 16)])
def test_outputs_into_a_wider_buffer(slm, dtype, hd, gap):
    """Outputs as a column range of a wider buffer (row strides of 16 mod 32 bytes among them):
    the columns beside it stay as they were."""
    b = Batch(dtype, 6, 2, hd, [150, 1, 40], None, 16, None, 0, 3, seed=hd + gap)
    wide = torch.full((b.rows, 6 * hd + gap), 7.0, dtype=dtype, device="cuda")
    out = wide[:, gap:].unflatten(1, (6, hd))
    slm.attention_prompt(b.q, b.k, b.v, b.row_start, out, b.workspace(slm), b.status)
    parts = [slice(b.starts[s], b.starts[s] + n) for s, n in enumerate(b.new)]
    check_attention(b, out, [b.k[p] for p in parts], [b.v[p] for p in parts], dtype)
    assert bool((wide[:, :gap] == 7.0).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_one_long_context_over_the_whole_gpu(slm, dtype):
    """One kv head, one token, a context that every CTA gets a piece of: the join of many pieces."""
    b = Batch(dtype, 5, 1, 64, [1], [40001], 64, seed=80)
    b.fill([40002])
    out = b.out()
    slm.attention_paged(b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, out, b.workspace(slm), b.status)
    check_attention(b, out, b.seq_k, b.seq_v, dtype)


def test_no_rows(slm):
    b = Batch(BF16, 4, 2, 64, [0, 0], [5, 0], 16, seed=1, pad=2)
    b.fill([5, 0])
    out, ws = b.out(), b.workspace(slm)
    slm.attention_paged(b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, out, ws, b.status)
    slm.attention_prompt(b.q, b.k, b.v, b.row_start, out, ws, b.status)
    assert bool((out == 7.0).all())
    assert int(b.status.item()) == 0


def test_many_sequences(slm):
    """1,024 sequences of one token each, the most a call takes."""
    b = Batch(BF16, 4, 2, 64, [1] * 1024, [(i * 37) % 200 for i in range(1024)], 16, seed=60)
    b.fill([n + c for n, c in zip(b.new, b.ctx)])
    out = b.out()
    slm.attention_paged(b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, out, b.workspace(slm), b.status)
    check_attention(b, out, b.seq_k, b.seq_v, BF16)
    assert ctypes.sizeof(slm.slm_kv_cache) == 48
