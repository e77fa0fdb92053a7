"""The calls of a serving step around the packed-row attention on the GPU -- slm_rows_plan,
slm_kv_append_axes, slm_sample_rows -- against their definitions in plain Python, and a step of all of
them together.

Tolerances: the plan and the tokens are whole numbers and have to be equal (the tests' uniforms stay
2^-18 away from every border of the draw, the kernel's weights are within 2^-20); a rotated value is off by
2 u (|a c| + |b s|), a bf16 result by h |y| besides, as in test_gpu_rows; what is not turned is exact."""
import math
import random

import numpy as np
import pytest

from test_gpu_rows import BF16, F32, H16, U, Batch, rope_table, slm  # noqa: F401  (slm: the fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


# ------------------------------------------------------------------ plan

class Pool:
    """A page pool, its expected state in Python lists."""

    def __init__(self, lens, page, ld, n_pages, seed=0):
        r = random.Random(seed)
        ids = r.sample(range(n_pages), n_pages)
        self.page, self.ld, self.n_pages, self.len = page, ld, n_pages, list(lens)
        self.table = [[-1] * ld for _ in lens]
        for s, c in enumerate(lens):
            for b in range(-(-c // page)):
                self.table[s][b] = ids.pop()
        self.free = ids
        S = len(lens)
        self.seq_len, self.free_count = ints(self.len), ints([len(ids)])
        self.page_table = ints(self.table)
        self.free_pages = ints(ids + [-7] * (n_pages - len(ids)))
        self.row_start, self.ctx_len, self.status = ints([9] * (S + 1)), ints([9] * S), ints([0])

    def call(self, slm, new, rows, in_place=False):
        S = len(new)
        self.positions, self.slots = ints([9] * rows), ints([9] * rows, torch.int64)
        self.seq_out = self.seq_len if in_place else ints([9] * S)
        self.free_out = self.free_count if in_place else ints([9])
        self.new = ints(new)
        slm.rows_plan(self.new, self.seq_len, self.page_table, self.page, self.free_pages, self.free_count, self.row_start,
                      self.ctx_len, self.positions, self.slots, self.seq_out, self.free_out, self.status)

    def expect(self, new):
        """Move the lists on by one step; (row_start, ctx_len, positions, slots)."""
        P = self.page
        for s, n in enumerate(new):
            if n < 0:
                self.free += self.table[s][:-(-self.len[s] // P)]
                self.len[s] = 0
        start, pos, slots, ctx = [0], [], [], list(self.len)
        for s, n in enumerate(new):
            for _ in range(max(n, 0)):
                p = self.len[s]
                if p % P == 0:
                    self.table[s][p // P] = self.free.pop()
                pos.append(p)
                slots.append(self.table[s][p // P] * P + p % P)
                self.len[s] += 1
            start.append(len(pos))
        return start, ctx, pos, slots

    def check(self, new, rows):
        start, ctx, pos, slots = self.expect(new)
        assert self.row_start.tolist() == start and self.ctx_len.tolist() == ctx
        assert self.positions.tolist() == pos + [-1] * (rows - len(pos))
        assert self.slots.tolist() == slots + [-1] * (rows - len(pos))
        assert self.page_table.tolist() == self.table
        assert self.seq_out.tolist() == self.len and self.free_out.tolist() == [len(self.free)]
        assert self.free_pages[:len(self.free)].tolist() == self.free
        assert int(self.status.item()) == 0


@pytest.mark.parametrize("page", [16, 64, 1 << 20])
@pytest.mark.parametrize("lens,new", [
    ([0], [0]), ([0], [1]), ([15], [1]), ([16], [1]), ([40], [-1]), ([0], [-3]), ([0], [5000]),
    ([5, 0, 31, 16, 7, 0], [1, 0, 1, 17, -1, 40]), ([33, 64, 0, 100], [-1, -1, 200, 0]), ([0, 0, 0], [0, 0, 0]),
    ([i * 7 % 90 for i in range(1024)], [(i * 13) % 11 - 1 for i in range(1024)]),
    ([100] * 300, [64] * 300), ([i % 50 for i in range(33)], [-1] * 33)])
def test_plan(slm, page, lens, new):  # noqa: F811
    ld = max(-(-(c + max(n, 0)) // page) for c, n in zip(lens, new)) + 2
    need = sum(-(-(c + max(n, 0)) // page) for c, n in zip(lens, new))
    rows = sum(max(n, 0) for n in new) + 3
    p = Pool(lens, page, ld, max(need, 1) + 4, seed=page)
    p.call(slm, new, rows)
    p.check(new, rows)


def test_plan_uses_the_pages_given_back(slm):  # noqa: F811
    """The stack is empty: the new rows get the ended sequences' pages, the last one first."""
    p = Pool([64, 32, 0], 16, 6, 6)
    p.call(slm, [-1, -1, 90], 90)
    p.check([-1, -1, 90], 90)
    assert p.free == []


def test_plan_in_place_steps(slm):  # noqa: F811
    """A captured step that goes on from replay to replay."""
    p = Pool([10, 0, 100, 31], 16, 40, 100, seed=3)
    new = [1, 3, 1, 2]
    p.call(slm, new, 9, in_place=True)
    p.check(new, 9)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        slm.rows_plan(p.new, p.seq_len, p.page_table, 16, p.free_pages, p.free_count, p.row_start, p.ctx_len, p.positions,
                      p.slots, p.seq_len, p.free_count, p.status)
    for step in range(20):
        new = [1, 3, -1 if step == 11 else 1, 0 if step % 2 else 2]
        p.new.copy_(ints(new))
        g.replay()
        p.check(new, 9)


@pytest.mark.parametrize("rows", [40, 9000])
@pytest.mark.parametrize("lens,new,kw,bit", [
    ([10, 20], [20, 30], dict(n_pages=4), "POOL"),          # four pages: three held, three needed
    ([10, 20], [-1, 100], dict(n_pages=5), "POOL"),
    ([10, 20], [30, 11], dict(ld=2), "LENGTH"),             # a third entry
    ([10, 20], [20, 10000], dict(ld=900, n_pages=900), "LENGTH"),  # more rows than `rows`
    ([10, 20], [1 << 30, (1 << 31) - 1], {}, "LENGTH")])
def test_plan_that_does_not_fit(slm, lens, new, kw, bit, rows):  # noqa: F811
    p = Pool(lens, 16, kw.get("ld", 100), kw.get("n_pages", 200))
    before = [x.clone() for x in (p.page_table, p.free_pages)]
    p.call(slm, new, rows)
    assert int(p.status.item()) & getattr(slm, "SLM_ROWS_" + bit)
    assert p.row_start.tolist() == [0] * 3 and p.ctx_len.tolist() == lens and p.seq_out.tolist() == lens
    assert p.free_out.tolist() == p.free_count.tolist()
    assert bool((p.positions == -1).all()) and bool((p.slots == -1).all())
    assert all(bool((a == b).all()) for a, b in zip(before, (p.page_table, p.free_pages)))


@pytest.mark.parametrize("field,value,bit", [("seq_len", -1, "LENGTH"), ("seq_len", (1 << 31) - 1, "LENGTH"),
                                             ("free_count", -1, "POOL"), ("free_count", 201, "POOL"),
                                             ("free_count", 199, "POOL")])
def test_plan_with_bad_state(slm, field, value, bit):  # noqa: F811
    p = Pool([10, 40], 16, 100, 200)
    getattr(p, field)[0] = value
    p.call(slm, [3, -1], 8)  # three pages come back
    assert int(p.status.item()) == getattr(slm, "SLM_ROWS_" + bit)
    assert p.row_start.tolist() == [0, 0, 0] and bool((p.slots == -1).all())


def test_plan_with_bad_pages(slm):  # noqa: F811
    p = Pool([10, 40], 16, 100, 200)
    p.page_table[0, 0] = 200
    p.free_pages[p.free_count.item() - 1] = -5
    p.call(slm, [3, 9], 12)
    assert int(p.status.item()) == slm.SLM_ROWS_PAGE
    assert p.slots[:3].tolist() == [-1] * 3 and p.page_table[1, 3].item() == -5
    assert p.slots[3:11].tolist() == [p.table[1][2] * 16 + i for i in range(8, 16)] and p.slots[11].item() == -1


# ------------------------------------------------------------------ append

def turned(x, rope, positions, axis):
    """(y, tolerance without the type's rounding) of x [n][heads][hd], in 64 bits."""
    half = x.shape[-1] // 2
    y, tol = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    for j, a in enumerate(axis):
        if a < 0:
            continue
        cs = rope[positions[a].long(), j].double()
        c, s = cs[:, None, 0], cs[:, None, 1]
        u, v = x[..., j].double(), x[..., j + half].double()
        y[..., j], y[..., j + half] = u * c - v * s, u * s + v * c
        tol[..., j] = 2 * U * ((u * c).abs() + (v * s).abs())
        tol[..., j + half] = 2 * U * ((u * s).abs() + (v * c).abs())
    return y, tol


@pytest.mark.parametrize("pattern", ["sections", "turns", "part", "one", "none"])
@pytest.mark.parametrize("dtype,cache,H,KV,hd", [(BF16, BF16, 9, 3, 64), (F32, BF16, 32, 8, 128), (BF16, F32, 4, 2, 24),
                                                 (F32, F32, 8, 1, 256), (BF16, BF16, 2, 2, 8)])
def test_append_axes(slm, dtype, cache, H, KV, hd, pattern):  # noqa: F811
    new, ctx = [5, 1, 0, 70, 33], [0, 300, 4, 16, 1000]
    b = Batch(dtype, H, KV, hd, new, ctx, 16, cache, lead=2, pad=3, seed=hd, fused=True)
    half, n = hd // 2, {"one": 1, "none": 8}.get(pattern, 3)
    axis = {"sections": [min(2, 3 * j // half) for j in range(half)], "turns": [j % 3 for j in range(half)],
            "part": [j % 3 if j < half // 2 else -1 for j in range(half)], "one": [0] * half, "none": [-1] * half}[pattern]
    rope = rope_table(200, hd)
    g = torch.Generator().manual_seed(5)
    positions = torch.randint(0, 200, (n, b.rows + 6), generator=g, dtype=torch.int32).cuda()
    positions[:, :2] = -9  # rows of nobody
    positions[:, 2 + sum(new):] = 1 << 30
    q_out = b.out()
    k0, v0 = b.k_cache.clone(), b.v_cache.clone()
    slm.kv_append_axes(b.k, b.v, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, b.status, rope, axis,
                       positions[:, :b.rows], q=b.q, q_out=q_out)
    assert int(b.status.item()) == 0
    rnd = H16 if cache == BF16 else U
    for s, (m, c) in enumerate(zip(new, ctx)):
        rows = slice(b.starts[s], b.starts[s] + m)
        pos = positions[:, rows]
        for x, got in ((b.q, q_out[rows]), (b.k, None)):
            y, tol = turned(x[rows], rope, pos, axis)
            if got is None:
                p = torch.arange(c, c + m, device="cuda")
                pages = b.page_table[s].long()[p // 16]
                got = b.k_cache[pages, :, p % 16]
                assert bool((b.v_cache[pages, :, p % 16] == b.v[rows].to(cache)).all())
                k0[pages, :, p % 16] = got
                v0[pages, :, p % 16] = b.v_cache[pages, :, p % 16]
            still = [j for j, a in enumerate(axis) if a < 0]
            still += [j + half for j in still]
            assert bool((got[..., still] == x[rows][..., still].to(cache)).all())
            assert bool(((got.double() - y).abs() <= tol + rnd * y.abs()).all())
    for a, w in ((b.k_cache, k0), (b.v_cache, v0)):  # and nothing else
        assert bool(((a == w) | (a.isnan() & w.isnan())).all())
    assert bool((q_out[:2] == 7).all()) and bool((q_out[b.starts[-1]:] == 7).all())


def test_append_axes_agrees_with_one_axis(slm):  # noqa: F811
    b = Batch(BF16, 9, 3, 64, [40, 1], [7, 90], 16, seed=1)
    rope = rope_table(100, 64)
    p = torch.cat([torch.arange(7, 47), torch.tensor([90])]).int().cuda()
    one, two = b.out(), b.out()
    k, v = b.k_cache.clone(), b.v_cache.clone()
    slm.kv_append(b.k, b.v, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, b.status, rope, b.q, one)
    slm.kv_append_axes(b.k, b.v, k, v, b.page_table, b.row_start, b.ctx_len, b.status, rope, [0, 1] * 16,
                       torch.stack([p, p]), q=b.q, q_out=two)
    for x, y in ((one, two), (k, b.k_cache), (v, b.v_cache)):
        assert bool((x.nan_to_num(nan=3.0) == y.nan_to_num(nan=3.0)).all())


def test_append_axes_positions_outside(slm):  # noqa: F811
    """A row with a position outside the table is reported and left out; its neighbours are written."""
    for bad in (-1, 50, 1 << 30):
        b = Batch(F32, 4, 2, 16, [12], [3], 16, seed=1)
        positions = torch.zeros(2, 12, dtype=torch.int32, device="cuda")
        positions[1, 5] = bad
        out = b.out()
        slm.kv_append_axes(b.k, b.v, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, b.status,
                           rope_table(50, 16), [0] * 8, positions, q=b.q, q_out=out)
        assert int(b.status.item()) == slm.SLM_ROWS_LENGTH
        assert bool((out[5] == 7).all()) and bool(b.k_cache[b.table[0][0], :, 8].isnan().all())
        assert bool((out[:5] != 7).any(-1).all()) and not bool(b.k_cache[b.table[0][0], :, [3, 4, 5, 6, 7, 9]].isnan().any())


# ------------------------------------------------------------------ sampling

def kept(x, T, k, p, m):
    """The ids that the cuts leave, ascending, and their weights; x fp64, NaN counted as -inf."""
    x = np.where(np.isnan(x), -math.inf, x)
    order = np.lexsort((np.arange(x.size), -x))
    if k > 0:
        order = order[:k]
    top = x[order[0]]
    w = np.where(x[order] == top, 1.0, np.exp(np.where(np.isneginf(x[order] - top), -math.inf, x[order] - top) / T))
    if p < 1:
        n = int(np.flatnonzero(np.cumsum(w) >= max(p, 0.0) * w.sum())[0]) + 1
        order, w = order[:n], w[:n]
    ok = w >= min(m, 1.0)
    order, w = order[ok], w[ok]
    by = np.argsort(order)
    return order[by], w[by]


def draws(ids, w, rng, n):
    """n uniforms that stay away from the borders, and the ids they draw."""
    c = np.cumsum(w) / w.sum()
    out = []
    while len(out) < n:
        u = np.float32(rng.random())
        i = int(np.searchsorted(c, u, side="right"))
        if u < 1 and i < len(ids) and np.abs(c - u).min() > 2.0 ** -18 and w[i] / w.sum() > 2.0 ** -22:
            out.append((u, int(ids[i])))
    return out


PARAMS = [(0.0, 0, 1.0, 0.0), (1.0, 0, 1.0, 0.0), (0.7, 1, 1.0, 0.0), (1.0, 40, 1.0, 0.0), (1.3, 0, 0.9, 0.0),
          (0.8, 50, 0.8, 0.0), (1.0, 0, 1.0, 0.05), (1.0, 300, 0.95, 0.02), (0.05, 0, 0.99, 0.0), (5.0, 7, 0.5, 0.3),
          (1.0, -3, 2.0, -1.0), (1.0, 10 ** 6, 0.999, 0.0), (0.9, 0, 0.0, 0.0), (1.0, 0, 1.0, 7.0), (1e-30, 5, 1.0, 0.0)]


def sample(slm, logits, T, k, p, m, u):  # noqa: F811
    ids = ints([-9] * logits.shape[0])
    f = [None if x is None else torch.tensor(np.asarray(x, dtype=np.float32), device="cuda") for x in (T, p, m, u)]
    slm.sample_rows(logits, f[0], None if k is None else ints(list(k)), f[1], f[2], f[3], ids)
    return ids.tolist()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", [1, 2, 31, 1000, 32769, 128256, 262144])
def test_sample(slm, vocab, dtype):  # noqa: F811
    rng = np.random.default_rng(vocab)
    rows = []
    buf = torch.full((2 * len(PARAMS), vocab + 5), float("inf"), device="cuda", dtype=dtype)
    for i in range(2 * len(PARAMS)):
        x = rng.standard_normal(vocab) * 2.5
        x[rng.integers(0, vocab, 6)] += rng.random(6) * 9
        if i % 5 == 4:  # ties: a few values only
            x = np.round(x * 2) / 2
        if i % 7 == 6:  # what a mask leaves
            x[rng.random(vocab) < 0.5] = -math.inf
            x[int(rng.integers(0, vocab))] = 1.0
        buf[i, :vocab] = torch.from_numpy(x).to("cuda", dtype)
        rows.append(buf[i, :vocab].double().cpu().numpy())
    T, k, p, m = (list(c) * 2 for c in zip(*PARAMS))
    for _ in range(3):
        u, want = [], []
        for i, x in enumerate(rows):
            if not T[i] > 0:
                u.append(rng.random())
                want.append(int(np.lexsort((np.arange(vocab), -x))[0]))
                continue
            ids, w = kept(x, np.float64(np.float32(T[i])), k[i], np.float64(np.float32(p[i])), np.float64(np.float32(m[i])))
            (a, b), = draws(ids, w, rng, 1)
            u.append(a)
            want.append(b)
        assert sample(slm, buf[:, :vocab], T, k, p, m, u) == want


def test_sample_defaults(slm):  # noqa: F811
    """Parameters that are left out: the draw from softmax(logits) in index order."""
    rng = np.random.default_rng(1)
    x = torch.randn(40, 777, device="cuda")
    u, want = [], []
    for r in x.double().cpu().numpy():
        (a, b), = draws(*kept(r, 1.0, 0, 1.0, 0.0), rng, 1)
        u.append(a)
        want.append(b)
    assert sample(slm, x, None, None, None, None, u) == want


@pytest.mark.parametrize("vocab", [5, 5000, 200000])
def test_sample_odd_logits(slm, vocab):  # noqa: F811
    inf, nan = math.inf, math.nan
    x = torch.zeros(8, vocab, device="cuda")
    x[0] = -inf                       # nothing: token 0
    x[1] = nan
    x[2, 1], x[2, 3] = inf, inf       # equal parts of the infinite ones
    x[3] = nan
    x[3, 4] = -5.0                    # the only one
    x[4] = -inf
    x[4, 2] = -3e38
    x[5, 3] = 3e38                    # far above the rest
    x[6] = torch.arange(vocab, device="cuda") * -1e4
    x[7, 2] = nan                     # zeros: one of them, not the NaN
    for T, k, p, m in ((1.0, 0, 1.0, 0.0), (0.5, 3, 0.9, 0.1), (0.0, 0, 1.0, 0.0), (math.nan, 0, math.nan, math.nan),
                       (math.inf, 2, 1.0, 0.0)):
        ids = sample(slm, x, [T] * 8, [k] * 8, [p] * 8, [m] * 8, [0.0] * 8)
        last = sample(slm, x, [T] * 8, [k] * 8, [p] * 8, [m] * 8, [1.0 - 2.0 ** -24] * 8)
        assert ids[:7] == [0, 0, 1, 4, 2, 0 if T == inf and k == 2 else 3, 0], (T, ids)
        greedy = not T > 0
        if T != inf:
            assert last[:7] == [0, 0, 1 if greedy else 3, 4, 2, 3, 0], (T, last)
        assert ids[7] == 0 and last[7] == (0 if greedy else vocab - 1 if k == 0 else 1 if T == inf else [0, 1, 3][k - 1])
    assert sample(slm, x[7:], [1.0], [0], [nan], [nan], [1.0 - 2.0 ** -24]) == [vocab - 1]  # neither cut
    # uniforms outside [0, 1): cut to it
    z = torch.zeros(4, vocab, device="cuda")
    assert sample(slm, z, None, None, None, None, [-3.0, nan, 1.0, 7.0]) == [0, 0, vocab - 1, vocab - 1]


def test_sample_many_rows(slm):  # noqa: F811
    """More rows than a grid's waves; each its own draw.  The same call gives the same ids."""
    rows, vocab = 3001, 333
    rng = np.random.default_rng(3)
    x = torch.randn(rows, vocab, device="cuda") * 3
    T, k = [(0.0, 1.0, 0.6)[i % 3] for i in range(rows)], [(0, 9)[i % 2] for i in range(rows)]
    p, m = [(1.0, 0.9)[i // 2 % 2] for i in range(rows)], [(0.0, 0.1)[i // 4 % 2] for i in range(rows)]
    u, want = [], []
    for i, r in enumerate(x.double().cpu().numpy()):
        if T[i] == 0:
            u.append(0.5)
            want.append(int(r.argmax()))
            continue
        (a, b), = draws(*kept(r, np.float64(np.float32(T[i])), k[i], np.float64(np.float32(p[i])), np.float64(np.float32(m[i]))), rng, 1)
        u.append(a)
        want.append(b)
    assert sample(slm, x, T, k, p, m, u) == want
    assert sample(slm, x, T, k, p, m, u) == want


@pytest.mark.parametrize("k,p", [(0, 0.5), (0, 0.99), (700, 1.0), (3000, 0.9), (1, 0.5), (5000, 0.2)])
def test_sample_ties(slm, k, p):  # noqa: F811
    """Thousands of equal logits next to the border: the lowest indices come first, whichever way finds them."""
    vocab, rng = 20000, np.random.default_rng(2)
    for values in ([0.0], [0.0, 1.0], [0.0, 0.001], [-3.0, 0.0, 0.1]):
        x = torch.from_numpy(rng.choice(values, vocab)).float().cuda()
        ids, w = kept(x.double().cpu().numpy(), 1.0, k, np.float64(np.float32(p)), 0.0)
        got = draws(ids, w, rng, 8)
        assert sample(slm, x.expand(8, vocab), [1.0] * 8, [k] * 8, [p] * 8, [0.0] * 8, [g[0] for g in got]) == [g[1] for g in got]


def test_sample_largest_vocabulary(slm):  # noqa: F811
    vocab = 1 << 22
    x = torch.randn(2, vocab, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) * 3
    x[:, 4000000] = 16.0
    rng = np.random.default_rng(4)
    for T, k, p in ((0.0, 0, 1.0), (1.0, 30, 1.0), (0.7, 0, 0.8), (1.0, 0, 1.0)):
        u, want = [], []
        for r in x.double().cpu().numpy():
            if T == 0:
                u.append(0.3)
                want.append(int(r.argmax()))
                continue
            ids, w = kept(r, np.float64(np.float32(T)), k, np.float64(np.float32(p)), 0.0)
            c = np.cumsum(w) / w.sum()  # millions of borders: the middle of a token's part, the largest of some
            i = int(np.argmax(w * (rng.random(w.size) < 0.2)))
            a = np.float32((c[i] + (c[i - 1] if i else 0.0)) / 2)
            u.append(a)
            want.append(int(ids[i]))
        assert sample(slm, x, [T] * 2, [k] * 2, [p] * 2, None, u) == want


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("offset", [0, 1, 2, 3])
def test_sample_alignment(slm, dtype, offset):  # noqa: F811
    """Rows that begin anywhere."""
    vocab, rng = 5003, np.random.default_rng(offset)
    buf = torch.full((7, vocab + 9), float("inf"), device="cuda", dtype=dtype)
    x = buf[:, offset:offset + vocab]
    x.copy_(torch.randn(7, vocab, device="cuda") * 2)
    params = [(0.0, 0, 1.0), (1.0, 12, 1.0), (1.0, 0, 0.9), (1.0, 0, 1.0), (0.5, 900, 0.7), (2.0, 0, 0.3), (1.0, 5000, 1.0)]
    u, want = [], []
    for r, (T, k, p) in zip(x.double().cpu().numpy(), params):
        if T == 0:
            u.append(0.1)
            want.append(int(np.lexsort((np.arange(vocab), -r))[0]))
            continue
        (a, b), = draws(*kept(r, T, k, np.float64(np.float32(p)), 0.0), rng, 1)
        u.append(a)
        want.append(b)
    assert sample(slm, x, [q[0] for q in params], [q[1] for q in params], [q[2] for q in params], None, u) == want


def test_sample_distribution(slm):  # noqa: F811
    """A grid of uniforms over one row: every token as often as its probability says, to one draw."""
    x = torch.tensor([2.0, -1.0, 0.5, 2.0, -math.inf, 1.0, 0.0], device="cuda")
    n = 4096
    ids = sample(slm, x.expand(n, 7), None, [5] * n, None, None, [(i + 0.5) / n for i in range(n)])
    w = np.exp(x.double().cpu().numpy())
    w[1] = w[4] = 0
    got = np.bincount(ids, minlength=7)
    assert np.abs(got - n * w / w.sum()).max() <= 1.0 and got[1] == got[4] == 0


def test_sample_refusals(slm):  # noqa: F811
    x, u, ids = torch.zeros(2, 8, device="cuda"), torch.zeros(2, device="cuda"), ints([5, 5])
    one = torch.ones(2, device="cuda")
    for args, why in [((x.double(), None, None, None, None, u, ids), "float64"),
                      ((x.t(), None, None, None, None, u, ids), "adjacent"),
                      ((x, one[:1], None, None, None, u, ids), "temperature"),
                      ((x, None, one, None, None, u, ids), "top_k"),
                      ((x, None, None, one.double(), None, u, ids), "top_p"),
                      ((x, None, None, None, None, None, ids), "uniforms"),
                      ((x, None, None, None, None, u, ids.long()), "next_ids")]:
        with pytest.raises(ValueError, match=why):
            slm.sample_rows(*args)
    with pytest.raises(slm.SlmError, match="uniforms is not device memory"):
        slm.sample_rows(x, None, None, None, None, u.cpu(), ids)
    assert ids.tolist() == [5, 5]
    slm.sample_rows(x[:0], None, None, None, None, u[:0], ids[:0])  # no rows: nothing to do


# ------------------------------------------------------------------ all together

def test_steps_together(slm):  # noqa: F811
    """Prompts and then decode steps of three requests through a captured step of all calls, one of the
    requests ending on the way, against a cache kept in Python."""
    H, KV, hd, page, vocab, R = 4, 2, 64, 16, 500, 96
    g = torch.Generator(device="cuda").manual_seed(1)
    rope, axis = rope_table(400, hd), [j % 2 for j in range(hd // 2)]
    p = Pool([0, 0, 0], page, 12, 24, seed=2)
    kc = torch.full((24, KV, page, hd), float("nan"), device="cuda", dtype=BF16)
    vc = kc.clone()
    qkv = torch.zeros(R, (H + 2 * KV) * hd, device="cuda")
    q, k, v = (t.unflatten(1, (n, hd)) for t, n in zip(qkv.split([H * hd, KV * hd, KV * hd], 1), (H, KV, KV)))
    head = torch.randn(H * hd, vocab, device="cuda", generator=g) * 0.3
    q_rot, out = torch.zeros(R, H, hd, device="cuda", dtype=BF16), torch.zeros(R, H, hd, device="cuda", dtype=BF16)
    new, rows = ints([30, 17, 40]), R
    pos, slots, u = ints([0] * R), ints([0] * R, torch.int64), torch.zeros(R, device="cuda")
    ids, top_k = ints([0] * R), ints([20] * R)
    ws = torch.empty(slm.attention_rows_workspace_bytes(BF16, R, 3, H, KV, hd), dtype=torch.uint8, device="cuda")

    def step():
        slm.rows_plan(new, p.seq_len, p.page_table, page, p.free_pages, p.free_count, p.row_start, p.ctx_len, pos, slots,
                      p.seq_len, p.free_count, p.status)
        slm.kv_append_axes(k, v, kc, vc, p.page_table, p.row_start, p.ctx_len, p.status, rope, axis,
                           torch.stack([pos, pos // 2]), q=q, q_out=q_rot)
        slm.attention_paged_scored(q_rot, kc, vc, p.page_table, p.row_start, p.ctx_len, out, ws, p.status, cap=20.0, window=33)
        slm.sample_rows(out.float().flatten(1) @ head, None, top_k, None, None, u, ids)

    graph, hist = None, [[], [], []]
    for n in ([30, 17, 40], [1, 1, 1], [1, -1, 1], [1, 45, 1], [1, 1, 1]):
        qkv.copy_(torch.randn(qkv.shape, device="cuda", generator=g))
        u.copy_(torch.rand(R, device="cuda", generator=g))
        new.copy_(ints(n))
        if graph is None:
            side = torch.cuda.Stream()  # the first step eagerly, on a stream of its own
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step()
            torch.cuda.current_stream().wait_stream(side)
        else:
            graph.replay()
        start, ctx, want_pos, want_slots = p.expect(n)
        used = start[-1]
        assert p.row_start.tolist() == start and pos.tolist() == want_pos + [-1] * (R - used)
        assert slots.tolist()[:used] == want_slots and int(p.status.item()) == 0
        got = out.clone()
        at = torch.stack([pos, pos // 2])
        there = slots[:used]
        for x, y in ((k, kc[there // page, :, there % page]), (q, q_rot[:used])):  # fp32 in, bf16 out
            want, tol = turned(x[:used], rope, at[:, :used], axis)
            assert bool(((y.double() - want).abs() <= tol + H16 * want.abs()).all())
        assert bool((vc[there // page, :, there % page] == v[:used].to(BF16)).all())
        for s in range(3):
            if n[s] < 0:
                hist[s] = []
            for i in range(start[s], start[s + 1]):
                hist[s].append(int(slots[i]))
                at = ints(hist[s][-33:], torch.int64)
                K, V = (x[at // page, :, at % page].double() for x in (kc, vc))
                for h in range(H):
                    w = torch.softmax(20 * torch.tanh(K[:, h // 2] @ q_rot[i, h].double() / 8 / 20), 0)
                    want, mean = w @ V[:, h // 2], w @ V[:, h // 2].abs()
                    # roundings of weights and result; scores of up to 20 are within 2^-14
                    tol = H16 * (mean + want.abs()) + 2 * 2.0 ** -14 * 6
                    assert bool(((got[i, h].double() - want).abs() <= tol).all())
        logits = got.float().flatten(1) @ head
        assert ids[:used].tolist() == [int(i) for i in _pick(logits[:used], 20, u)]
        if graph is None:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            state = [x.clone() for x in (p.seq_len, p.free_count, p.row_start, p.ctx_len, p.page_table, p.free_pages)]
            with torch.cuda.graph(graph):
                step()
            for x, y in zip((p.seq_len, p.free_count, p.row_start, p.ctx_len, p.page_table, p.free_pages), state):
                x.copy_(y)


def _pick(logits, k, u):
    for i, x in enumerate(logits.double().cpu().numpy()):
        ids, w = kept(x, 1.0, k, 1.0, 0.0)
        c = np.cumsum(w) / w.sum()
        yield ids[int(np.searchsorted(c, float(u[i]), side="right"))]
