"""NaN and infinite scores in the packed-row attention, where a row's positions are shared by
several CTAs: the partial states are joined as the definition has it.

* A NaN score makes every weight of its row NaN, so a row that sees a NaN key is NaN, whichever
  pieces the key's positions make up.
* A score of -infinity has the weight 0: a row that also sees finite scores is the softmax over
  those.  Where every score is -infinity the row is 0 / 0, and a weight of 0 times a NaN value that
  the row sees is NaN.

Where a piece begins and ends depends on the GPU and on the batch, so the stretches are tried at
every block from the first on and at every length up to one and a half pieces: some of them are
exactly what one piece has.
"""
import pytest

from test_gpu_rows import BF16, F32, Batch, check_attention, slm  # noqa: F401  (slm: the fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

# H, KV, hd, new, ctx: a join of many pieces, of a few pieces with few rows, of a few pieces with
# 32 rows and more, and one-tile items of 64-wide and 128-wide heads
SHAPES = [
    (5, 1, 64, [1], [40001]),
    (6, 2, 64, [1] * 20, [4000] * 20),
    (6, 2, 64, [40] * 12, [3000] * 12),
    (6, 2, 128, [1] * 20, [4000] * 20),
    (8, 2, 128, [40, 150], [9000, 9000]),
]
SHAPES_F32 = SHAPES[:3] + [(4, 2, 256, [1] * 20, [2000] * 20), (4, 2, 256, [40, 50], [3000, 3000])]
CASES = [(BF16, *s) for s in SHAPES] + [(F32, *s) for s in SHAPES_F32]
PAGE = 64  # a block of the CUDA-core kernels, half of one of the tensor-core kernel


class Poisoned(Batch):
    """A batch in the cache whose stretches of one kv head of one sequence can be overwritten."""

    def __init__(self, slm, dtype, H, KV, hd, new, ctx, seed, positive=False):  # noqa: F811
        super().__init__(dtype, H, KV, hd, new, ctx, PAGE, seed=seed)
        if positive:
            self.q = self.q.abs() + 0.125
        self.slm, self.ws = slm, self.workspace(slm)
        self.s, self.g, self.G = len(new) // 2, KV - 1, H // KV
        self.fill([n + c for n, c in zip(self.new, self.ctx)])

    def run(self):
        out = self.out()
        self.slm.attention_paged(self.q, self.k_cache, self.v_cache, self.page_table, self.row_start, self.ctx_len, out,
                                 self.ws, self.status)
        return out

    def stretches(self):
        """(pages, first position, position behind) of the stretches, all of them seen by every row."""
        step = 2 if self.dtype == BF16 and self.hd <= 128 else 1
        for n in range(1, 14):
            for a in range(n + 2):
                lo, hi = a * step, (a + n) * step
                if hi * PAGE <= self.ctx[self.s]:
                    yield torch.tensor(self.table[self.s][lo:hi], device="cuda"), lo * PAGE, hi * PAGE

    def mine(self, out):
        rows = slice(self.starts[self.s], self.starts[self.s + 1])
        return out[rows, self.g * self.G:(self.g + 1) * self.G]


@pytest.mark.parametrize("dtype,H,KV,hd,new,ctx", CASES)
def test_nan_keys_are_seen(slm, dtype, H, KV, hd, new, ctx):  # noqa: F811
    """That head's rows are NaN, every other result keeps its bits."""
    b = Poisoned(slm, dtype, H, KV, hd, new, ctx, 5)
    want = b.run()
    assert bool(torch.isfinite(want).all())
    b.mine(want).zero_()
    for pages, lo, hi in b.stretches():
        keep = b.k_cache[pages, b.g].clone()
        b.k_cache[pages, b.g] = float("nan")
        got = b.run()
        b.k_cache[pages, b.g] = keep
        assert bool(torch.isnan(b.mine(got)).all()), (lo, hi)
        b.mine(got).zero_()
        assert torch.equal(got, want), (lo, hi)
    assert int(b.status.item()) == 0


@pytest.mark.parametrize("dtype,H,KV,hd,new,ctx", CASES)
def test_nan_values_under_scores_of_minus_infinity(slm, dtype, H, KV, hd, new, ctx):  # noqa: F811
    b = Poisoned(slm, dtype, H, KV, hd, new, ctx, 6, positive=True)
    for pages, lo, hi in b.stretches():
        k, v = b.k_cache[pages, b.g].clone(), b.v_cache[pages, b.g].clone()
        b.k_cache[pages, b.g] = float("-inf")
        b.v_cache[pages, b.g] = float("nan")
        got = b.run()
        b.k_cache[pages, b.g], b.v_cache[pages, b.g] = k, v
        assert bool(torch.isnan(b.mine(got)).all()), (lo, hi)


@pytest.mark.parametrize("dtype,H,KV,hd,new,ctx", CASES)
def test_scores_of_minus_infinity_weigh_nothing(slm, dtype, H, KV, hd, new, ctx):  # noqa: F811
    """Keys of -infinity over three quarters of a context under positive queries: those positions
    drop out.  Over all of it: 0 / 0."""
    b = Poisoned(slm, dtype, H, KV, hd, new, ctx, 7, positive=True)
    s = b.s
    lo, hi = ctx[s] // 8, 7 * ctx[s] // 8
    b.seq_k[s][lo:hi] = float("-inf")
    b.fill([n + c for n, c in zip(b.new, b.ctx)])
    out = b.run()
    # the definition over the positions that are left (the stretch is seen by every row)
    keep = torch.cat([torch.arange(0, lo), torch.arange(hi, new[s] + ctx[s])]).to("cuda")
    keys, values = list(b.seq_k), list(b.seq_v)
    keys[s], values[s] = keys[s][keep], values[s][keep]
    b.ctx[s] -= hi - lo
    check_attention(b, out, keys, values, dtype)
    b.ctx[s] = ctx[s]
    b.seq_k[s][:] = float("-inf")
    b.fill([n + c for n, c in zip(b.new, b.ctx)])
    assert bool(torch.isnan(b.mine(b.run())).all())
