"""Long contexts and long prompts in the packed-row attention, with values that show what every
block of positions contributed.

Position t has the value 1 in column (t // 64) % head_dim and 0 in the others, so an output's column
is the sum of its blocks' softmax weights -- all of one sign, so that errors are relative, and a
block that is lost, doubled or weighed wrongly changes its column by its share.  Keys and queries
have one non-zero element each, so a score is one product.

Tolerances, relative to the column (u = 2^-24, h = 2^-8 half a step of bf16):
* equal scores (queries of zero): every weight is exactly 1, every sum a whole number below 2^24 and
  exact, in fp32 and on the tensor cores; 1 / l and the product with it round once each: 2 u, and h
  for the bf16 result.
* unequal scores: a score is off by ds <= 2^-22 * 8 |q k| / sqrt(hd) (the terms of the sum besides the one
  product are zero, and a step of the tensor core cuts the sum at 2^-22), a weight and the sum of
  weights by ds + 8 u each, the sums over L positions by L 2^-22 at the very most each (column and
  total), and bf16 calls round the weights (h) and the result (h).
Each test checks first that the smallest block's share is at least twice its tolerance.
"""
import math

import pytest

from test_gpu_rows import BF16, F32, Batch, slm  # noqa: F401  (slm: the fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U, H16 = 2.0 ** -24, 2.0 ** -8
STEPS = (-0.25, 0.0, 0.25, 0.125, -0.125)  # keys of the blocks, in a mixed order
Q = 8.0  # queries: scores of at most 0.25 * 8 / sqrt(64)


def positions(L, hd, KV, equal, dtype):
    """Keys and values [L][KV][hd]; the scores [L][KV] that a query of (Q, 0, ...) meets."""
    t = torch.arange(L, device="cuda")
    step = torch.tensor(STEPS, device="cuda")
    key = torch.stack([step[((t // 64) * (7 + 2 * g) + (t // 64) // 5) % len(STEPS)] for g in range(KV)], 1)
    k = torch.zeros(L, KV, hd, device="cuda")
    k[:, :, 0] = key  # exact in bf16
    score = torch.zeros_like(key) if equal else key
    v = torch.zeros(L, KV, hd, device="cuda")
    v[t, :, (t // 64) % hd] = 1.0
    return k.to(dtype), v.to(dtype), score.double() * (Q / math.sqrt(hd))


def check(out, score, ctx, equal, dtype):
    """out [n][H][hd] against the weights of the positions, row by row."""
    n, H, hd = out.shape
    L, KV = score.shape
    col = (torch.arange(L, device="cuda") // 64) % hd
    for g in range(KV):
        w = score[:, g].exp()
        part = torch.zeros(L, hd, dtype=torch.float64, device="cuda")
        part[torch.arange(L, device="cuda"), col] = w
        part = part.cumsum(0)[ctx:]  # row i sees positions 0 .. ctx + i
        want = part / w.cumsum(0)[ctx:, None]
        if equal:
            rel = 2.01 * U
        else:
            rel = 2 * (2.0 ** -22 * 8 * 0.25 + 8 * U) + 2 * L * 2.0 ** -22 + (H16 if dtype == BF16 else 0)
        rel += H16 if dtype == BF16 else 0
        share = math.exp(-0.5) * 64 / (64 * math.ceil(L / 64 / hd))  # the lightest block of the fullest column
        assert share > 2 * rel, (share, rel)
        for h in range(g * (H // KV), (g + 1) * (H // KV)):
            err = (out[:, h].double() - want).abs()
            assert bool((err <= rel * want).all()), (g, h, float((err / (rel * want)).nan_to_num(0.0).max()))


def queries(n, H, hd, equal, dtype):
    q = torch.zeros(n, H, hd, device="cuda")
    if not equal:
        q[:, :, 0] = Q
    return q.to(dtype)


CASES = [(BF16, 64), (BF16, 128), (BF16, 256), (F32, 64), (F32, 128), (F32, 256)]


@pytest.mark.parametrize("equal", [True, False])
@pytest.mark.parametrize("dtype,hd", CASES)
@pytest.mark.parametrize("H,KV,new,ctx", [
    (5, 1, [1], [40001]),            # one token: a piece for every CTA
    (5, 1, [40], [40001]),           # many rows and many pieces
    (4, 2, [1, 30, 1], [20000, 9000, 64]),
    (3, 3, [150, 1], [6000, 12000]),
])
def test_long_contexts(slm, dtype, hd, equal, H, KV, new, ctx):  # noqa: F811
    b = Batch(dtype, H, KV, hd, new, ctx, 256, seed=1)
    scores = []
    for s, (n, c) in enumerate(zip(new, ctx)):
        b.seq_k[s], b.seq_v[s], score = positions(n + c, hd, KV, equal, dtype)
        scores.append(score)
    b.fill([n + c for n, c in zip(new, ctx)])
    b.q[:] = queries(b.rows, H, hd, equal, dtype)
    out = b.out()
    slm.attention_paged(b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, out, b.workspace(slm), b.status)
    for s, (n, c) in enumerate(zip(new, ctx)):
        check(out[b.starts[s]:b.starts[s + 1]], scores[s], c, equal, dtype)
    assert int(b.status.item()) == 0


@pytest.mark.parametrize("equal", [True, False])
@pytest.mark.parametrize("dtype,hd", CASES)
@pytest.mark.parametrize("H,KV,lens", [(4, 2, [5000]), (6, 2, [2049, 1, 700, 3000])])
def test_long_prompts(slm, dtype, hd, equal, H, KV, lens):  # noqa: F811
    b = Batch(dtype, H, KV, hd, lens, None, 16, seed=2)
    scores = []
    for s, n in enumerate(lens):
        rows = slice(b.starts[s], b.starts[s + 1])
        b.k[rows], b.v[rows], score = positions(n, hd, KV, equal, dtype)
        scores.append(score)
    b.q[:] = queries(b.rows, H, hd, equal, dtype)
    out = b.out()
    slm.attention_prompt(b.q, b.k, b.v, b.row_start, out, b.workspace(slm), b.status)
    for s in range(len(lens)):
        check(out[b.starts[s]:b.starts[s + 1]], scores[s], 0, equal, dtype)
    assert int(b.status.item()) == 0
