"""Capped scores far below 0, next to keys that a row does not see: what a row does not see must not count
for the maximum that its weights are taken from, whether it is the rest of a block, another document, what
lies before a window or what other rows of the same warp see.  With scores below -126 in the log2 domain a
maximum of 0 leaves no weight at all, with somewhat larger ones not all of them.

The tolerances are those of test_gpu_scored.  Where a bound stands for the maximum it is at most 80 above the
largest score in the log2 domain, so weights of 2^-24 of the largest are normal numbers."""
import math

import pytest

from test_gpu_rows import BF16, F32, Batch, slm  # noqa: F401  (slm: the fixture)
from test_gpu_scored import arguments, check, documents

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def low(dtype, H, KV, hd, new, ctx, size, equal=False, seed=0):
    """A batch whose scores before the cap are all between -size and -0.9 size (`equal`: -size, exactly
    where size / sqrt(hd) is a bf16)."""
    b = Batch(dtype, H, KV, hd, new, ctx, 16, seed=hd + seed, lead=1, pad=2)
    g = torch.Generator(device="cuda").manual_seed(seed + 5)
    u = torch.where(torch.rand(hd, device="cuda", generator=g) < 0.5, -1.0, 1.0)
    for keys in b.seq_k:
        r = 1.0 - torch.rand(keys.shape[0], KV, 1, device="cuda", generator=g) * (0.0 if equal else 0.1)
        keys.copy_((-r * u).to(keys.dtype))
    b.q.copy_((u * (size / math.sqrt(hd))).expand(b.rows, H, hd).to(b.q.dtype))
    b.fill([n + c for n, c in zip(new, ctx)])
    return b


def run(slm, b, m, dtype):  # noqa: F811
    kw, out = arguments(b, m), b.out()
    slm.attention_paged_scored(b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, out, b.workspace(slm), b.status, **kw)
    check(b, out, b.seq_k, b.seq_v, m, kw, dtype)


SIZES = [(60.0, 100.0), (80.0, 90.0), (100.0, 300.0), (150.0, 1000.0), (3000.0, 1e6)]


@pytest.mark.parametrize("H,KV,hd", [(8, 2, 64), (8, 2, 128), (4, 4, 64)])
@pytest.mark.parametrize("length", [1, 31, 33, 96, 128, 130, 161, 256, 257, 300, 1000])
def test_one_row(slm, H, KV, hd, length):  # noqa: F811
    """A decode step whose last block is filled in part: every score is -100, the answer the mean of v."""
    b = low(BF16, H, KV, hd, [1], [length - 1], 100.0, equal=True)
    run(slm, b, dict(cap=1000.0), BF16)


@pytest.mark.parametrize("dtype,H,KV,hd", [(BF16, 8, 2, 64), (BF16, 8, 2, 128), (BF16, 4, 2, 80), (F32, 4, 2, 64)])
@pytest.mark.parametrize("size,cap", SIZES)
@pytest.mark.parametrize("masks", ["causal", "documents", "window", "prefix", "slopes"])
@pytest.mark.parametrize("new,ctx", [
    ([1] * 40, [(i * 97) % 700 for i in range(40)]),                  # steps; every length of a last block
    ([5, 3, 8, 2, 7], [126, 250, 123, 511, 300]),                     # a few rows, some on both sides of a block's edge
    ([150, 3, 40, 130, 64], [333, 2500, 0, 70, 127]),                 # chunks: rows of a warp end in different blocks
    ([2300, 40], [0, 2000])])                                         # long items
def test_masks(slm, dtype, H, KV, hd, size, cap, masks, new, ctx):  # noqa: F811
    b = low(dtype, H, KV, hd, new, ctx, size, seed=len(new))
    m = dict(cap=cap)
    if masks == "documents":
        m["first"] = documents(b, 7, 150)
    if masks == "window":
        m["window"] = 100
    if masks == "prefix":
        m["prefix"] = [((n + c) * (i % 4)) // 3 for i, (n, c) in enumerate(zip(new, ctx))]
    if masks == "slopes":
        m["slopes"] = True
    run(slm, b, m, dtype)


@pytest.mark.parametrize("H,KV,hd", [(8, 2, 64), (8, 2, 128)])
@pytest.mark.parametrize("cap", [90.0, 1000.0])
def test_two_levels(slm, H, KV, hd, cap):  # noqa: F811
    """Documents in turns of scores near 20 and near -100: rows of one warp take their maximum from a bound
    that holds for one document and not for the other."""
    # A warp has the positions 380 to 387, and a document ends at 383, with a block.  Tables of up to 512
    # positions leave items whole.
    b = low(BF16, H, KV, hd, [400, 20], [44, 100], 100.0)
    first = []
    for s, keys in enumerate(b.seq_k):
        L = keys.shape[0]
        of = [t // 24 * 24 for t in range(L)]
        keys[(torch.tensor(of, device="cuda") // 24) % 2 == 1] *= -0.2
        first.append(of[b.ctx[s]:])
    b.fill([n + c for n, c in zip(b.new, b.ctx)])
    run(slm, b, dict(cap=cap, first=first), BF16)


@pytest.mark.parametrize("H,KV,hd", [(8, 2, 64), (8, 2, 128)])
@pytest.mark.parametrize("new", [[700], [40, 1, 260], [3, 130]])
def test_prompts(slm, H, KV, hd, new):  # noqa: F811
    b = low(BF16, H, KV, hd, new, [0] * len(new), 150.0)
    k, v = (torch.full((b.rows, KV, hd), float("nan"), device="cuda", dtype=BF16) for _ in range(2))
    for s, n in enumerate(new):
        k[b.starts[s]:b.starts[s] + n], v[b.starts[s]:b.starts[s] + n] = b.seq_k[s], b.seq_v[s]
    m = dict(cap=500.0, first=documents(b, 2, 60))
    kw, out = arguments(b, m), b.out()
    slm.attention_prompt_scored(b.q, k, v, b.row_start, out, b.workspace(slm), b.status, **kw)
    check(b, out, b.seq_k, b.seq_v, m, kw, BF16)
