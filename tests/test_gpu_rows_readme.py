"""The README's packed-row example, run as it stands."""
import os
import re

import pytest

from test_gpu_rows import BF16, F32, Batch, check_attention, rope_table, slm  # noqa: F401  (slm: the fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


@pytest.mark.parametrize("dtype,cache", [(F32, BF16), (F32, F32), (BF16, BF16), (BF16, F32)])
def test_example(slm, dtype, cache):  # noqa: F811
    """Rows straight from a projection in either type, into a cache of either type."""
    blocks = [t for t in re.findall(r"```python\n(.*?)```", open(README).read(), re.S) if "kv_append" in t]
    assert len(blocks) == 1
    H, KV, hd, new, ctx = 9, 3, 64, [200, 1, 30], [10, 300, 0]
    b = Batch(dtype, H, KV, hd, new, ctx, 16, cache, seed=4)
    b.fill(b.ctx)
    q_rotated, out = b.out(), b.out()
    names = dict(slm=slm, torch=torch, q=b.q, k=b.k, v=b.v, q_rotated=q_rotated, out=out, k_cache=b.k_cache,
                 v_cache=b.v_cache, page_table=b.page_table, row_start=b.row_start, ctx_len=b.ctx_len, status=b.status,
                 rope=rope_table(301, hd), rows=b.rows, nseq=len(new), heads=H, kv_heads=KV, head_dim=hd)
    exec(blocks[0], names)  # noqa: S102  (the repository's own text)
    keys, values = [], []
    for s, (n, c) in enumerate(zip(new, ctx)):  # what the cache holds now
        pos = torch.arange(n + c, device="cuda")
        pages = b.page_table[s].long()[pos // 16]
        keys.append(b.k_cache[pages, :, pos % 16])
        values.append(b.v_cache[pages, :, pos % 16])
    b.q = q_rotated
    check_attention(b, out, keys, values, cache)
