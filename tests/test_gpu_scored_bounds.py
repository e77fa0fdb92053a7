"""Capped scores far from 0 and all of one sign: the maximum that a row's weights are taken from may be a
bound, the cap of the largest |q . k|, which then lies up to twice that above the largest score.  The
tolerances are those of test_gpu_scored: a score is rounded at a size of up to twice X in the log2 domain,
2.9 X u, and so is the bound, 1.5 X u, in all 4.4 X u log2 = 3 X u in the natural one, of the 4 X u there."""
import math

import pytest

from test_gpu_rows import BF16, F32, Batch, slm  # noqa: F401  (slm: the fixture)
from test_gpu_scored import arguments, check, documents

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype,H,KV,hd", [(BF16, 8, 2, 64), (BF16, 8, 2, 128), (F32, 4, 2, 64)])
@pytest.mark.parametrize("size,cap", [(20.0, 30.0), (27.7, 300.0), (28.0, 50.0), (60.0, 100.0), (300.0, 25.0), (300.0, 60.0)])
@pytest.mark.parametrize("signs", ["negative", "positive", "last", "rows"])
@pytest.mark.parametrize("docs", [False, True])
def test_one_sign(slm, dtype, H, KV, hd, size, cap, signs, docs):  # noqa: F811
    """size: the largest |score| before the cap; `last`: only a sequence's last keys are positive; `rows`:
    every other row is turned round."""
    new, ctx = [1, 150, 3, 40, 2300], [900, 333, 2500, 0, 0]
    b = Batch(dtype, H, KV, hd, new, ctx, 16, seed=hd, lead=1, pad=2)
    g = torch.Generator(device="cuda").manual_seed(int(size))
    u = torch.where(torch.rand(hd, device="cuda", generator=g) < 0.5, -1.0, 1.0)
    s = size / math.sqrt(hd)
    for keys in b.seq_k:
        n = keys.shape[0]
        r = (torch.rand(n, KV, 1, device="cuda", generator=g) * 0.5 + 0.5) * (1.0 if signs == "positive" else -1.0)
        if signs == "last":
            r[n - n // 9:] *= -1
        keys.copy_((r * u).to(keys.dtype))
    q = (u * s).expand(b.rows, H, hd).clone()
    if signs == "rows":
        q[::2] *= -1
    b.q.copy_(q.to(b.q.dtype))
    b.fill([n + c for n, c in zip(new, ctx)])
    m = dict(cap=cap)
    if docs:
        m["first"] = documents(b, 5, 700)
    kw, out = arguments(b, m), b.out()
    slm.attention_paged_scored(b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, out, b.workspace(slm), b.status, **kw)
    check(b, out, b.seq_k, b.seq_v, m, kw, dtype)
