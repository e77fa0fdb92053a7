"""The same scored attention call gives the same bits, whatever ran before it: what earlier tiles left
behind a sequence's last key or row in the kernel's memories must not choose how a score is computed."""
import pytest

from test_gpu_rows import BF16, F32, Batch, slm  # noqa: F401  (slm: the fixture)
from test_gpu_scored import arguments, documents

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("masks", ["cap", "cap_slopes", "window_cap", "documents_cap", "prefix_slopes_cap"])
@pytest.mark.parametrize("hd,H,KV,new,ctx", [
    (64, 6, 2, [(1, 70, 0, 150)[i % 4] for i in range(41)], [(i * 211) % 1500 for i in range(41)]),
    (128, 6, 2, [(1, 70, 0, 150)[i % 4] for i in range(41)], [(i * 211) % 1500 for i in range(41)]),
    (128, 8, 1, [1] * 23, [(i * 397) % 3000 for i in range(23)]),
    (64, 8, 8, [(300, 37)[i % 2] for i in range(9)], [0] * 9),
    (128, 4, 2, [2500], [700]),
])
def test_same_bits(slm, dtype, masks, hd, H, KV, new, ctx):  # noqa: F811
    b = Batch(dtype, H, KV, hd, new, ctx, 16, seed=hd + H)
    b.fill([n + c for n, c in zip(b.new, b.ctx)])
    ws = b.workspace(slm)
    m = {"cap": 10.0, "slopes": "slopes" in masks}
    if "window" in masks:
        m["window"] = 100
    if "documents" in masks:
        m["first"] = documents(b, 3, 200)
    if "prefix" in masks:
        m["prefix"] = [(i * 61) % 500 for i in range(len(new))]
    kw = arguments(b, m)
    loud = [t.clone() for t in (b.q, b.k_cache, b.v_cache)]
    for t in loud:
        t.copy_(torch.nan_to_num(t.float(), 0.0, 0.0, 0.0) * 40)
    lengths = b.ctx_len // 2

    def call(q, k, v, ctx_len):
        out = b.out()
        slm.attention_paged_scored(q, k, v, b.page_table, b.row_start, ctx_len, out, ws, b.status, **kw)
        assert int(b.status.item()) == 0
        return out

    want = call(b.q, b.k_cache, b.v_cache, b.ctx_len)
    for i in range(12):
        if i % 2:
            call(*loud, lengths)
        assert torch.equal(call(b.q, b.k_cache, b.v_cache, b.ctx_len), want)
