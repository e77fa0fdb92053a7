"""The README's serving step, run as it stands."""
import os
import re

import pytest

from test_gpu_rows import BF16, F32, rope_table, slm  # noqa: F401  (slm: the fixture)
from test_gpu_step import Pool, _pick, ints

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


@pytest.mark.parametrize("cache", [BF16, F32])
def test_example(slm, cache):  # noqa: F811
    blocks = [t for t in re.findall(r"```py\n(.*?)```", open(README).read(), re.S) if "rows_plan" in t]
    assert len(blocks) == 1
    H, KV, hd, page, rows, vocab, new = 4, 2, 64, 16, 60, 700, [20, 1, 30]
    g = torch.Generator(device="cuda").manual_seed(5)
    p = Pool([0, 0, 0], page, 12, 24, seed=4)
    k, v = (torch.randn(rows, KV, hd, device="cuda", generator=g) for _ in range(2))
    q = torch.randn(rows, H, hd, device="cuda", generator=g)
    q_rotated, out = (torch.zeros(rows, H, hd, device="cuda", dtype=cache) for _ in range(2))
    head = torch.randn(H * hd, vocab, device="cuda", generator=g) * 0.3
    uniforms = torch.rand(rows, device="cuda", generator=g)
    names = dict(
        slm=slm, new_len=ints(new), seq_len=p.seq_len, page_table=p.page_table, page_size=page, free_pages=p.free_pages,
        free_count=p.free_count, row_start=p.row_start, ctx_len=p.ctx_len, positions=ints([0] * rows),
        slots=ints([0] * rows, torch.int64), status=p.status, k=k, v=v, q=q, q_rotated=q_rotated, out=out,
        k_cache=torch.zeros(24, KV, page, hd, device="cuda", dtype=cache), rope=rope_table(100, hd),
        v_cache=torch.zeros(24, KV, page, hd, device="cuda", dtype=cache), axis_of_pair=[j % 3 for j in range(hd // 2)],
        axis_positions=ints([[i % 50 for i in range(rows)]] * 3), head=head, uniforms=uniforms, temperature=None, top_p=None,
        min_p=None, top_k=ints([20] * rows), next_ids=ints([0] * rows),
        ws=torch.empty(slm.attention_rows_workspace_bytes(cache, rows, 3, H, KV, hd), dtype=torch.uint8, device="cuda"))
    exec(blocks[0], names)  # noqa: S102  (the repository's own text)
    used = sum(new)
    assert int(p.status.item()) == 0 and p.seq_len.tolist() == new
    assert names["positions"].tolist()[:used] == [i for n in new for i in range(n)]
    for r in (0, 20, 21):  # the first row of a sequence sees itself alone: its weight, near 1, is divided by itself
        want = v[r].to(cache).float().repeat_interleave(H // KV, 0)
        assert bool(((out[r].float() - want).abs() <= 2.0 ** -20 * want.abs()).all())
    logits = names["logits"][:used]
    assert names["next_ids"].tolist()[:used] == [int(i) for i in _pick(logits, 20, uniforms)]
