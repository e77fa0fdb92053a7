"""Abandoned scored attention calls on the tensor cores, as test_gpu_rows_abandoned does for the plain
ones: a hand-off that never completes ends the call with SLM_ROWS_TIMEOUT -- no hang, no fault -- and the
next call is right.  Split items (up to 32 rows) hand more over among the softmax's warps; the code for
long items has two more warps."""
import pytest

from test_gpu_rows import BF16, Batch, slm  # noqa: F401  (slm: the fixture)
from test_gpu_rows_abandoned import faults  # noqa: F401  (the fixture)
from test_gpu_scored import arguments, documents

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("lost", [1, 2])  # keys and values; a finished output tile
@pytest.mark.parametrize("hd,wide,new,ctx", [
    (64, False, [1], [20]), (64, True, [1, 1], [300, 700]), (128, True, [1, 1], [300, 700]), (128, True, [300], [0]),
    (64, False, [(1, 70, 0, 150)[i % 4] for i in range(41)], [(i * 211) % 1500 for i in range(41)]),
    (128, True, [(1, 70, 0, 150)[i % 4] for i in range(41)], [(i * 211) % 1500 for i in range(41)]),
])
def test_timeout(slm, faults, lost, hd, wide, new, ctx):  # noqa: F811
    b = Batch(BF16, 6, 2, hd, new, ctx, 16, seed=hd)
    b.fill([n + c for n, c in zip(b.new, b.ctx)])
    if wide:
        b.page_table = torch.cat([b.page_table, torch.full((len(new), 200), -1, dtype=torch.int32, device="cuda")], 1)
    ws = b.workspace(slm)
    m = dict(cap=20.0, slopes=True)
    if not wide:
        m["first"] = documents(b, 2, 200)
    kw = arguments(b, m)

    def call():
        out = b.out()
        slm.attention_paged_scored(b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, out, ws, b.status, **kw)
        status = int(b.status.item())
        b.status.zero_()
        return out, status

    want, status = call()
    assert status == 0
    assert faults(lost) == 0
    assert call()[1] == slm.SLM_ROWS_TIMEOUT
    assert faults(0) == 0
    for _ in range(2):
        out, status = call()
        assert status == 0 and torch.equal(out, want)
