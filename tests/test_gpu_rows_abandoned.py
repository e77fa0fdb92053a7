"""Abandoned packed-row attention calls on the tensor cores: a hand-off that never completes ends
the call with SLM_ROWS_TIMEOUT -- no hang, no fault -- and the next call is right.

slm_debug_rows_faults lets one kind of barrier wait for an arrival more than it gets.  Nothing else
is disturbed: the copies and the multiplications that were issued run, every other wait ends as
always, and those behind the missing hand-off end by the limit of a second or by the stop flag that
the first expired wait raises."""
import pytest

from test_gpu_rows import BF16, Batch, slm  # noqa: F401  (slm: the fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture
def faults(slm):  # noqa: F811
    yield slm.slm_debug_rows_faults
    assert slm.slm_debug_rows_faults(0) == 0


@pytest.mark.parametrize("lost", [1, 2])  # keys and values; a finished output tile
@pytest.mark.parametrize("hd,paged,new,ctx", [
    (64, True, [1], [20]),                           # a block per CTA: the other roles are done by then
    (64, True, [1, 1], [300, 700]),                  # one-tile items
    (128, False, [300], [0]),                        # two-tile items
    (64, True, [(1, 70, 0, 150)[i % 4] for i in range(41)], [(i * 211) % 1500 for i in range(41)]),  # many per CTA
    (128, True, [(1, 70, 0, 150)[i % 4] for i in range(41)], [(i * 211) % 1500 for i in range(41)]),
])
def test_timeout(slm, faults, lost, hd, paged, new, ctx):  # noqa: F811
    b = Batch(BF16, 6, 2, hd, new, ctx, 16, seed=hd)
    b.fill([n + c for n, c in zip(b.new, b.ctx)])
    ws = b.workspace(slm)

    def call():
        out = b.out()
        if paged:
            slm.attention_paged(b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, out, ws, b.status)
        else:
            slm.attention_prompt(b.q, b.k, b.v, b.row_start, out, ws, b.status)
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


def test_hook_checks_its_argument(slm):  # noqa: F811
    for lost in (-1, 3):
        assert slm.slm_debug_rows_faults(lost) == slm.SLM_EINVAL
