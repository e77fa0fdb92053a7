"""slm_rows_plan without positions, without slots and without both: the other outputs are the same."""
import pytest

from test_gpu_rows import slm  # noqa: F401  (slm: the fixture)
from test_gpu_step import Pool, ints

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("kept", [(), ("positions",), ("slots",), ("positions", "slots")])
@pytest.mark.parametrize("rows", [70, 9000])
def test_some_outputs(slm, kept, rows):  # noqa: F811
    p = Pool([5, 0, 31, 16, 7, 0], 16, 8, 30, seed=1)
    new = [1, 0, 1, 17, -1, 40]
    positions, slots = ints([9] * rows), ints([9] * rows, torch.int64)
    p.seq_out, p.free_out = ints([9] * 6), ints([9])
    slm.rows_plan(ints(new), p.seq_len, p.page_table, 16, p.free_pages, p.free_count, p.row_start, p.ctx_len,
                  positions if "positions" in kept else None, slots if "slots" in kept else None, p.seq_out, p.free_out,
                  p.status, rows=None if kept else rows)
    start, ctx, pos, at = p.expect(new)
    want_pos, want_at = pos + [-1] * (rows - len(pos)), at + [-1] * (rows - len(at))
    assert positions.tolist() == (want_pos if "positions" in kept else [9] * rows)
    assert slots.tolist() == (want_at if "slots" in kept else [9] * rows)
    assert p.row_start.tolist() == start and p.ctx_len.tolist() == ctx
    assert p.page_table.tolist() == p.table and p.seq_out.tolist() == p.len and p.free_out.tolist() == [len(p.free)]
    assert p.free_pages[:len(p.free)].tolist() == p.free and int(p.status.item()) == 0


@pytest.mark.parametrize("kept", [(), ("positions",), ("slots",), ("positions", "slots")])
def test_more_rows_than_there_is_room_for(slm, kept):  # noqa: F811
    p = Pool([5, 0], 16, 8, 30)
    positions, slots, out, free = ints([9] * 7), ints([9] * 7, torch.int64), ints([9, 9]), ints([9])
    slm.rows_plan(ints([4, 4]), p.seq_len, p.page_table, 16, p.free_pages, p.free_count, p.row_start, p.ctx_len,
                  positions if "positions" in kept else None, slots if "slots" in kept else None, out, free, p.status, rows=7)
    assert int(p.status.item()) == slm.SLM_ROWS_LENGTH and p.row_start.tolist() == [0, 0, 0] and out.tolist() == [5, 0]
    assert positions.tolist() == [-1 if "positions" in kept else 9] * 7
    assert slots.tolist() == [-1 if "slots" in kept else 9] * 7


def test_refused(slm):  # noqa: F811
    p = Pool([5, 0], 16, 8, 30)
    positions, slots, out, free = ints([9] * 7), ints([9] * 7, torch.int64), ints([9, 9]), ints([9])

    def call(positions, slots, rows):
        slm.rows_plan(ints([1, 1]), p.seq_len, p.page_table, 16, p.free_pages, p.free_count, p.row_start, p.ctx_len, positions,
                      slots, out, free, p.status, rows=rows)

    for a, b, rows, why in ((None, None, None, "rows"), (positions, None, 8, "positions"), (None, slots, 8, "slots"),
                            (positions, slots[:6], None, "slots"), (None, slots.int(), None, "slots"), (slots, None, None, "positions")):
        with pytest.raises(ValueError, match=why):
            call(a, b, rows)
    with pytest.raises(slm.SlmError, match="rows"):
        call(None, None, -1)
