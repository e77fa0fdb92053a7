"""slm_rows_plan ends sequences whose first pages were given back before (a window has left them behind, and
their entries are negative): only the others go onto the stack, so that no page is on it twice and none that
is no page.  Ids outside the pool are reported when they are put there.  Whole numbers throughout: they have
to be equal."""
import random

import pytest

from test_gpu_rows import BF16, Batch, slm  # noqa: F401  (slm: the fixture)
from test_gpu_scored import arguments, check
from test_gpu_step import Pool, ints

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


class Windowed(Pool):
    """A pool whose caller gives pages back itself."""

    def give_back(self, s, n):
        """The first n pages of sequence s, those that are left of them."""
        for b in range(n):
            if self.table[s][b] >= 0:
                self.free.append(self.table[s][b])
                self.table[s][b] = -1
        self.page_table[s, :n] = -1
        self.free_pages[:len(self.free)] = ints(self.free)
        self.free_count[0] = len(self.free)

    def expect(self, new):
        P = self.page
        for s, n in enumerate(new):
            if n < 0:
                self.free += [p for p in self.table[s][:-(-self.len[s] // P)] if p >= 0]
                self.len[s] = 0
        return super().expect([max(n, 0) for n in new])


@pytest.mark.parametrize("rows", [40, 9000])
@pytest.mark.parametrize("lens,gone,new", [
    ([40], [1], [-1]), ([40], [2], [-1]), ([40], [3], [-1]), ([16], [1], [-1]), ([1], [1], [-1]), ([15], [0], [-1]),
    ([100, 0, 70, 333], [3, 0, 5, 20], [-1, 3, -1, -1]), ([100, 64, 70, 333], [6, 4, 0, 7], [-1, 1, -1, 9]),
    ([5000, 40], [300, 1], [-1, 1]), ([5000, 200], [312, 7], [-1, 20]), ([5000, 200], [313, 0], [-1, -1]),
    ([i * 7 % 900 for i in range(1024)], [i % 30 for i in range(1024)], [-(i % 3 == 0) for i in range(1024)])])
def test_ends(slm, lens, gone, new, rows):  # noqa: F811
    held = [-(-c // 16) for c in lens]
    p = Windowed(lens, 16, max(held) + 3, sum(held) + 5, seed=len(lens))
    for s, n in enumerate(gone):
        p.give_back(s, min(n, held[s]))
    p.call(slm, new, rows)
    p.check(new, rows)
    assert len(set(p.free)) == len(p.free) and min(p.free) >= 0


def test_full_pool(slm):  # noqa: F811
    """Every page is free again: counted twice, they would be more than there are."""
    p = Windowed([64, 160], 16, 12, 14)
    p.give_back(0, 2)
    p.give_back(1, 9)
    p.call(slm, [-1, -1], 4)
    p.check([-1, -1], 4)
    assert sorted(p.free) == list(range(14))


def test_pages_in_the_same_step(slm):  # noqa: F811
    """What comes back is handed out in the same step, from the last one on."""
    p = Windowed([64, 32, 0], 16, 6, 6)
    p.give_back(0, 3)
    p.call(slm, [-1, -1, 90], 90)
    p.check([-1, -1, 90], 90)
    assert p.free == []


@pytest.mark.parametrize("rows", [12, 9000])
@pytest.mark.parametrize("entry,value", [(0, 200), (2, 1 << 30), (1, -1), (2, -7)])
def test_bad_ids(slm, entry, value, rows):  # noqa: F811
    """An id that is no page's, and a negative one behind the first that is not, is reported and passed on."""
    p = Pool([10, 40], 16, 100, 200)
    p.page_table[1, entry] = value
    p.table[1][entry] = value
    p.call(slm, [3, -1], rows)
    assert int(p.status.item()) == slm.SLM_ROWS_PAGE
    p.status.zero_()
    p.check([3, -1], rows)


def test_replayed_steps(slm):  # noqa: F811
    """A captured step in place, a caller that gives the pages before the window back between replays, ends and
    requests that come: every page is in one place all the time."""
    window, page, S, r = 70, 16, 6, random.Random(2)
    p = Windowed([0] * S, page, 40, 60, seed=5)
    new = [0] * S
    p.call(slm, new, 200, in_place=True)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        slm.rows_plan(p.new, p.seq_len, p.page_table, page, p.free_pages, p.free_count, p.row_start, p.ctx_len, p.positions,
                      p.slots, p.seq_len, p.free_count, p.status)
    for step in range(60):
        new = [-1 if p.len[s] and r.random() < 0.12 else r.choice([1, 1, 3, 33]) if p.len[s] < 500 else -1 for s in range(S)]
        p.new.copy_(ints(new))
        g.replay()
        p.check(new, 200)
        for s in range(S):
            if p.len[s]:
                p.give_back(s, max(0, p.len[s] + 1 - window) // page)  # the next row sees from here on
        used = [x for s in range(S) for x in p.table[s][:-(-p.len[s] // page)] if x >= 0]
        assert sorted(used + p.free) == list(range(60))


def test_window_goes_on_after_an_end(slm):  # noqa: F811
    """Plan and windowed attention together: a sequence that has lost its first pages ends, another one takes
    its pages, and each row sees its own keys only."""
    page, window = 16, 50
    b = Batch(BF16, 8, 2, 64, [1, 70], [299, 0], page, seed=3, spare=0)
    p = Windowed([300, 0], page, 25, 24)
    kc, vc = (torch.full((24, 2, page, 64), float("nan"), device="cuda", dtype=BF16) for _ in range(2))
    m = dict(window=window, cap=30.0)
    kw = arguments(b, m)
    p.give_back(0, 15)
    new = [-1, 1]
    for step in range(3):  # sequence 0 ends, sequence 1 comes and grows
        p.call(slm, new, b.rows)
        p.check(new, b.rows)
        p.seq_len, p.free_count = p.seq_out, p.free_out
        new = [0, 60] if step == 0 else [0, 9]
    n, L = 9, 70
    assert p.len == [0, L]
    for t in range(L):
        kc[p.table[1][t // page], :, t % page] = b.seq_k[1][t]
        vc[p.table[1][t // page], :, t % page] = b.seq_v[1][t]
    out = torch.full((b.rows, 8, 64), 7.0, device="cuda", dtype=BF16)
    slm.attention_paged_scored(b.q, kc, vc, p.page_table, p.row_start, p.ctx_len, out, b.workspace(slm), b.status, **kw)
    b.new, b.ctx, b.starts = [0, n], [0, L - n], [0, 0, n]
    check(b, out, b.seq_k, b.seq_v, m, kw, BF16)
