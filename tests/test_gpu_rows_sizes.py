"""The sizes at the ends of what the packed-row calls take: no row at all, the most sequences, and a
workspace that is kept for the largest batch."""
import itertools

import pytest

from test_gpu_rows import BF16, F32, Batch, check_attention, rope_table, slm  # noqa: F401  (slm: the fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_empty_tensors(slm, dtype):  # noqa: F811
    """rows = 0: empty tensors have no address, and the calls do nothing."""
    b = Batch(dtype, 4, 2, 64, [0, 0], [5, 0], 16, seed=1)
    assert b.q.data_ptr() == 0 and b.rows == 0
    out, ws = b.out(), b.workspace(slm)
    kc, vc = b.k_cache.clone(), b.v_cache.clone()
    qr = torch.empty_like(out)
    slm.kv_append(b.k, b.v, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, b.status, rope_table(6, 64), b.q, qr)
    slm.kv_append(b.k, b.v, b.k_cache, b.v_cache, b.page_table, b.row_start, None, b.status)
    slm.attention_paged(b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, out, ws, b.status)
    slm.attention_prompt(b.q, b.k, b.v, b.row_start, out, ws, b.status)
    torch.cuda.synchronize()
    assert torch.equal(b.k_cache.nan_to_num(9.0), kc.nan_to_num(9.0)) and torch.equal(b.v_cache.nan_to_num(9.0), vc.nan_to_num(9.0))
    assert int(b.status.item()) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_workspace_of_a_large_batch_serves_the_smaller_ones(slm, dtype):  # noqa: F811
    """The bytes do not grow when rows or nseq shrink."""
    rows, seqs = (1, 2, 5, 16, 17, 63, 64, 65, 500, 5000), (1, 2, 5, 64, 300, 523, 524, 1024)
    for G, hd in itertools.product((1, 3, 4, 7, 16, 17, 32), (8, 64, 72, 128, 136, 256)):
        size = lambda r, n: slm.attention_rows_workspace_bytes(dtype, r, n, 2 * G, 2, hd)  # noqa: E731, B023
        for i, j in itertools.product(range(len(rows)), range(len(seqs))):
            here = size(rows[i], seqs[j])
            assert here > 0
            assert i == 0 or size(rows[i - 1], seqs[j]) <= here, (G, hd, rows[i - 1], seqs[j])
            assert j == 0 or size(rows[i], seqs[j - 1]) <= here, (G, hd, rows[i], seqs[j - 1])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_one_workspace_for_a_shrinking_batch(slm, dtype):  # noqa: F811
    """A workspace of 64 tokens in 64 sequences, then a chunk of 64 tokens in one."""
    keep = None
    for new in ([1] * 64, [64]):
        b = Batch(dtype, 6, 2, 64, new, [700] * len(new), 16, seed=len(new))
        b.fill([n + c for n, c in zip(b.new, b.ctx)])
        keep = b.workspace(slm) if keep is None else keep
        out = b.out()
        slm.attention_paged(b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, out, keep, b.status)
        check_attention(b, out, b.seq_k, b.seq_v, dtype)


def test_workspace_of_more_rows_than_a_call_takes_is_zero(slm):  # noqa: F811
    assert slm.attention_rows_workspace_bytes(BF16, 1 << 30, 4, 4, 2, 64) > 0
    assert slm.attention_rows_workspace_bytes(BF16, (1 << 30) + 1, 4, 4, 2, 64) == 0


@pytest.mark.parametrize("dtype,hd", [(BF16, 64), (BF16, 128), (BF16, 256), (F32, 64), (F32, 128), (F32, 256)])
@pytest.mark.parametrize("new", [[1] * 1024, [(3, 0, 40, 1)[i % 4] for i in range(1024)]])
def test_the_most_sequences(slm, dtype, hd, new):  # noqa: F811
    """1,024 sequences, whose lengths leave the least shared memory to the kernels (the shallowest
    rings): single tokens, and chunks on the wide tiles."""
    b = Batch(dtype, 4, 2, hd, new, [(i * 37) % 200 for i in range(1024)], 16, seed=61)
    b.fill([n + c for n, c in zip(b.new, b.ctx)])
    out = b.out()
    slm.attention_paged(b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, out, b.workspace(slm), b.status)
    check_attention(b, out, b.seq_k, b.seq_v, dtype)
