"""The sizes at the ends of what the packed-row calls take: no row at all."""
import pytest

from test_gpu_rows import BF16, F32, Batch, rope_table, slm  # noqa: F401  (slm: the fixture)

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
