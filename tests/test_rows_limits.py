"""Head counts beyond what the packed-row kernels count in 32 bits are refused (on the CPU)."""
from test_rows_refusals import _append, _cache, _paged, _prompt, _rows, _why, slm


def test_head_counts():
    most = 65536
    wide = _rows(rows=1)  # one row: its stride has no meaning
    # (n_heads + 2 n_kv_heads) of a row would pass 2^31
    assert _append(rows=wide, n_heads=2 ** 31 - 2) == slm.SLM_EINVAL and "n_heads" in _why()
    assert _append(rows=wide, n_heads=most + 2) == slm.SLM_EINVAL and "n_heads" in _why()
    for call in (_append, _paged):
        assert call(cache=_cache(n_kv_heads=most + 1), rows=wide, n_heads=most + 1) == slm.SLM_EINVAL and "n_kv_heads" in _why()
    assert _prompt(rows=_rows(rows=1, ctx_len=None), n_heads=most + 2, n_kv_heads=most + 2) == slm.SLM_EINVAL and "n_heads" in _why()
    assert slm.slm_attention_rows_workspace_bytes(1, 1, 1, most + 2, most + 2, 64) == 0 and "n_heads" in _why()
    # the most: accepted by the checks, stopped by the missing device or by the made-up addresses
    for rc in (_append(rows=wide, n_heads=most), _append(cache=_cache(n_kv_heads=most), rows=wide, n_heads=most)):
        assert rc == slm.SLM_ECUDA or "not device memory" in _why()
