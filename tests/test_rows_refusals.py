"""What the packed-row calls (slm_kv_append, slm_attention_paged, slm_attention_prompt) refuse,
on the CPU: every argument check comes before the first look at a device, so made-up addresses
serve."""
import ctypes

import pytest

slm = pytest.importorskip("llama_decode_kv_gb300", reason="libslm.so not built")

A = 0x10000  # an aligned address that nothing dereferences


def _cache(**kw):
    d = dict(k=A, v=A, page_table=A, n_pages=4, page_size=16, table_ld=2, n_kv_heads=2, head_dim=16, kv_dtype=slm.SLM_BF16)
    d.update(kw)
    return slm.slm_kv_cache(**d)


def _rows(**kw):
    d = dict(row_start=A, ctx_len=A, nseq=2, rows=8)
    d.update(kw)
    return slm.slm_rows(**d)


def _append(cache=None, rows=None, **kw):
    d = dict(dtype=slm.SLM_BF16, k=A, k_ld=32, v=A, v_ld=32, rope=A, rope_len=9, n_heads=4, q=A, q_ld=64, q_out=A,
             q_out_ld=64, status=A)
    d.update(kw)
    c, r = cache or _cache(), rows or _rows()
    return slm.slm_kv_append(ctypes.byref(c), ctypes.byref(r), d["dtype"], d["k"], d["k_ld"], d["v"], d["v_ld"],
                             d["rope"], d["rope_len"], d["n_heads"], d["q"], d["q_ld"], d["q_out"], d["q_out_ld"],
                             d["status"], None)


def _paged(cache=None, rows=None, **kw):
    d = dict(n_heads=4, q=A, q_ld=64, out=A, out_ld=64, ws=A, ws_bytes=1 << 40, status=A)
    d.update(kw)
    c, r = cache or _cache(), rows or _rows()
    return slm.slm_attention_paged(ctypes.byref(c), ctypes.byref(r), d["n_heads"], d["q"], d["q_ld"], d["out"],
                                   d["out_ld"], d["ws"], d["ws_bytes"], d["status"], None)


def _prompt(rows=None, **kw):
    d = dict(dtype=slm.SLM_F32, n_heads=4, n_kv_heads=2, head_dim=16, q=A, q_ld=64, k=A, k_ld=32, v=A, v_ld=32, out=A,
             out_ld=64, ws=A, ws_bytes=1 << 40, status=A)
    d.update(kw)
    r = rows or _rows(ctx_len=None)
    return slm.slm_attention_prompt(ctypes.byref(r), d["dtype"], d["n_heads"], d["n_kv_heads"], d["head_dim"], d["q"],
                                    d["q_ld"], d["k"], d["k_ld"], d["v"], d["v_ld"], d["out"], d["out_ld"], d["ws"],
                                    d["ws_bytes"], d["status"], None)


def _why():
    return slm.slm_last_error(None).decode()


CACHES = [(dict(kv_dtype=2), "kv_dtype"), (dict(n_kv_heads=0), "n_kv_heads"), (dict(head_dim=12), "head_dim"),
          (dict(head_dim=264), "head_dim"), (dict(head_dim=0), "head_dim"), (dict(page_size=8), "page_size"),
          (dict(page_size=24), "page_size"), (dict(page_size=1 << 21), "page_size"), (dict(page_size=-16), "page_size"),
          (dict(n_pages=0), "n_pages"), (dict(table_ld=0), "table_ld"), (dict(k=None), "non-NULL"),
          (dict(page_table=None), "non-NULL"), (dict(v=A + 8), "aligned"), (dict(page_table=A + 2), "aligned")]
ROWS = [(dict(nseq=0), "nseq"), (dict(nseq=1025), "nseq"), (dict(rows=-1), "rows"), (dict(rows=(1 << 30) + 1), "rows"), (dict(row_start=None), "row_start"),
        (dict(row_start=A + 1), "aligned")]


@pytest.mark.parametrize("kw,why", CACHES)
def test_cache_is_checked(kw, why):
    for call in (_append, _paged):
        assert call(cache=_cache(**kw)) == slm.SLM_EINVAL and why in _why()


@pytest.mark.parametrize("kw,why", ROWS)
def test_rows_are_checked(kw, why):
    assert _append(rows=_rows(**kw)) == slm.SLM_EINVAL and why in _why()
    assert _paged(rows=_rows(**kw)) == slm.SLM_EINVAL and why in _why()
    assert _prompt(rows=_rows(**{"ctx_len": None, **kw})) == slm.SLM_EINVAL and why in _why()


@pytest.mark.parametrize("kw,why", [
    (dict(dtype=2), "dtype"), (dict(k=None), "k is NULL"), (dict(v=A + 8), "v must be 16-byte"), (dict(k_ld=31), "stride"),
    (dict(k_ld=36), "multiple of 16 bytes"), (dict(status=None), "status"), (dict(n_heads=3), "multiple"),
    (dict(q_out=None), "q_out is NULL"), (dict(q=None), "q is NULL"), (dict(rope=A + 4), "rope"), (dict(rope_len=0), "rope"),
    (dict(dtype=slm.SLM_F32), "in place"), (dict(q_ld=72, q_out_ld=64), "in place"), (dict(k_ld=1 << 33), "stride"),
])
def test_append_is_checked(kw, why):
    assert _append(**kw) == slm.SLM_EINVAL and why in _why()


@pytest.mark.parametrize("kw,why", [
    (dict(n_heads=3), "multiple"), (dict(n_heads=0), "multiple"), (dict(q=None), "q is NULL"), (dict(out=A + 2), "out must"),
    (dict(q_ld=60), "stride"), (dict(out_ld=68), "multiple of 16"), (dict(status=A + 1), "status"),
])
def test_attention_paged_is_checked(kw, why):
    assert _paged(**kw) == slm.SLM_EINVAL and why in _why()


@pytest.mark.parametrize("kw,why", [
    (dict(dtype=9), "dtype"), (dict(n_kv_heads=3), "multiple"), (dict(head_dim=20), "head_dim"), (dict(k=None), "k is NULL"),
    (dict(v_ld=30), "stride"), (dict(out=None), "out is NULL"), (dict(status=None), "status"),
])
def test_attention_prompt_is_checked(kw, why):
    assert _prompt(**kw) == slm.SLM_EINVAL and why in _why()


def test_prompt_refuses_cached_positions():
    assert _prompt(rows=_rows()) == slm.SLM_EINVAL and "ctx_len" in _why()


def test_large_groups_are_unsupported():
    c = _cache(n_kv_heads=1)
    assert _paged(cache=c, n_heads=65, q_ld=65 * 16, out_ld=65 * 16) == slm.SLM_EUNSUPPORTED and "at most 64" in _why()
    c = _cache(n_kv_heads=1, head_dim=136)
    assert _paged(cache=c, n_heads=33, q_ld=33 * 136, out_ld=33 * 136) == slm.SLM_EUNSUPPORTED and "at most 32" in _why()


def test_null_structs():
    assert slm.slm_kv_append(None, None, 0, A, 1, A, 1, None, 0, 0, None, 0, None, 0, A, None) == slm.SLM_EINVAL
    assert slm.slm_attention_paged(None, None, 1, A, 1, A, 1, A, 1, A, None) == slm.SLM_EINVAL
    assert slm.slm_attention_prompt(None, 0, 1, 1, 8, A, 8, A, 8, A, 8, A, 8, A, 1, A, None) == slm.SLM_EINVAL


def test_workspace_of_refused_shapes_is_zero():
    for a in ((2, 1, 1, 4, 2, 16), (0, -1, 1, 4, 2, 16), (0, 1, 0, 4, 2, 16), (0, 1, 1, 3, 2, 16), (0, 1, 1, 4, 2, 12),
              (1, 1, 1, 65, 1, 64)):
        assert slm.slm_attention_rows_workspace_bytes(*a) == 0


def test_binding_checks_tensors():
    torch = pytest.importorskip("torch")
    k = torch.zeros(3, 2, 16)
    kc = torch.zeros(4, 2, 16, 16)
    tab, rs, st = torch.zeros(1, 2, dtype=torch.int32), torch.tensor([0, 3], dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for bad in (dict(k=k.half()), dict(v=k[:2]), dict(k_cache=kc.transpose(1, 2)), dict(page_table=tab.long()),
                dict(row_start=rs.long()), dict(status=st[:0]), dict(rope=torch.zeros(3, 16, 2)), dict(q=k),
                dict(k=torch.zeros(3, 16, 2).transpose(1, 2)), dict(ctx_len=rs)):
        a = dict(k=k, v=k, k_cache=kc, v_cache=kc, page_table=tab, row_start=rs, ctx_len=None, status=st)
        a.update(bad)
        with pytest.raises(ValueError):
            slm.kv_append(**a, stream=0)
