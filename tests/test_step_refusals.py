"""What the calls of a serving step (slm_rows_plan, slm_kv_append_axes, slm_attention_*_scored,
slm_sample_rows) refuse, on the CPU: every argument check comes before the first look at a device, so
made-up addresses serve."""
import ctypes
import math
import os

import pytest

from test_rows_refusals import A, CACHES, ROWS, _cache, _rows, _why

slm = pytest.importorskip("llama_decode_kv_gb300", reason="libslm.so not built")

AXES = (ctypes.c_int8 * 8)(*[0, 1, 2, 0, 1, 2, -1, -1])


def _plan(**kw):
    d = dict(page_table=A, free_pages=A, free_count=A, seq_len=A, nseq=3, table_ld=4, n_pages=9, page_size=16, new_len=A,
             rows=8, row_start=A, ctx_len=A, positions=A, slots=A, seq_len_out=A, free_count_out=A, status=A)
    d.update(kw)
    pool = slm.slm_page_pool(*[d[n] for n, _ in slm.slm_page_pool._fields_])
    return slm.slm_rows_plan(ctypes.byref(pool) if d.get("pool", True) else None, d["new_len"], d["rows"], d["row_start"],
                             d["ctx_len"], d["positions"], d["slots"], d["seq_len_out"], d["free_count_out"], d["status"], None)


@pytest.mark.parametrize("kw,why", [
    (dict(pool=None), "pool"), (dict(nseq=0), "nseq"), (dict(nseq=1025), "nseq"), (dict(rows=-1), "rows"),
    (dict(rows=(1 << 30) + 1), "rows"), (dict(page_size=8), "page_size"), (dict(page_size=48), "page_size"),
    (dict(page_size=1 << 21), "page_size"), (dict(n_pages=0), "n_pages"), (dict(table_ld=0), "table_ld")] +
    [({n: None}, n) for n in ("page_table", "free_pages", "free_count", "seq_len", "new_len", "row_start", "ctx_len",
                              "seq_len_out", "free_count_out", "status")] +
    [({n: A + 2}, n) for n in ("page_table", "free_pages", "free_count", "seq_len", "new_len", "row_start", "ctx_len",
                               "positions", "seq_len_out", "free_count_out", "status")] + [(dict(slots=A + 4), "slots")])
def test_plan(kw, why):
    assert _plan(**kw) == slm.SLM_EINVAL and why in _why()


def _axes(cache=None, rows=None, **kw):
    d = dict(dtype=slm.SLM_BF16, k=A, k_ld=32, v=A, v_ld=32, rope=A, rope_len=9, n_axes=3, axis=AXES, positions=A, pos_ld=8,
             n_heads=4, q=A, q_ld=64, q_out=A, q_out_ld=64, status=A)
    d.update(kw)
    c, r = cache or _cache(), rows or _rows()
    return slm.slm_kv_append_axes(ctypes.byref(c), ctypes.byref(r), d["dtype"], d["k"], d["k_ld"], d["v"], d["v_ld"],
                                  d["rope"], d["rope_len"], d["n_axes"], d["axis"], d["positions"], d["pos_ld"], d["n_heads"],
                                  d["q"], d["q_ld"], d["q_out"], d["q_out_ld"], d["status"], None)


@pytest.mark.parametrize("kw,why", [
    (dict(n_axes=0), "n_axes"), (dict(n_axes=9), "n_axes"), (dict(n_axes=2), "axis_of_pair[2]"), (dict(axis=None), "axis_of_pair"),
    (dict(axis=(ctypes.c_int8 * 8)(0, 0, -2)), "axis_of_pair[2]"), (dict(rope=None), "rope"), (dict(rope=A + 8), "rope"),
    (dict(rope_len=0), "rope"), (dict(positions=None), "positions"), (dict(positions=A + 1), "positions"),
    (dict(pos_ld=7), "positions_ld"), (dict(pos_ld=-8), "positions_ld"), (dict(dtype=2), "dtype"), (dict(k=None), "k is NULL"),
    (dict(v_ld=31), "stride"), (dict(n_heads=3), "n_heads"), (dict(q_out=None), "q_out"), (dict(status=None), "status")])
def test_append_axes(kw, why):
    assert _axes(**kw) == slm.SLM_EINVAL and why in _why()


def _paged(cache=None, rows=None, scores=True, **kw):
    d = dict(scale=0.0, cap=0.0, slopes=None, prefix_len=None, first=None, window=0)
    d.update(kw)
    s = slm.slm_scores(*[d[n] for n, _ in slm.slm_scores._fields_])
    c, r = cache or _cache(), rows or _rows()
    return slm.slm_attention_paged_scored(ctypes.byref(c), ctypes.byref(r), ctypes.byref(s) if scores else None, 4, A, 64, A, 64,
                                          A, 1 << 40, A, None)


def _prompt(rows=None, scores=True, **kw):
    d = dict(scale=0.0, cap=0.0, slopes=None, prefix_len=None, first=None, window=0)
    d.update(kw)
    s = slm.slm_scores(*[d[n] for n, _ in slm.slm_scores._fields_])
    r = rows or _rows(ctx_len=None)
    return slm.slm_attention_prompt_scored(ctypes.byref(r), ctypes.byref(s) if scores else None, slm.SLM_F32, 4, 2, 16, A, 64, A,
                                           32, A, 32, A, 64, A, 1 << 40, A, None)


@pytest.mark.parametrize("kw,why", [
    (dict(scores=False), "scores"), (dict(scale=-1.0), "scale"), (dict(scale=math.nan), "scale"), (dict(scale=math.inf), "scale"),
    (dict(cap=-0.5), "cap"), (dict(cap=math.nan), "cap"), (dict(cap=math.inf), "cap"), (dict(window=-1), "window"),
    (dict(slopes=A + 2), "aligned"), (dict(prefix_len=A + 2), "aligned"), (dict(first=A + 1), "aligned")])
def test_scores(kw, why):
    for call in (_paged, _prompt):
        assert call(**kw) == slm.SLM_EINVAL and why in _why()


@pytest.mark.parametrize("kw,why", CACHES)
def test_cache_is_checked(kw, why):
    for call in (_axes, _paged):
        assert call(cache=_cache(**kw)) == slm.SLM_EINVAL and why in _why()


@pytest.mark.parametrize("kw,why", ROWS)
def test_rows_are_checked(kw, why):
    assert _axes(rows=_rows(**kw)) == slm.SLM_EINVAL and why in _why()
    assert _paged(rows=_rows(**kw)) == slm.SLM_EINVAL and why in _why()
    assert _prompt(rows=_rows(**{"ctx_len": None, **kw})) == slm.SLM_EINVAL and why in _why()


def _sample(**kw):
    d = dict(rows=2, vocab=50, dtype=slm.SLM_F32, logits=A, ld=50, temperature=A, top_k=A, top_p=A, min_p=A, uniforms=A, ids=A)
    d.update(kw)
    return slm.slm_sample_rows(*d.values(), None)


@pytest.mark.parametrize("kw,why", [
    (dict(rows=-1), "rows"), (dict(vocab=0), "vocab"), (dict(vocab=(1 << 22) + 1), "vocab"), (dict(dtype=2), "dtype"),
    (dict(ld=49), "stride"), (dict(ld=-50), "stride"), (dict(logits=None), "logits"), (dict(uniforms=None), "uniforms"),
    (dict(ids=None), "next_ids"), (dict(logits=A + 2), "logits"), (dict(top_k=A + 1), "top_k"), (dict(ids=A + 2), "next_ids")])
def test_sample(kw, why):
    assert _sample(**kw) == slm.SLM_EINVAL and why in _why()


def test_without_a_device():
    """Good arguments get as far as the device."""
    if os.path.exists("/dev/nvidiactl"):
        pytest.skip("a device is there")
    for rc in (_plan(), _axes(), _paged(), _prompt(), _sample()):
        assert rc == slm.SLM_ECUDA
