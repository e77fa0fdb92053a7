"""Empty tensors and tensors with gaps in the packed-row calls, on the CPU: what the argument checks
make of them before the first look at a device."""
import pytest

from test_rows_refusals import _append, _paged, _prompt, _rows, _why, slm


def _passes_the_checks(rc):
    """The arguments were accepted: what stops the call is the missing device, or, with a device,
    that the made-up addresses are not its memory."""
    return rc == slm.SLM_ECUDA or (rc == slm.SLM_EINVAL and "not device memory" in _why())


def test_no_rows_need_no_address():
    none = dict(q=None, q_ld=0)
    assert _passes_the_checks(_append(rows=_rows(rows=0), k=None, v=None, q=None, q_out=None, k_ld=0, v_ld=0)), _why()
    assert _passes_the_checks(_paged(rows=_rows(rows=0), out=None, out_ld=0, ws=None, ws_bytes=0, **none)), _why()
    assert _passes_the_checks(_prompt(rows=_rows(rows=0, ctx_len=None), k=None, v=None, out=None, ws=None, **none)), _why()


def test_one_row_needs_its_addresses():
    assert _append(rows=_rows(rows=1), k=None) == slm.SLM_EINVAL and "k is NULL" in _why()
    assert _paged(rows=_rows(rows=1), out=None) == slm.SLM_EINVAL and "out is NULL" in _why()


def test_binding_takes_empty_tensors():
    torch = pytest.importorskip("torch")
    k, kc = torch.zeros(0, 2, 16), torch.zeros(4, 2, 16, 16)
    tab, rs, st = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)
    for call in (lambda: slm.kv_append(k, k, kc, kc, tab, rs, None, st, stream=0),
                 lambda: slm.kv_append(k, k, kc, kc, tab, rs, None, st, torch.zeros(3, 8, 2), k, k, stream=0),
                 lambda: slm.attention_paged(k, kc, kc, tab, rs, None, k, ws, st, stream=0),
                 lambda: slm.attention_prompt(k, k, k, rs, k, ws, st, stream=0)):
        with pytest.raises(slm.SlmError) as e:  # host memory, or no device to look at
            call()
        assert _passes_the_checks(e.value.code), e.value


def test_binding_refuses_an_empty_rotation_table():
    """A table of no positions is not the same as no table (nothing rotated)."""
    torch = pytest.importorskip("torch")
    k, kc = torch.zeros(3, 2, 16), torch.zeros(4, 2, 16, 16)
    tab, rs, st = torch.zeros(1, 2, dtype=torch.int32), torch.tensor([0, 3], dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="no position"):
        slm.kv_append(k, k, kc, kc, tab, rs, None, st, torch.zeros(0, 8, 2), stream=0)


def test_binding_refuses_a_workspace_with_gaps():
    """The library writes nbytes from the first element on: with gaps, past the tensor's elements
    into its neighbours'."""
    torch = pytest.importorskip("torch")
    k, kc = torch.zeros(3, 2, 16), torch.zeros(4, 2, 16, 16)
    tab, rs, st = torch.zeros(1, 2, dtype=torch.int32), torch.tensor([0, 3], dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)[::2]
    with pytest.raises(ValueError, match="workspace"):
        slm.attention_paged(k, kc, kc, tab, rs, None, k, ws, st, stream=0)
    with pytest.raises(ValueError, match="workspace"):
        slm.attention_prompt(k, k, k, rs, k, ws, st, stream=0)
