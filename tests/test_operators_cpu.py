"""Refusals of the operators on the caller's buffers that need no GPU: sizes and types are
checked before any address, and host addresses are never accepted."""
import ctypes

import numpy as np
import pytest


@pytest.fixture(scope="module")
def sd():
    from tests.conftest import build_library
    build_library()
    import stateful_decoding_b200 as sd
    return sd


def _aligned(nbytes):
    raw = np.zeros(nbytes + 16, np.uint8)
    return raw[-raw.ctypes.data % 16:][:nbytes]


def _cache(sd, **kw):
    buf = _aligned(1 << 16)
    f = dict(pages=buf.ctypes.data, scales=buf.ctypes.data, table=buf.ctypes.data, status=None,
             n_pages=4, rows=2, row_pages=2, page=16, kv_heads=2, dh=64)
    f.update(kw)
    c = sd.rlt_cache8(*[f[n] for n, _ in sd.rlt_cache8._fields_])
    c.keep = buf
    return c


def _append(sd, cache, dtype=0, n=1, k=None, rope=None, tok=128, row=128):
    a = cache.keep.ctypes.data if k is None else k
    return sd._lib.rlt_cache8_append(ctypes.byref(cache), dtype, a, row, tok, a, row, tok, a, None, n,
                                     ctypes.byref(rope) if rope else None, None)


def _attend(sd, cache, dtype=0, n=1, heads=2, scale=0.125, rope=None, tok=128, row=128):
    a = cache.keep.ctypes.data
    return sd._lib.rlt_cache8_attend(ctypes.byref(cache), dtype, a, row, tok, a, row, tok, heads, n, a,
                                     scale, ctypes.byref(rope) if rope else None, None)


@pytest.mark.parametrize("field,value,code", [
    ("page", 8, "UNSUPPORTED"), ("page", 48, "UNSUPPORTED"), ("dh", 80, "UNSUPPORTED"),
    ("dh", 256, "UNSUPPORTED"), ("n_pages", 0, "ARG"), ("row_pages", 0, "ARG"),
    ("kv_heads", 0, "ARG"), ("rows", -1, "ARG"), ("page", 0, "ARG"), ("dh", -64, "ARG"),
    ("row_pages", 1 << 30, "UNSUPPORTED"), ("pages", None, "ARG"), ("scales", None, "ARG"),
    ("table", None, "ARG")])
def test_cache_fields_refused(sd, field, value, code):
    want = getattr(sd, "RLT_E_" + code)
    c = _cache(sd, **{field: value})
    assert _append(sd, c) == want
    assert _attend(sd, c) == want


def test_host_buffers_and_nulls_refused(sd):
    c = _cache(sd)
    assert _append(sd, c) == sd.RLT_E_ARG          # host memory
    assert _attend(sd, c) == sd.RLT_E_ARG
    assert sd._lib.rlt_cache8_append(None, 0, None, 0, 0, None, 0, 0, None, None, 1, None,
                                     None) == sd.RLT_E_ARG
    assert sd._lib.rlt_cache8_attend(None, 0, None, 0, 0, None, 0, 0, 1, 1, None, 1.0, None,
                                     None) == sd.RLT_E_ARG
    odd = _cache(sd)
    odd.pages = odd.keep.ctypes.data + 8           # not on 16 bytes
    assert _append(sd, odd) == sd.RLT_E_ARG


def test_selection_refused(sd):
    a = _aligned(4096).ctypes.data
    ok = dict(dtype=0, finished=None, eos=-1, temperature=1.0, groups=1, beams=2, vocab=8, k=2)

    def call(**kw):
        f = {**ok, **kw}
        return sd._lib.rlt_beam_select(f["dtype"], a, a, f["finished"], f["eos"], f["temperature"],
                                       f["groups"], f["beams"], f["vocab"], f["k"], a, a, a, None,
                                       None)
    assert call() == sd.RLT_E_ARG                  # host memory
    for kw in (dict(dtype=2), dict(beams=0), dict(beams=65), dict(k=0), dict(k=65), dict(vocab=0),
               dict(vocab=1 << 24), dict(k=17), dict(groups=-1), dict(temperature=0.0),
               dict(temperature=float("nan")), dict(temperature=1e-9), dict(finished=a),
               dict(finished=a, eos=8)):
        assert call(**kw) == sd.RLT_E_ARG, kw
    assert call(groups=0) == sd.RLT_OK             # nothing to do


def test_reordering_refused(sd):
    a = _aligned(4096).ctypes.data
    call = lambda groups=1, beams=2, row=64, planes=2, plane=32, off=0, n=32: (  # noqa: E731
        sd._lib.rlt_rows_reorder(a, a, groups, beams, row, planes, plane, off, n, None))
    for kw in (dict(groups=-1), dict(beams=0), dict(beams=65), dict(planes=-1), dict(off=-1),
               dict(n=-1), dict(row=-64), dict(plane=-32), dict(n=33), dict(row=63),
               dict(plane=1 << 60), dict(planes=1, row=16)):
        assert call(**kw) == sd.RLT_E_ARG, kw
    assert call() == sd.RLT_E_ARG                  # host memory
    assert call(groups=0) == call(n=0) == call(planes=0) == sd.RLT_OK


def test_owners_refuse_host_tensors_and_wrong_types(sd):
    torch = pytest.importorskip("torch")
    with pytest.raises(TypeError):
        sd.Cache8(torch.zeros(4, 2, 2, 16, 64, dtype=torch.uint8), torch.ones(4, 2, 2),
                  torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(TypeError):
        sd.Cache8(np.zeros((4, 2, 2, 16, 64), np.uint8), None, None)
    with pytest.raises(TypeError):
        sd.rows_reorder(torch.zeros(2, 1, 1, 4), torch.zeros(1, 2, dtype=torch.int32))
    with pytest.raises(TypeError):
        sd.Rope(torch.zeros(4, 32), torch.zeros(4, 32))
    with pytest.raises(TypeError):
        sd.beam_select(torch.zeros(1, 2, 8), torch.zeros(1, 2), None, None, None)


def test_state_calls_refuse_nulls(sd):
    out = ctypes.c_void_p()
    assert sd._lib.rlt_state_create_with(None, 1, 8, 0, ctypes.byref(out)) == sd.RLT_E_ARG
    assert sd.rlt_state_create_with(None, 1, 8, sd.STATE_MEM8)[0] == sd.RLT_E_ARG
    a = np.zeros(4, np.int32)
    assert sd.rlt_state_reorder(None, a, 2) == sd.RLT_E_ARG
    assert sd.rlt_beam_step(None, a, None, -1, 1.0, 2, 0, a, a) == sd.RLT_E_ARG
