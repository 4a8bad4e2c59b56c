"""Reordering the rows of searches that stand at unequal positions: of each search the e_t not yet
consumed move, consumed ones stay, and nothing behind its positions is touched."""
import numpy as np
import pytest

import rlt_inputs as ri
from tests.test_beam_state_gpu import BASE, _model, _tokens, sd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mem8", [False, True])
@pytest.mark.parametrize("kw", [dict(), dict(dtype=ri.DT_BF16), dict(variant=2, chunk=2)])
@pytest.mark.parametrize("first,then,steps", [(5, 6, 2), (70, 3, 0), (3, 4, 4)])
def test_each_search_moves_what_it_has_not_consumed(sd, mem8, kw, first, then, steps):  # noqa: F811
    cfg = BASE.replace(**kw)
    model, _ = _model(sd, cfg)
    T, dh = 90, cfg.d // cfg.heads
    st = sd.State(model, 6, T, mem8=mem8)
    st.encode(_tokens(cfg, 6, T))                   # something behind every position
    st.reset()
    st.encode(_tokens(cfg, 6, first, seed=2))
    st.prefill(first)
    st.reset(np.array([2, 3], np.int32))            # the second search starts again
    st.encode(_tokens(cfg, 6, then, seed=3))
    st.prefill(steps)
    enc, dec = (p.tolist() for p in st.positions())
    assert enc[1] == first + then and enc[3] == then and dec[1] == first + steps and dec[3] == steps
    el = np.uint16 if cfg.dtype == ri.DT_BF16 else np.uint32

    def parts():
        out = {"e": st.read(sd.PART_E).view(np.uint32).reshape(6, 1, T, -1).copy(),
               "enc": st.read(sd.PART_ENC).view(el).reshape(6, -1, T, dh).copy()}
        if not mem8:
            out["mem"] = st.read(sd.PART_MEM).view(el).reshape(6, -1, T, dh).copy()
        return out
    before = parts()
    parents = [1, 0, 1, 0, 0, 0]
    st.reorder(np.array(parents, np.int32), 2)
    after = parts()
    for b, p in enumerate(parents):
        source = b // 2 * 2 + p
        for k in before:
            lo = dec[b] if k == "e" else 0
            want = before[k][b].copy()
            want[:, lo:enc[b]] = before[k][source][:, lo:enc[b]]
            assert np.array_equal(after[k][b], want), (k, b)
