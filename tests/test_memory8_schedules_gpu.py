"""An 8-bit memory under schedules that other states have: row groups of a captured run, bf16 heads of 128
(the oracle given the memory as held)."""
import numpy as np
import pytest

import rlt_inputs as ri
from tests.rlt_testlib import tol_for
from tests.test_beam_state_gpu import BASE, _memory, _model, _tokens, sd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(), dict(dtype=ri.DT_BF16), dict(dtype=ri.DT_BF16, groups=1),
                                dict(variant=2, chunk=4, dtype=ri.DT_BF16)])
@pytest.mark.parametrize("rows", [512, 1024, 1300])
def test_row_groups_of_a_captured_run(sd, kw, rows):  # noqa: F811
    """Concurrent branches, each over a range of the rows: bit for bit what one chain gives."""
    import torch
    cfg = BASE.replace(**kw)
    model, _ = _model(sd, cfg)
    tok = _tokens(cfg, rows, 70)
    got = []
    for stream in (None, torch.cuda.Stream()):
        st = sd.State(model, rows, 80, mem8=True)
        st.encode(tok[:, :5].copy(), stream=stream)
        st.prefill(5, stream=stream)
        st.reset(np.arange(0, rows, 3, dtype=np.int32), stream=stream)      # a third of them at the start again
        st.encode(tok[:, 5:].copy(), stream=stream)
        st.prefill(64, stream=stream)
        out = np.zeros((rows, cfg.vocab), np.float32)
        st.readout(logits=out, stream=stream)
        st.check()
        got.append(out)
    assert np.isfinite(got[0]).all() and np.array_equal(*got)


@pytest.mark.parametrize("kw,T", [(dict(dtype=ri.DT_BF16, d=256, heads=2), 40), (dict(dtype=ri.DT_BF16, d=256, heads=2, groups=1), 20),
                                  (dict(dtype=ri.DT_BF16, d=128, heads=1, variant=2, chunk=8), 33),
                                  (dict(dtype=ri.DT_BF16, d=128, heads=1, variant=0), 40)])
def test_bf16_transitions_with_heads_of_128(sd, kw, T):  # noqa: F811
    """The oracle, given the memory as the library holds it, reads out the same logits."""
    cfg = BASE.replace(**kw)
    model, oracle = _model(sd, cfg)
    st = sd.State(model, 2, T + 30, mem8=True)
    tok = _tokens(cfg, 2, T + 3)
    st.encode(tok)
    mem, _ = _memory(sd, st, cfg)
    st.prefill(T)
    got = np.zeros((2, cfg.vocab), np.float32)
    st.readout(logits=got)
    st.check()
    for b in range(2):
        row = oracle.new_state()
        oracle.encode(row, tok[b])
        for g in range(cfg.groups):
            row.mem_k[g], row.mem_v[g] = (mem[g, b, w][:, :T + 3].transpose(1, 0, 2) for w in (0, 1))
        oracle.prefill(row, T)
        err = np.abs(got[b] - oracle.readout(row))
        assert (err <= tol_for(cfg)).all(), (b, err.max())
