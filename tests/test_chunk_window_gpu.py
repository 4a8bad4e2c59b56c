"""RLT-2 chunks at least as long as the decoder's window, bf16: the block's first keys are outside
its last queries' windows, and the ring's outside most."""
import numpy as np
import pytest

import rlt_inputs as ri
from oracle.rlt_oracle import RLTOracle
from tests.rlt_testlib import TOL_BF16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("chunk,window,heads", [(16, 8, 2), (8, 8, 2), (16, 8, 1), (5, 2, 2)])
def test_chunks_longer_than_the_window(chunk, window, heads):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tests.conftest import build_library
    build_library()
    import stateful_decoding_b200 as sd
    cfg = ri.RLTConfig("small", vocab=40, d=128, heads=heads, n_enc=2, n_dec=2, ffn=256, window=window, groups=2,
                       chunk=chunk, variant=2, dtype=ri.DT_BF16)
    blob = ri.write_blob(cfg, ri.generate_weights(cfg, seed=7), seed=7)
    oracle = RLTOracle(cfg, ri.read_blob(blob)[1], "bf16")
    tok = np.random.default_rng(1).integers(0, cfg.vocab, (2, 40)).astype(np.int32)
    st = sd.State(sd.Model(blob), 2, 64)
    st.encode(tok)
    st.prefill(40)
    got = np.zeros((2, cfg.vocab), np.float32)
    st.readout(logits=got)
    st.check()
    for b in range(2):
        row = oracle.new_state()
        oracle.encode(row, tok[b])
        oracle.prefill(row, 40, chunked=True)
        assert np.abs(got[b] - oracle.readout(row)).max() <= TOL_BF16
