"""A launch that the library itself refuses (a grid or a cluster that the device does not take) is the
call's error, also inside a state's schedule.  The refusal is made on the host: a preloaded library
stands in for the launcher and returns cudaErrorInvalidConfiguration."""
import json
import os
import re
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import json, sys
import numpy as np
import torch
import rlt_inputs as ri
import stateful_decoding_b200 as sd

cfg = ri.RLTConfig("small", vocab=40, d=128, heads=2, n_enc=1, n_dec=2, ffn=256, window=8, groups=2,
                   chunk=1, variant=1, tied=0, dtype={"fp32": ri.DT_F32, "bf16": ri.DT_BF16}[sys.argv[1]])
model = sd.Model(ri.write_blob(cfg, ri.generate_weights(cfg, seed=7, std=0.02), seed=7))
tok = np.random.default_rng(1).integers(0, cfg.vocab, (2, 20)).astype(np.int32)
st = sd.State(model, 2, 64, mem8=True)
side = torch.cuda.Stream()
rows = torch.zeros(2, 16, dtype=torch.uint8, device="cuda")
i32 = lambda: torch.zeros(2, dtype=torch.int32, device="cuda")
lp = np.zeros((2, 20), np.float32)
calls = {
    "encode": lambda: sd.rlt_encode(st.handle, tok, 20),
    "step": lambda: sd.rlt_step(st.handle),
    "prefill": lambda: sd.rlt_prefill(st.handle, 20),
    "prefill by graph": lambda: sd.rlt_prefill(st.handle, 20, stream=side),
    "replay": lambda: sd.rlt_replay_logprobs(st.handle, tok, 20, lp, 1.0),
    "packed": lambda: sd.rlt_prefill_packed(st.handle, tok, np.eye(2, 20, dtype=np.uint8), 20),
    "reorder": lambda: sd._lib.rlt_rows_reorder(rows.data_ptr(), i32().data_ptr(), 1, 2, 16, 1, 0, 0, 16, None),
    "beam": lambda: sd.rlt_beam_step(st.handle, torch.zeros(2, device="cuda"), None, -1, 1.0, 2, 0, i32(), i32()),
}
got = {}
for name in sys.argv[2].split(","):
    code = calls[name]()
    torch.cuda.synchronize()
    got[name] = [int(code)] + [[int(x) for x in p] for p in st.positions()]
print(json.dumps(got))
"""


@pytest.fixture(scope="module")
def library():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tests.conftest import build_library
    return build_library()


def _symbol(library, pattern):
    names = subprocess.run(["nm", "-D", "--defined-only", library], capture_output=True, text=True, check=True).stdout
    found = [n for n in re.findall(r"\S+$", names, re.M) if re.search(pattern, n)]
    assert len(found) == 1, found
    return found[0]


def _run(library, tmp_path, pattern, dtype, calls, error=9):
    src, so = tmp_path / "refuse.c", tmp_path / "refuse.so"
    src.write_text('int refuse(void) __asm__("%s");\nint refuse(void) { return %d; }\n' % (
        _symbol(library, pattern), error))
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(so), str(src)], check=True)
    env = dict(os.environ, LD_PRELOAD=str(so), PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", CHILD, dtype, calls], capture_output=True, text=True, cwd=ROOT, env=env,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    return json.loads(r.stdout.strip().splitlines()[-1])


UNSUPPORTED, ARG, DEVICE = -8, -1, -6


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_a_refused_append_is_the_calls_error(library, tmp_path, dtype):
    got = _run(library, tmp_path, r"launch_cache8_appendIf", dtype, "encode,replay,packed,beam")
    for name, (code, enc, dec) in got.items():
        assert code == UNSUPPORTED, (name, code)
        assert enc == [0, 0] and dec == [0, 0], (name, enc, dec)


@pytest.mark.parametrize("dtype,pattern", [("fp32", r"launch_cache8_attendIffE"), ("bf16", r"launch_cache8_attendIf13__nv_bfloat16E")])
def test_a_refused_attention_is_the_calls_error(library, tmp_path, dtype, pattern):
    got = _run(library, tmp_path, pattern, dtype, "encode,step,prefill,prefill by graph,beam")
    assert got["encode"] == [0, [20, 20], [0, 0]]
    for name in ("step", "prefill", "prefill by graph"):
        assert got[name] == [UNSUPPORTED, [20, 20], [0, 0]], (name, got[name])
    got = _run(library, tmp_path, pattern, dtype, "beam")
    assert got["beam"][0] == UNSUPPORTED and got["beam"][2] == [0, 0], got


def test_a_refused_selection_is_the_calls_error(library, tmp_path):
    got = _run(library, tmp_path, r"launch_beam_selectIfE", "fp32", "beam")
    assert got["beam"] == [UNSUPPORTED, [0, 0], [0, 0]]


@pytest.mark.parametrize("error,code", [(400, ARG), (9, UNSUPPORTED), (719, DEVICE)])
def test_a_stream_of_another_device_is_an_argument_error(library, tmp_path, error, code):
    """The launch then fails with cudaErrorInvalidResourceHandle (400); other errors are what they were."""
    got = _run(library, tmp_path, r"14launch_reorderE", "fp32", "reorder", error)
    assert got["reorder"][0] == code
