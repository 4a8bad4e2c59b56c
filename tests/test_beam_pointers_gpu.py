"""The arrays of a state's beam calls: on the model's device and on four bytes, else RLT_E_ARG before
anything runs."""
import json
import os
import subprocess
import sys

import numpy as np
import pytest

import rlt_inputs as ri
from tests.test_beam_state_gpu import BASE, _model, _tokens, sd  # noqa: F401

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_arrays_off_four_bytes_are_refused(sd):  # noqa: F811
    import torch
    model, _ = _model(sd, BASE)
    st = sd.State(model, 4, 16)
    st.encode(_tokens(BASE, 4, 3))
    st.prefill(3)
    before = st.read(sd.PART_S).copy()
    buf = torch.zeros(4, 64, dtype=torch.uint8, device="cuda")
    at = [b.data_ptr() for b in buf]
    step = lambda a: sd._lib.rlt_beam_step(st.handle, a[0], a[1], 2, 1.0, 2, 0, a[2], a[3], None)  # noqa: E731
    for off in (1, 2, 3):
        assert sd._lib.rlt_state_reorder(st.handle, at[0] + off, 2, 0, None) == sd.RLT_E_ARG
        for i in (0, 2, 3):
            a = list(at)
            a[i] += off
            assert step(a) == sd.RLT_E_ARG, (i, off)
    torch.cuda.synchronize()
    assert np.array_equal(st.read(sd.PART_S), before) and [p.tolist() for p in st.positions()] == [[3] * 4] * 2
    assert not buf.any()
    assert step([at[0], at[1] + 1, at[2], at[3]]) == 0          # one byte a row: anywhere
    assert sd._lib.rlt_state_reorder(st.handle, at[2] + 4, 2, 0, None) == 0
    torch.cuda.synchronize()


FAKE = r"""
#define _GNU_SOURCE
#include <dlfcn.h>
#include <stdlib.h>
/* device memory is said to be on the next device */
int cudaPointerGetAttributes(int *a, const void *p) {
    static int (*real)(int *, const void *);
    if (!real) real = (int (*)(int *, const void *))dlsym(RTLD_NEXT, "cudaPointerGetAttributes");
    int rc = real ? real(a, p) : 1;
    if (rc == 0 && a[0] == 2) a[1] += 1;
    return rc;
}
"""

CHILD = r"""
import json
import numpy as np, torch
import rlt_inputs as ri
import stateful_decoding_b200 as sd
from tests.test_beam_state_gpu import BASE
st = sd.State(sd.Model(ri.write_blob(BASE, ri.generate_weights(BASE, seed=7, std=0.02), seed=7)), 4, 16)
i32 = lambda: torch.zeros(4, dtype=torch.int32, device="cuda")
scores = torch.zeros(4, device="cuda")
got = [int(sd.rlt_beam_step(st.handle, scores, None, -1, 1.0, 2, 0, i32(), i32())),
       int(sd.rlt_state_reorder(st.handle, i32(), 2)),
       int(sd.rlt_state_reorder(st.handle, np.zeros(4, np.int32), 2))]
torch.cuda.synchronize()
print(json.dumps(got))
"""


def test_arrays_of_another_device_are_refused(sd, tmp_path):  # noqa: F811
    (tmp_path / "fake.c").write_text(FAKE)
    so = str(tmp_path / "fake.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", so, str(tmp_path / "fake.c"), "-ldl"], check=True)
    env = dict(os.environ, LD_PRELOAD=so, PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, cwd=ROOT, env=env, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert json.loads(r.stdout.strip().splitlines()[-1]) == [-1, -1, 0]
