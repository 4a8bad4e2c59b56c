"""Host checks of device addresses, without a device: a preloaded library answers for the runtime that
every address is device memory, and refuses the device itself, so that nothing is ever launched (a call that
passes its checks returns RLT_E_DEVICE)."""
import json
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FAKE = """
int cudaPointerGetAttributes(int *a, const void *p) { a[0] = 2; a[1] = 0; return 0; }  /* device memory */
int cudaGetDevice(int *d) { *d = -1; return 100; }                                      /* no device */
int cudaSetDevice(int d) { return 100; }
int cudaGetLastError(void) { return 0; }
"""

CHILD = r"""
import ctypes, json, sys
import numpy as np
import stateful_decoding_b200 as sd

raw = np.zeros((1 << 16) + 16, np.uint8)
at = raw.ctypes.data + -raw.ctypes.data % 16
cache = sd.rlt_cache8(at, at, at, None, 4, 2, 2, 16, 2, 64)
ref = ctypes.byref(cache)
append = lambda start=at, counts=at, n=1: sd._lib.rlt_cache8_append(
    ref, 0, at, 128, 128, at, 128, 128, start, counts, n, None, None)
attend = lambda lens=at: sd._lib.rlt_cache8_attend(ref, 0, at, 128, 128, at, 128, 128, 2, 1, lens, 0.125, None, None)
cache.rows, cache.table = 0, None
got = {"append no rows": append(), "attend no rows": attend()}
cache.rows = 2
got.update({"append no table": append(), "attend no table": attend()})
cache.table = at
got |= {"append": append(), "append all": append(counts=None), "attend": attend()}
for off in (1, 2, 3, 4, 6):
    got["start %d" % off] = append(start=at + off)
    got["counts %d" % off] = append(counts=at + off)
    got["lens %d" % off] = attend(lens=at + off)
print(json.dumps(got))
"""


@pytest.fixture(scope="module")
def answers(tmp_path_factory):
    from tests.conftest import build_library
    build_library()
    d = tmp_path_factory.mktemp("fake")
    (d / "fake.c").write_text(FAKE)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(d / "fake.so"), str(d / "fake.c")], check=True)
    env = dict(os.environ, LD_PRELOAD=str(d / "fake.so"), PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, cwd=ROOT, env=env, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    return json.loads(r.stdout.strip().splitlines()[-1])


RLT_E_ARG, RLT_E_DEVICE = -1, -6


def test_aligned_addresses_pass(answers):
    for name in ("append", "append all", "attend", "start 4", "counts 4", "lens 4"):
        assert answers[name] == RLT_E_DEVICE, name


@pytest.mark.parametrize("what", ["start", "counts", "lens"])
def test_lengths_off_four_bytes_are_refused(answers, what):
    for off in (1, 2, 3, 6):
        assert answers["%s %d" % (what, off)] == RLT_E_ARG, (what, off)


def test_no_rows_need_no_table(answers):
    """A call for 0 rows does nothing; an empty table has no address."""
    assert answers["append no rows"] == answers["attend no rows"] == 0
    assert answers["append no table"] == answers["attend no table"] == RLT_E_ARG
