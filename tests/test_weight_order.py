"""Which streams count as having unfinished weight writes: the host's table behind
the early weight loads of the GEMV, shared-expert and batch-1 layer kernels."""
import ctypes
import subprocess
import sys

from conftest import ROOT
from mxfp4_routed_expert_select_gb300 import k3moe as k


def _table():
    L = ctypes.CDLL(k.SO)
    note, take = L._ZN2k312written_noteEmy, L._ZN2k312written_takeEmy
    for f in (note, take):
        f.argtypes = [ctypes.c_ulong, ctypes.c_ulonglong]
    note.restype, take.restype = None, ctypes.c_bool
    return note, take


def test_a_mark_goes_with_the_first_taker():
    note, take = _table()
    assert not take(0x1000, 0)
    note(0x1000, 0)
    note(0x1000, 0)
    note(0x2000, 0)
    note(0, 0)  # the legacy default stream
    assert not take(0x3000, 0)
    assert take(0x1000, 0) and not take(0x1000, 0)
    assert take(0x2000, 0) and not take(0x2000, 0)
    assert take(0, 0) and not take(0, 0)


def test_the_per_thread_default_stream_stays_marked():
    note, take = _table()
    note(2, 0)  # one handle for the streams of all threads
    assert take(2, 0) and take(2, 0)


def test_a_capture_keeps_its_mark_and_leaves_the_streams_alone():
    note, take = _table()
    note(0x5000, 71)
    assert take(0x5000, 71) and take(0x5000, 71) and take(0x6000, 71)
    assert not take(0x5000, 0) and not take(0x5000, 72)
    note(0x5000, 0)
    assert take(0x5000, 71) and not take(0x5000, 73) and take(0x5000, 0)


_FULL = """
import sys
sys.path.insert(0, %r)
from test_weight_order import _table
note, take = _table()
for i in range(1, 1000):  # more captures than are remembered: old ones count as marked
    note(8, 10 * i)
    assert take(8, 10 * i) and not take(8, 10 * i + 1)
assert all(take(8, 10 * i) for i in range(1, 1000))
assert not take(8, 0)
for i in range(1, 257):
    note(0x100 * i, 0)
assert not take(8, 0)
for i in range(256, 0, -1):
    assert take(0x100 * i, 0)
for i in range(1, 257):
    assert not take(0x100 * i, 0)
for i in range(1, 258):  # more streams than the table holds: from then on all are marked
    note(0x100 * i, 0)
assert all(take(0x100 * i, 0) for i in range(1, 400)) and take(8, 0)
print("ok")
"""


def test_full_tables_err_on_the_safe_side():
    r = subprocess.run([sys.executable, "-c", _FULL % (ROOT + "/tests")], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr
