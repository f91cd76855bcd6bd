"""The calls over the paged 4-bit cache let other Python threads run while the library
works (a launch waits where a stream's queue is full).  CPU: a stand-in for the
library's entry points, found before it, sleeps."""
import os
import subprocess
import sys

import pytest

from conftest import ROOT

pytest.importorskip("torch")

STAND_IN = "#include <unistd.h>\n" + "".join(
    f"int {name}(void) {{ usleep(400000); return 0; }}\n"
    for name in ("nt_kv4_pages", "nt_kv4_append", "nt_kv4_read", "nt_attn_kv4", "nt_rope_rows"))

PROGRAM = """
import ctypes, sys, threading, time
import torch
from block_quantized_gemv_nt_gb300 import nt
ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
calls = nt.load_calls()
i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)
rows, slots = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int64)
todo = {
    "append": lambda: calls.kv4_rows(False, None, None, 2, 64, -1, rows, rows, slots, None),
    "read": lambda: calls.kv4_rows(True, None, None, 2, 64, -1, rows, rows, slots, None),
    "attend": lambda: calls.attn_kv4(None, None, 64, -1, rows, rows, i32(2), i32(1), i32(1, 4), None),
    "pages": lambda: calls.kv4_pages(None, -1, i32(1, 4), i32(1), i32(4), i32(1), i32(1), i32(2), slots, i32(3), None, None, None,
                                     None),
    "rope": lambda: calls.rope_rows(None, None, 64, -1, ((rows, rows),), None, 0, None)}
ticks, stop = [], False
def tick():
    while not stop:
        ticks.append(time.perf_counter())
        time.sleep(0.005)
t = threading.Thread(target=tick)
t.start()
for name, call in todo.items():
    t0 = time.perf_counter()
    status = call()
    t1 = time.perf_counter()
    print(name, status, t1 - t0, sum(t0 < x < t1 for x in ticks))
stop = True
t.join()
"""


def test_other_threads_run_during_a_call(tmp_path):
    src, lib = tmp_path / "stand_in.c", tmp_path / "libstandin.so"
    src.write_text(STAND_IN)
    subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    r = subprocess.run([sys.executable, "-c", PROGRAM, str(lib)], capture_output=True, text=True, cwd=ROOT, timeout=300,
                       env={**os.environ, "PYTHONPATH": ROOT})
    assert r.returncode == 0, r.stderr
    seen = [line.split() for line in r.stdout.splitlines()]
    assert [s[0] for s in seen] == ["append", "read", "attend", "pages", "rope"]
    for name, status, took, ticks in seen:
        # 0.4 s of about 80 ticks; with the lock held there is none
        assert status == "0" and float(took) >= 0.4 and int(ticks) >= 5, (name, took, ticks)
