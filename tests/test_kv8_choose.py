"""The choice of blocks by their keys (csrc/kv8_choose.cuh) on the host, under
schedules of the CTA's warps that a GPU rarely takes (tests/c/choose_host.cpp):
the list is the same whichever warp runs ahead, and nothing beside it is written."""
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FORCED = 0xFFFFFFFF
SCHEDULES = {"low": 0, "high": 1, "mixed": 2}
TORN = 3


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    out = str(tmp_path_factory.mktemp("choose") / "choose_host")
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wno-unknown-pragmas",
                    "-I", os.path.join(ROOT, "block_quantized_gemv_nt_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "c", "choose_host.cpp"), "-o", out], check=True)
    return out


def _want(keys, n_sel):
    order = np.lexsort((np.arange(len(keys)), -keys.astype(np.int64)))
    return np.sort(order[:n_sel])


def _run(exe, cases):
    """cases: (threads, K, n_sel, n_first, n_last, keys, schedule, seed)."""
    text = "".join("%d %d %d %d %d %d %d %d\n%s\n" % (t, K, ns, a, b, len(k), s, seed, " ".join(map(str, k)))
                   for t, K, ns, a, b, k, s, seed in cases)
    r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-200:] + r.stderr
    lines = r.stdout.splitlines()
    assert len(lines) == len(cases)
    for (t, K, ns, a, b, keys, s, seed), line in zip(cases, lines):
        got = np.array(line.split(), dtype=np.int64)
        where = (t, K, ns, a, b, len(keys), s, seed)
        assert got[-1] == 0, ("written beside the list", where)
        if s != TORN:
            assert np.array_equal(got[:-1], _want(keys, ns)), where


def _keys(rng, blocks, kind, first=0, last=0):
    if kind == "spread":      # all bits differ: four rounds, the short list from the second
        k = rng.integers(1, 2 ** 32 - 2, size=blocks, dtype=np.uint64)
    elif kind == "scores":    # order keys of floats around a common size
        k = np.abs(rng.normal(size=blocks)).astype(np.float32).view(np.uint32).astype(np.uint64) | 0x80000000
    elif kind == "ties":      # few values: a whole bin is more than the threads
        k = rng.integers(5, 9, size=blocks).astype(np.uint64) << 20
    else:                     # one value: no round at all
        k = np.full(blocks, 12345, np.uint64)
    k = k.astype(np.uint32)
    k[:first] = FORCED
    k[blocks - last:] = FORCED
    return k


@pytest.mark.parametrize("schedule", list(SCHEDULES))
@pytest.mark.parametrize("K,blocks", [(1, 300), (1, 1024), (5, 1025), (5, 5000), (0, 5121), (0, 9001), (0, 17409)])
def test_choice_is_the_same_under_every_schedule(exe, K, blocks, schedule):
    rng = np.random.default_rng(blocks)
    cases = []
    for kind in ("spread", "scores", "ties", "one"):
        for n_sel, first, last in ((1, 0, 0), (37, 1, 4), (blocks // 2, 0, 1), (blocks - 1, 2, 1)):
            if blocks > 6000 and (n_sel == 1 or kind == "one"):
                continue
            cases.append((1024, K, n_sel, first, last, _keys(rng, blocks, kind, first, last), SCHEDULES[schedule],
                          len(cases)))
    cases.append((1024, K, 8, 3, 5, _keys(rng, blocks, "spread", 3, 5), SCHEDULES[schedule], 99))  # all forced
    _run(exe, cases)


@pytest.mark.parametrize("schedule", list(SCHEDULES))
def test_counting_choice(exe, schedule):
    """Up to 256 blocks: each thread counts the keys before its own."""
    rng = np.random.default_rng(3)
    cases = []
    for blocks in (2, 3, 65, 130, 253, 256):
        for kind in ("spread", "ties", "one"):
            for n_sel in {1, blocks // 2, blocks - 1}:
                cases.append((256, -1, n_sel, 0, 0, _keys(rng, blocks, kind), SCHEDULES[schedule], len(cases)))
    _run(exe, cases)


def test_changing_keys_write_nothing_beside_the_list(exe):
    """Keys in scratch that another call overwrites meanwhile (calls that share a context's scratch must not overlap, but
    one that does may not write over the caller's memory)."""
    rng = np.random.default_rng(4)
    cases = []
    for blocks in (1500, 5000):
        for kind in ("spread", "scores", "ties"):
            for n_sel, first, last in ((1, 0, 0), (37, 1, 4), (blocks // 2, 0, 1), (blocks - 1, 2, 1)):
                cases.append((1024, 0, n_sel, first, last, _keys(rng, blocks, kind, first, last), TORN, len(cases)))
    _run(exe, cases)
