"""Pins of the 64-bit oracle of the 8-bit KV cache (kv8_ref), and what the
binding and its cache class refuse without a GPU."""
import ctypes
import math

import numpy as np
import pytest

import kv8_ref as ref

torch = pytest.importorskip("torch")


def test_e4m3_table_is_the_format():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    ok = ~np.isnan(t)
    assert ok.sum() == 254
    assert np.array_equal(t[ok], ref.E4M3_VALUES[ok])


@pytest.mark.parametrize("fmt", [ref.I8, ref.E4M3])
def test_rounding_is_nearest_even(fmt):
    grid = np.unique(ref.E4M3_VALUES[:127]) if fmt == ref.E4M3 else np.arange(0.0, 128.0)
    mid = (grid[1:] + grid[:-1]) / 2
    # a tie goes to the neighbour with an even last bit: every second grid value
    even = np.where(np.arange(len(mid)) % 2 == 0, grid[:-1], grid[1:])
    for s in (1.0, -1.0):
        assert np.array_equal(ref.round8(s * mid, fmt), s * even)
        assert np.array_equal(ref.round8(s * np.nextafter(mid, 0), fmt), s * grid[:-1])
        assert np.array_equal(ref.round8(s * np.nextafter(mid, 1e9), fmt), s * grid[1:])
        assert np.array_equal(ref.to_values(ref.to_bytes(s * grid, fmt), fmt), s * grid)
    if fmt == ref.E4M3:
        x = np.random.default_rng(0).normal(size=4000) * 30
        want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy()
        assert np.array_equal(ref.round8(x.astype(np.float32).astype(np.float64), fmt), want)


@pytest.mark.parametrize("qmax", [127.0, 448.0, 2047.0])
def test_scale_is_the_least_power_of_two(qmax):
    for a in [0.0, 1e-38, 127.0 * 2.0 ** -100, 1.0, qmax, np.nextafter(qmax, 1e9), 3.3e38, qmax * 2.0 ** 7]:
        t = ref.scale_for(a, qmax)
        assert a <= qmax * t and math.frexp(t)[0] == 0.5 and t >= 2.0 ** -100
        assert t == 2.0 ** -100 or a > qmax * t / 2


@pytest.mark.parametrize("fmt", [ref.I8, ref.E4M3])
def test_cache_error_is_half_a_step(fmt):
    """Rows written at once: |value - x| <= half a step of the block's scale (I8), or of the value (E4M3: 2^-4 of
    it, and half the smallest subnormal)."""
    rng = np.random.default_rng(1)
    c = ref.Cache(fmt, 2, 64, 200)
    k, v = rng.normal(size=(150, 2, 64)) * 5, rng.normal(size=(150, 2, 64))
    c.append(k, v, 0)
    for w, x in (("k", k), ("v", v)):
        got = c.read(w, np.arange(150))
        t = c.scale[w][:, np.arange(150) // 64][..., None]
        half = t / 2 if fmt == ref.I8 else np.maximum(np.abs(x.transpose(1, 0, 2)) * 2.0 ** -4, t * 2.0 ** -10)
        assert np.all(np.abs(got - x.transpose(1, 0, 2)) <= half)


def test_token_by_token_keeps_the_scale_rule():
    """A block written token by token ends at the scale of the rows written at once."""
    rng = np.random.default_rng(2)
    x = rng.normal(size=(100, 1, 64)) * np.linspace(0.1, 9, 100)[:, None, None]
    a, b = ref.Cache(ref.I8, 1, 64, 100), ref.Cache(ref.I8, 1, 64, 100)
    a.append(x, x, 0)
    for i in range(100):
        b.append(x[i:i + 1], x[i:i + 1], i)
    assert np.array_equal(a.scale["k"], b.scale["k"])
    at = np.arange(100)
    t = a.scale["k"][:, at // 64][..., None]
    # each of at most log2 growths of the scale adds half a step of the scale it goes to: less than one step in all
    assert np.all(np.abs(a.read("k", at) - b.read("k", at)) <= 1.0 * t)


def test_selection_bound_holds():
    """Up to q's rounding the score bounds sum_h q_h . k of every key of the block."""
    rng = np.random.default_rng(3)
    for fmt in (ref.I8, ref.E4M3):
        c = ref.Cache(fmt, 1, 64, 64 * 9)
        x = rng.normal(size=(64 * 9, 1, 64))
        c.append(x, x, 0)
        unit = 1.0 if fmt == ref.I8 else 4.0
        k = c.read("k", np.arange(64 * 9))[0].reshape(9, 64, 64)
        q = rng.integers(-2047, 2048, size=(3, 64)).astype(np.float64)
        lo, hi = c.kmin[0] * unit * c.scale["k"][0][:, None], c.kmax[0] * unit * c.scale["k"][0][:, None]
        bound = np.maximum(q[:, None] * lo, q[:, None] * hi).sum(axis=(0, 2))
        assert np.all((k @ q.T).sum(axis=2).max(axis=1) <= bound + 1e-6)


def test_empty_attention_is_zero():
    out, tol = ref.attend(np.ones((2, 64)), np.zeros((0, 64)), np.zeros((0, 64)))
    assert not out.any() and not tol.any()


def test_struct_layout_matches_c(tmp_path):
    """The binding's nt_kv8 has the C compiler's size and offsets."""
    import os
    import shutil
    import subprocess
    from block_quantized_gemv_nt_gb300 import nt
    gcc = shutil.which("gcc")
    if not gcc:
        pytest.skip("no C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = [f[0] for f in nt.nt_kv8._fields_]
    src = tmp_path / "s.c"
    src.write_text('#include "nt.h"\n#include <stdio.h>\nint main(void){printf("%zu", sizeof(nt_kv8));' +
                   "".join(f'printf(" %zu", offsetof(nt_kv8, {n}));' for n in names) + "return 0;}\n")
    subprocess.run([gcc, "-std=c99", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "s")],
                   check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "s")], capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(nt.nt_kv8)] + [getattr(nt.nt_kv8, n).offset for n in names]


def test_cache_class_refuses_ill_shaped_tensors():
    from block_quantized_gemv_nt_gb300 import engine, nt
    c = engine.KV8Cache(None, nt.KV8_I8, 2, 64, 100, device="cpu")
    f = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt)  # noqa: E731
    with pytest.raises(ValueError):
        engine.KV8Cache(None, nt.KV8_I8, 2, 64, 100, buffers=dict(c.buffers, k=f(2, 100, 64)))
    bad = [lambda: c.append(f(1, 3, 64), f(1, 3, 64), 0), lambda: c.append(f(1, 2, 64), f(2, 2, 64), 0),
           lambda: c.append(f(1, 2, 64, dt=torch.float64), f(1, 2, 64, dt=torch.float64), 0),
           lambda: c.append(f(1, 64, 2).transpose(1, 2), f(1, 64, 2).transpose(1, 2), 0),
           lambda: c.read(0, f(2, 64, 5).transpose(1, 2), f(2, 64, 5).transpose(1, 2)),
           lambda: c.read(0, f(2, 10, 64)[:, ::2], f(2, 10, 64)[:, ::2]),
           lambda: c.attend(f(1, 4, 128), f(1, 4, 128), 5), lambda: c.attend(f(1, 4, 64), f(1, 2, 64), 5),
           lambda: c.attend(f(1, 64, 4).transpose(1, 2), f(1, 4, 64), 5),
           lambda: c.select(f(1, 4, 64), torch.zeros(1, 2, 8), 5),
           lambda: c.attend_blocks(f(1, 4, 64), f(1, 4, 64), 5, torch.zeros(2, 2, 8, dtype=torch.int32))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
