"""What KV8Cache refuses as a position held on the device, without a GPU: the
kernels would read past an int32 tensor, and read a host address."""
import types

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def cache():
    from block_quantized_gemv_nt_gb300 import engine, nt
    c = engine.KV8Cache(None, nt.KV8_I8, 2, 64, 100, device="cpu")
    return c


def _calls(c):
    f, i = torch.zeros(1, 2, 64), torch.zeros(1, 2, 4, dtype=torch.int32)
    h = torch.zeros(2, 1, 64)
    return {"append": lambda p: c.append(f, f, 0, pos_dev=p), "append_from_heads": lambda p: c.append_from_heads(h, h, 0, pos_dev=p),
            "attend": lambda p: c.attend(f, f, 0, pos_dev=p), "select": lambda p: c.select(f, i, 0, pos_dev=p),
            "attend_blocks": lambda p: c.attend_blocks(f, f, 0, i, pos_dev=p)}


@pytest.mark.parametrize("call", ["append", "append_from_heads", "attend", "select", "attend_blocks"])
def test_bad_device_positions_are_refused(cache, call, monkeypatch):
    from block_quantized_gemv_nt_gb300 import nt
    reached = []
    for name in ("nt_kv8_append", "nt_attn_kv8", "nt_kv8_select", "nt_attn_kv8_blocks"):
        monkeypatch.setattr(nt, name, lambda *a, **k: reached.append(a))
    elsewhere = types.SimpleNamespace(dtype=torch.int64, numel=lambda: 1, get_device=lambda: 3)  # a tensor of another device
    for bad in (torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1),
                torch.zeros(0, dtype=torch.int64), elsewhere):
        with pytest.raises(ValueError, match="pos_dev"):
            _calls(cache)[call](bad)
    assert not reached
    for good in (None, torch.zeros(1, dtype=torch.int64), torch.zeros((), dtype=torch.int64), 4096):
        _calls(cache)[call](good)
    assert len(reached) == 4
    cache.index = 0  # a cache on the GPU: a position in host memory
    monkeypatch.setattr(cache, "_rows", lambda *a: (0, 1, 0, 0))
    monkeypatch.setattr(cache, "_queries", lambda *a: (1, 2))
    monkeypatch.setattr(cache, "_list", lambda *a: 4)
    with pytest.raises(ValueError, match="pos_dev"):
        _calls(cache)[call](torch.zeros(1, dtype=torch.int64))
    assert len(reached) == 4
