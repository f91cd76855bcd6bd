"""What the sync after a call over the paged 4-bit cache says was wrong."""
import numpy as np
import pytest

from gpu_util import dev, need_gpu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from block_quantized_gemv_nt_gb300 import engine, nt  # noqa: E402


@pytest.fixture(scope="module")
def ctx():
    need_gpu()
    c = nt.Context(0)
    yield c
    c.close()


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _too_much(ctx, cache):
    """2^22 pages of 64 heads and one more page: 2^28 steps and 64 (the table holds no page)."""
    pages = 2 ** 22 + 1
    table = torch.full((1, pages), -1, dtype=torch.int32, device="cuda")
    q, out = torch.zeros(1, 64, 64, device="cuda"), torch.full((1, 64, 64), 7.0, device="cuda")
    cache.attend(q, out, _i32(0, 1), _i32(64 * pages), table)
    return out


def test_more_work_than_a_call_takes_is_named(ctx):
    cache = engine.KV4Cache(ctx, nt.KV4_I4, 64, 64, 1)
    out = _too_much(ctx, cache)
    with pytest.raises(nt.NtError, match="more work") as e:
        ctx.sync()
    assert e.value.status == nt.NT_ERR_INVALID_ARG and "slot" not in str(e.value)
    assert bool((out == 7.0).all())
    ctx.sync()


def test_several_causes_are_all_named(ctx):
    cache = engine.KV4Cache(ctx, nt.KV4_I4, 64, 64, 1)
    _too_much(ctx, cache)
    k = dev(np.ones((2, 64, 64), dtype=np.float32))
    k[0, 3, 5] = float("nan")
    cache.append(k, k, torch.tensor([0, 64], device="cuda"))       # the second row's slot is behind the cache
    with pytest.raises(nt.NtError) as e:
        ctx.sync()
    for part in ("more work", "slot", "4-bit"):
        assert part in str(e.value)
    ctx.sync()
