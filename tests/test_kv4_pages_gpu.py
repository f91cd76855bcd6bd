"""Block tables, slots and positions built on the GPU (nt_kv4_pages) against the
sequential oracle (kv4_ref.pages_step)."""
import numpy as np
import pytest

import kv4_ref as ref
from gpu_util import dev, host, need_gpu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from block_quantized_gemv_nt_gb300 import engine, nt  # noqa: E402


@pytest.fixture(scope="module")
def ctx():
    need_gpu()
    c = nt.Context(0)
    yield c
    c.close()


class Tables:
    """The device's tables and the oracle's beside them."""

    def __init__(self, ctx, R, W, n_pages, seed=0):
        self.ctx, self.R, self.W, self.P = ctx, R, W, n_pages
        rng = np.random.default_rng(seed)
        self.free = rng.permutation(n_pages).tolist()
        self.n_free, self.held, self.table = n_pages, [0] * R, [[0] * W for _ in range(R)]
        self.pages = engine.KV4Pages(ctx, R, W, n_pages)
        self.pages.free.copy_(torch.tensor(self.free, dtype=torch.int32))

    def step(self, new, keep=None, n_tok=None, wrong=False, in_place=True):
        n_tok = sum(max(0, n) for n in new) if n_tok is None else n_tok
        q_start = torch.full((self.R + 1,), -9, dtype=torch.int32, device="cuda")
        slots = torch.full((n_tok + 1,), -9, dtype=torch.int64, device="cuda")
        positions = torch.full((n_tok + 1,), -9, dtype=torch.int32, device="cuda")
        kw = {}
        if not in_place:
            kw = dict(held_out=torch.empty_like(self.pages.held), n_free_out=torch.empty_like(self.pages.n_free))
        self.pages.step(dev(np.array(new, dtype=np.int32)), q_start, slots[:n_tok], positions[:n_tok],
                        keep=None if keep is None else dev(np.array(keep, dtype=np.int32)), **kw)
        before = list(self.held), self.n_free
        self.n_free, *want, was_wrong = ref.pages_step(self.table, self.held, keep, new, self.free, self.n_free, self.P, n_tok)
        assert was_wrong == wrong
        if wrong:
            with pytest.raises(nt.NtError, match="length"):
                self.ctx.sync()
        self.ctx.sync()
        if not in_place:
            assert (host(self.pages.held).tolist(), int(self.pages.n_free)) == before
            self.pages.held.copy_(kw["held_out"])
            self.pages.n_free.copy_(kw["n_free_out"])
        assert host(self.pages.held).tolist() == self.held
        assert int(self.pages.n_free) == self.n_free
        assert host(self.pages.table).tolist() == self.table
        assert host(self.pages.free).tolist() == self.free
        for got, w in zip((q_start, slots[:n_tok], positions[:n_tok]), want):
            assert host(got).tolist() == w
        assert int(slots[n_tok]) == -9 and int(positions[n_tok]) == -9


@pytest.mark.parametrize("R", [1, 2, 31, 33, 255, 257, 1000, 1024])
def test_requests_that_come_and_go(ctx, R):
    rng = np.random.default_rng(R)
    t = Tables(ctx, R, 9, 4 * R + 9, seed=R)
    for i in range(6):
        keep, new = [], []
        for h in t.held:
            kind = rng.integers(0, 5)
            k = 0 if kind == 0 else max(0, h - int(rng.integers(0, 130))) if kind == 1 else h
            n = int(rng.integers(0, 3 if kind < 3 else 150))
            keep.append(k)
            new.append(min(n, 9 * 64 - k))
        pages = sum(-(-(a + b) // 64) for a, b in zip(keep, new))
        if pages > t.P:
            new = [min(n, 1) for n in new]
            keep = [min(k, 64) for k in keep]
        t.step(new, keep, n_tok=sum(new) + int(rng.integers(0, 70)), in_place=bool(i % 2))


@pytest.mark.parametrize("n", [1, 63, 64, 65, 128, 5000, 40000])
def test_one_prompt_then_tokens(ctx, n):
    t = Tables(ctx, 3, 1 + (n + 70) // 64, 6 + n // 64)
    t.step([0, n, 0])
    t.step([1, 1, 0])
    t.step([1, 1, 1])
    t.step([0, 0, 0], keep=[0, 1, 1])     # without rows: pages go back
    t.step([0, 3, 0], n_tok=11)


def test_pages_given_back_are_taken_in_the_same_step(ctx):
    t = Tables(ctx, 4, 4, 8)
    t.step([256, 200, 0, 0])
    t.step([0, 0, 256, 130], keep=[0, 10, 0, 0])
    assert t.n_free == 0


@pytest.mark.parametrize("n_tok", [4095, 4096, 4097, 9000])
def test_few_and_many_rows(ctx, n_tok):
    """Either side of the number of rows from which a launch of their own writes them; some requests refused, some
    cut off by n_tok, some giving pages back."""
    t = Tables(ctx, 40, 60, 300, seed=n_tok)
    t.step([200] * 20 + [0] * 10 + [64] * 10, n_tok=n_tok, wrong=n_tok < 4640)
    t.step([1, 500] * 20, keep=[0 if i % 5 == 0 else h for i, h in enumerate(t.held)], n_tok=n_tok, wrong=True)
    t.step([0] * 40, keep=[h // 2 for h in t.held], n_tok=n_tok)
    t.step([2] * 39 + [5000], n_tok=n_tok, wrong=True)


def test_too_few_pages(ctx):
    """A request that the stack cannot serve, and the growing ones behind it, are refused; one that needs no page is not."""
    t = Tables(ctx, 5, 8, 6)
    t.step([60, 60, 60, 60, 60])
    t.step([4, 100, 1, 4, 100], wrong=True)
    assert t.held == [64, 60, 61, 64, 60] and t.n_free == 1
    t.step([0, 1, 1, 64, 1])              # request 3 takes the last page
    t.step([1, 1, 1, 1, 1], keep=[64, 61, 62, 10, 61], wrong=False)


@pytest.mark.parametrize("keep,new", [([0, 11, 0], [1, 1, 1]), ([0, -1, 0], [1, 1, 1]), ([0, 10, 0], [1, -3, 1]),
                                      ([0, 10, 0], [1, 300, 1]), ([0, 10, 0], [1, 2 ** 31 - 1, 1])])
def test_lengths_refused_one_by_one(ctx, keep, new):
    t = Tables(ctx, 3, 4, 12)
    t.step([0, 10, 0])
    t.step(new, keep, n_tok=min(310, sum(max(0, n) for n in new)), wrong=True)
    assert t.held == [1, 10, 1]
    t.step([1, 1, 1])


def test_more_rows_than_room(ctx):
    t = Tables(ctx, 3, 4, 12)
    t.step([3, 4, 5], n_tok=6, wrong=True)
    t.step([1, 0, 1], n_tok=0, wrong=True)


def test_lengths_that_the_tables_cannot_hold(ctx):
    t = Tables(ctx, 2, 4, 12)
    t.step([5, 5])
    t.pages.held.copy_(torch.tensor([-1, 257], dtype=torch.int32))
    t.held = [-1, 257]
    t.step([1, 1], wrong=True)


def test_stack_out_of_range(ctx):
    """A stack size that is no stack size is held to the stack; nothing is written outside it."""
    for wrong in (-3, 10, 2 ** 31 - 1):
        room = torch.full((9,), 77, dtype=torch.int32, device="cuda")
        p = engine.KV4Pages(ctx, 1, 4, 7, buffers=dict(
            table=torch.zeros(1, 4, dtype=torch.int32, device="cuda"), held=torch.tensor([200], dtype=torch.int32, device="cuda"),
            free=room[1:8], n_free=torch.tensor([wrong], dtype=torch.int32, device="cuda")))
        i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        p.step(i32(0), i32(0, 0), torch.zeros(0, dtype=torch.int64, device="cuda"), i32(), keep=i32(0))
        with pytest.raises(nt.NtError):
            ctx.sync()
        assert host(room)[[0, 8]].tolist() == [77, 77] and 0 <= int(p.n_free) <= 7


def test_captured_with_many_rows(ctx):
    """The two launches of a step with many rows, captured and replayed."""
    t = Tables(ctx, 9, 80, 400, seed=6)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    n_tok = 6000
    new, keep, q_start, slots, positions = i32(9), i32(9), i32(10), torch.zeros(n_tok, dtype=torch.int64, device="cuda"), i32(n_tok)
    t.pages.step(new, q_start, slots, positions, keep=keep)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.pages.step(new, q_start, slots, positions, keep=keep)
    rng = np.random.default_rng(7)
    for _ in range(30):
        ks = [h if rng.random() < 0.7 else int(rng.integers(0, h + 1)) for h in t.held]
        ns = [int(x) for x in rng.integers(0, 600, 9)]
        new.copy_(torch.tensor(ns, dtype=torch.int32))
        keep.copy_(torch.tensor(ks, dtype=torch.int32))
        graph.replay()
        t.n_free, *want, wrong = ref.pages_step(t.table, t.held, ks, ns, t.free, t.n_free, 400, n_tok)
        for got, w in zip((q_start, slots, positions), want):
            assert host(got).tolist() == w
        assert host(t.pages.table).tolist() == t.table and host(t.pages.held).tolist() == t.held
        assert int(t.pages.n_free) == t.n_free
        if wrong:
            with pytest.raises(nt.NtError):
                ctx.sync()
    ctx.sync()


def test_captured(ctx):
    """One captured step, replayed: the lengths are the device's."""
    t = Tables(ctx, 40, 5, 150, seed=3)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    new, q_start, slots, positions = i32(40), i32(41), torch.zeros(90, dtype=torch.int64, device="cuda"), i32(90)
    t.pages.step(new, q_start, slots, positions)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.pages.step(new, q_start, slots, positions)
    rng = np.random.default_rng(4)
    for _ in range(50):
        ns = [int(x) for x in rng.integers(0, 3, 40)]
        new.copy_(torch.tensor(ns, dtype=torch.int32))
        graph.replay()
        t.n_free, *want, wrong = ref.pages_step(t.table, t.held, None, ns, t.free, t.n_free, 150, 90)
        assert not wrong
        for got, w in zip((q_start, slots, positions), want):
            assert host(got).tolist() == w
        assert host(t.pages.table).tolist() == t.table and host(t.pages.held).tolist() == t.held
    ctx.sync()


def test_refusals(ctx):
    t = Tables(ctx, 2, 4, 9)
    p = t.pages
    i32 = torch.zeros(8, dtype=torch.int32, device="cuda")
    s = torch.zeros(4, dtype=torch.int64, device="cuda")
    good = dict(n_req=2, table=p.table, max_pages=4, held=p.held, keep=None, n_new=i32, free=p.free, n_pages=9,
                n_free=p.n_free, held_out=p.held, n_free_out=p.n_free, q_start=i32, slots=s, positions=i32, n_tok=4)
    bad = [dict(n_req=0), dict(n_req=1025), dict(max_pages=0), dict(max_pages=(1 << 24) + 1), dict(n_pages=0),
           dict(n_pages=(1 << 26) + 1), dict(n_tok=-1), dict(n_tok=1 << 26), dict(slots=s.data_ptr() + 4)]
    bad += [{n: None} for n in good if n not in ("n_req", "max_pages", "keep", "n_pages", "n_tok", "table")]
    bad += [{n: i32.data_ptr() + 2} for n in ("held", "keep", "n_new", "q_start", "positions")]
    for kw in bad:
        with pytest.raises(nt.NtError) as e:
            nt.nt_kv4_pages(ctx, **{**good, **kw})
        assert e.value.status in (nt.NT_ERR_INVALID_ARG, nt.NT_ERR_ALIGNMENT), kw
    with pytest.raises(nt.NtError):
        nt.nt_kv4_pages(ctx, **{**good, "table": None}, stream=0)
