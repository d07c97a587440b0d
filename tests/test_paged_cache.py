"""PagedCache and PagedDecoder never hand a call more than their buffers hold,
without a GPU: the calls are replaced by checks of what they are given."""
import pytest
import torch

from int4_expert_gemv_gb300 import build as nbuild


@pytest.fixture
def paged(monkeypatch):
    nbuild.build()
    from int4_expert_gemv_gb300 import paged
    seen = []

    def plan(seq, new, R, table, max_blocks, page, ring, n_pages, pool, seq_out, first, slots, places, cap, pool_out, status, stream=None):
        assert cap <= slots.numel() and cap <= places.numel()
        assert min(seq.numel(), new.numel(), seq_out.numel()) >= R and first.numel() >= R + 1
        assert table.numel() >= R * max_blocks and ring.numel() >= n_pages
        seen.append(("plan", cap))

    def append(desc, k, v, slots, N, stream=None):
        assert N <= slots.numel() and k.shape[0] >= N and v.shape[0] >= N
        seen.append(("append", N))

    monkeypatch.setattr(paged.moe, "moe_kv_plan", plan)
    monkeypatch.setattr(paged.moe, "moe_kv_append", append)
    paged.seen = seen
    return paged


def _cache(paged, R=8, max_new=3):
    return paged.PagedCache(R, 20, 16, 2, 32, 4, max_new, device="cpu")


def test_plan_keeps_to_the_places_there_are(paged):
    ca, new = _cache(paged), torch.zeros(8, dtype=torch.int32)
    ca.plan(new)
    ca.plan(new, 2)
    ca.plan(new, 0)
    assert paged.seen == [("plan", 3), ("plan", 2), ("plan", 0)]
    for most in (4, 8, -1):
        with pytest.raises(ValueError):
            ca.plan(new, most)
    for bad in (new[:7], new.long(), torch.zeros((16,), dtype=torch.int32)[::2]):
        with pytest.raises(ValueError):
            ca.plan(bad)
    assert len(paged.seen) == 3


def test_append_keeps_to_the_slots_there_are(paged):
    ca = _cache(paged)
    ca.append(torch.zeros((3, 64)), torch.zeros((3, 64)))
    ca.append(torch.zeros((2, 2, 32)), torch.zeros((2, 64)))
    for k, v in (((4, 64), (4, 64)), ((3, 64), (2, 64)), ((2, 32), (2, 64)), ((2, 64), (2, 128))):
        with pytest.raises(ValueError):
            ca.append(torch.zeros(k), torch.zeros(v))
    assert paged.seen == [("append", 3), ("append", 2)]


def test_a_step_of_a_cache_with_fewer_places_than_requests(paged):
    """Up to its first call after the plan, and no call of more tokens."""
    from types import SimpleNamespace
    ca = _cache(paged)
    dec = object.__new__(paged.PagedDecoder)
    dec.cache, dec.cfg = ca, SimpleNamespace(d=16)
    x, new = torch.zeros((8, 16)), torch.zeros(8, dtype=torch.int32)
    with pytest.raises(AttributeError):                  # no weights here
        dec.step(x, torch.arange(3), new)
    assert paged.seen == [("plan", 3)]
    with pytest.raises(ValueError):
        dec.step(x, torch.arange(4), new)
    assert len(paged.seen) == 1


def test_plans_go_on_from_the_same_addresses(paged, monkeypatch):
    """What a captured plan repeats: every call reads and writes at the same
    places, and each goes on from the last one's state."""
    where = []

    def plan(seq, new, R, table, max_blocks, page, ring, n_pages, pool, seq_out, first, slots, places, cap, pool_out, status, stream=None):
        where.append([t.data_ptr() for t in (seq, table, ring, pool, seq_out, first, slots, places, pool_out, status)])
        seq_out.copy_(seq + new)
        pool_out.copy_(pool + torch.tensor([1, -1], dtype=torch.int32))

    monkeypatch.setattr(paged.moe, "moe_kv_plan", plan)
    ca = _cache(paged)
    new = torch.arange(8, dtype=torch.int32)
    for n in range(1, 5):
        ca.plan(new, 3)
        assert ca.seq_len.tolist() == [n * i for i in range(8)] and ca.pool.tolist() == [n, 20 - n]
    assert len(where) == 4 and all(w == where[0] for w in where) and len(set(where[0])) == 10


def test_a_plan_that_does_not_fit_is_not_forgotten(paged, monkeypatch):
    """Between others that do, and until it has been told once."""
    codes = iter([0, paged.moe.MOE_ENOSPACE, 0, 0, 0, paged.moe.MOE_EINVAL])

    def plan(seq, new, *a, **kw):
        a[-1].fill_(next(codes))

    monkeypatch.setattr(paged.moe, "moe_kv_plan", plan)
    ca, new = _cache(paged), torch.zeros(8, dtype=torch.int32)
    ca.plan(new)
    ca.check()
    for _ in range(3):
        ca.plan(new)
    assert ca.status.tolist() == [0]
    with pytest.raises(paged.moe.MoEError) as e:
        ca.check()
    assert e.value.status == paged.moe.MOE_ENOSPACE
    ca.check()
    ca.plan(new)
    ca.check()
    ca.plan(new)
    with pytest.raises(paged.moe.MoEError):
        ca.check()


@pytest.mark.parametrize("steps", [0, -1])
def test_run_refuses_no_steps(paged, steps):
    with pytest.raises(ValueError):
        paged.run(None, 1, 1, steps)
