"""The paged key-value cache on the GPU (needs a GPU): the page plan against a
plain allocator, the append against elementwise rounding, the attention of
one new token per request against the formula in 64 bits."""
import ctypes as C
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

E4M3_MAX = 448.0


@pytest.fixture(scope="module")
def m():
    from int4_expert_gemv_gb300 import build
    build.build()
    from int4_expert_gemv_gb300 import moe
    moe.lib()
    return moe


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------ plan
class Plan:
    """The plan's buffers, and its rules written out one request at a time."""

    def __init__(self, R, max_blocks, page, n_pages, cap, seed=0):
        self.R, self.mb, self.page, self.P, self.cap = R, max_blocks, page, n_pages, cap
        self.rng = np.random.default_rng(seed)
        self.table = np.full((R, max_blocks), -7, np.int32)
        self.ring = self.rng.permutation(n_pages).astype(np.int32)
        self.pool = [int(self.rng.integers(0, n_pages)), n_pages]
        self.seq = np.zeros(R, np.int32)
        self.dev = None

    def expect(self, new):
        """(status, outputs) of one step; the state moves on when it is 0."""
        R, page, P, cap = self.R, self.page, self.P, self.cap
        have = [-(-int(s) // page) for s in self.seq]
        add = [max(0, int(n)) for n in new]
        after = [-(-(int(s) + a) // page) for s, a in zip(self.seq, add)]
        need = sum(a - h for a, h in zip(after, have))
        head, free = self.pool
        first = np.zeros(R + 1, np.int32)
        slots, places = np.full(cap, -1, np.int32), np.zeros(cap, np.int32)
        if max(after, default=0) > self.mb or need > free or sum(add) > cap:
            return 5, (self.seq.copy(), first, slots, places, list(self.pool))
        ring0, j, i, gone = self.ring.copy(), 0, 0, []
        out = self.seq.copy()
        for r in range(R):
            for b in range(have[r], after[r]):
                self.table[r, b] = ring0[(head + j) % P]
                j += 1
            first[r] = i
            for t in range(int(self.seq[r]), int(self.seq[r]) + add[r]):
                slots[i] = self.table[r, t // page] * page + t % page
                places[i] = t
                i += 1
            out[r] = self.seq[r] + add[r]
            if new[r] < 0:
                gone += list(self.table[r, : have[r]])
                out[r] = 0
        first[R] = i
        for k, g in enumerate(gone):
            self.ring[(head + free + k) % P] = g
        self.pool = [(head + need) % P, free - need + len(gone)]
        self.seq = out
        return 0, (out.copy(), first, slots, places, list(self.pool))

    def upload(self):
        self.dev = dict(table=torch.from_numpy(self.table.copy()).cuda(), ring=torch.from_numpy(self.ring.copy()).cuda(),
                        seq=torch.from_numpy(self.seq.copy()).cuda(), pool=_ints(self.pool))

    def call(self, m, new):
        d, R = self.dev, self.R
        fill = lambda n: torch.full((n,), 12345, dtype=torch.int32, device="cuda")  # noqa: E731
        o = dict(seq=fill(R), first=fill(R + 1), slots=fill(self.cap), places=fill(self.cap), pool=fill(2), status=fill(1))
        m.moe_kv_plan(d["seq"], _ints(list(new)), R, d["table"], self.mb, self.page, d["ring"], self.P, d["pool"],
                      o["seq"], o["first"], o["slots"], o["places"], self.cap, o["pool"], o["status"])
        got = {k: v.cpu().numpy() for k, v in o.items()}
        d["seq"], d["pool"] = o["seq"], o["pool"]
        return got


def _same_step(m, plan, new):
    st, (seq, first, slots, places, pool) = plan.expect(new)
    got = plan.call(m, new)
    assert got["status"][0] == st
    assert np.array_equal(got["seq"], seq) and np.array_equal(got["first"], first)
    assert np.array_equal(got["slots"], slots) and np.array_equal(got["places"], places)
    assert got["pool"].tolist() == pool
    assert np.array_equal(plan.dev["table"].cpu().numpy(), plan.table)
    assert np.array_equal(plan.dev["ring"].cpu().numpy(), plan.ring)
    return st


@pytest.mark.parametrize("R,max_blocks,page,n_pages,cap", [
    (1, 4, 16, 3, 64), (5, 9, 1, 20, 30), (33, 7, 24, 150, 700), (256, 40, 16, 5000, 4000), (1000, 3, 128, 2000, 999),
    (600, 64, 3, 9000, 20000)])
def test_plan_steps_follow_the_allocator(m, R, max_blocks, page, n_pages, cap):
    """Many steps in a row: requests grow, wait, end and start again, some
    steps ask for more than there is and change nothing."""
    p = Plan(R, max_blocks, page, n_pages, cap, seed=R)
    p.upload()
    seen = set()
    for step in range(12):
        big = p.rng.random(R) < 0.3
        new = np.where(big, p.rng.integers(0, 2 * page + 2, R), p.rng.integers(0, 2, R))
        new = np.where(p.rng.random(R) < 0.15, -1, new)
        if step % 4 != 3:                            # otherwise as drawn, too much or not
            over = p.seq + np.maximum(new, 0) > max_blocks * page
            new = np.where(over, -1, new)
            room = cap
            for r in range(R):
                new[r] = min(new[r], room)
                room -= max(0, new[r])
        seen.add(_same_step(m, p, new))
        held = [p.table[r, b] for r in range(R) for b in range(-(-int(p.seq[r]) // page))]
        free = [p.ring[(p.pool[0] + i) % n_pages] for i in range(p.pool[1])]
        assert sorted(held + free) == list(range(n_pages))   # every page once, always
    assert 0 in seen


def test_plan_refuses_what_does_not_fit(m):
    def step(seq, new, max_blocks=4, page=8, n_pages=10, cap=40, pool=(3, 5)):
        R = len(seq)
        table = torch.arange(R * max_blocks, dtype=torch.int32, device="cuda").view(R, max_blocks) % n_pages
        ring = torch.arange(n_pages, dtype=torch.int32, device="cuda")
        before = table.clone(), ring.clone()
        fill = lambda n: torch.full((n,), 9, dtype=torch.int32, device="cuda")  # noqa: E731
        so, fi, sl, pl, po, st = fill(R), fill(R + 1), fill(cap), fill(cap), fill(2), fill(1)
        m.moe_kv_plan(_ints(list(seq)), _ints(list(new)), R, table, max_blocks, page, ring, n_pages, _ints(list(pool)), so, fi, sl, pl,
                      cap, po, st)
        status = int(st[0])
        if status:
            assert torch.equal(table, before[0]) and torch.equal(ring, before[1])
            assert so.tolist() == list(seq) and fi.tolist() == [0] * (R + 1) and po.tolist() == list(pool)
            assert sl.tolist() == [-1] * cap and pl.tolist() == [0] * cap
        return status

    top = 2 ** 31 - 1
    assert step([8, 3], [1, 1]) == m.MOE_OK
    assert step([8, 3], [25, 0]) == m.MOE_ENOSPACE            # the row
    assert step([8, 3], [8, 8], pool=(3, 1)) == m.MOE_ENOSPACE   # the pages
    assert step([0, 0], [20, 21]) == m.MOE_ENOSPACE           # the slots
    assert step([0, 0], [top, top]) == m.MOE_ENOSPACE
    assert step([8, 3], [top, -1]) == m.MOE_ENOSPACE
    assert step([-1, 3], [0, 0]) == m.MOE_EINVAL
    assert step([33, 3], [0, 0]) == m.MOE_EINVAL              # longer than its row
    assert step([8, 3], [-2, 0]) == m.MOE_EINVAL
    for pool in [(10, 5), (-1, 5), (0, 11), (0, -1)]:
        assert step([8, 3], [0, 0], pool=pool) == m.MOE_EINVAL
    assert step([32, 32], [-1, -1], pool=(0, 5)) == m.MOE_EINVAL  # 8 pages back into a ring with 5 of 10
    assert step([], []) == m.MOE_OK


def test_plan_of_no_new_tokens_and_of_many_requests(m):
    p = Plan(16384, 2, 4, 20000, 0, seed=3)
    p.upload()
    assert _same_step(m, p, np.zeros(16384, np.int64)) == 0
    p = Plan(16384, 2, 4, 20000, 16384, seed=4)
    p.upload()
    assert _same_step(m, p, p.rng.integers(0, 2, 16384)) == 0
    assert _same_step(m, p, p.rng.integers(-1, 2, 16384)) == 0


def test_plan_marks_slots_of_pages_that_do_not_exist(m):
    one = lambda v: _ints([v])  # noqa: E731
    table, ring = _ints([[77, -1, 0, 0]]), _ints([5, 1, 2, 3, 0])
    so, fi, sl, pl, po, st = (_ints([0] * n) for n in (1, 2, 12, 12, 2, 1))
    m.moe_kv_plan(one(2), one(8), 1, table, 4, 4, ring, 5, _ints([0, 5]), so, fi, sl, pl, 12, po, st)
    assert st.tolist() == [0]
    # places 2..3 stand in page 77, 4..7 in ring entry 5 (neither is a page), 8..9 in page 1
    assert sl.tolist() == [-1] * 6 + [4, 5] + [-1] * 4
    assert pl.tolist() == list(range(2, 10)) + [0] * 4


# ------------------------------------------------------------ append
def _desc(m, kv, scales=(None, None), split=False):
    """kv [pages][2][Hkv][page][D], or with split two arrays [pages][Hkv][page][D]."""
    k, v = (kv[0], kv[1]) if split else (kv[:, 0], kv[:, 1])
    P, H, page, D = k.shape
    elt = k.element_size()
    return m.KVDesc(n_pages=P, page=page, Hkv=H, D=D, dtype=m.MOE_DTYPE_BF16 if elt == 2 else m.MOE_DTYPE_E4M3, k=k.data_ptr(),
                    v=v.data_ptr(), page_stride=k.stride(0) * elt, k_scale=None if scales[0] is None else scales[0].data_ptr(),
                    v_scale=None if scales[1] is None else scales[1].data_ptr())


@pytest.mark.parametrize("x", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cache", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("N,H,page,D", [(1, 1, 1, 16), (7, 3, 24, 80), (130, 8, 16, 128), (65, 2, 5, 256)])
def test_append_stores_rounded_rows_and_nothing_else(m, x, cache, N, H, page, D):
    g = torch.Generator(device="cuda").manual_seed(N + D)
    P = N // page + 3
    qkv = (3 * torch.randn((N, 4 * H * D), generator=g, device="cuda"))
    qkv[0, H * D: H * D + 8] = torch.tensor([float("nan"), float("inf"), -float("inf"), 1e30, -1e30, 0.0, -0.0, 2.0 ** -9],
                                            device="cuda")
    qkv = qkv.to(x)
    k, v = qkv[:, H * D: 2 * H * D], qkv[:, 3 * H * D:]
    sc = (None, None)
    if cache != torch.bfloat16:
        sc = tuple(0.01 + 0.01 * torch.rand(H, generator=g, device="cuda") for _ in range(2))
    bits = torch.int16 if cache == torch.bfloat16 else torch.uint8
    kv = torch.full((P, 2, H, page, D), 77, dtype=bits, device="cuda")
    ref = kv.clone().cpu()
    slots = torch.randperm(P * page, generator=g, device="cuda", dtype=torch.int32)[:N].clone()
    if N > 6:
        slots[3], slots[5] = -1, P * page                # padding, and outside the cache
    m.moe_kv_append(_desc(m, kv, sc), k, v, slots, N)
    for part, t, s in ((0, k, sc[0]), (1, v, sc[1])):
        t = t.reshape(N, H, D).float()
        if s is not None:
            t = (t / s[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        t = t.to(cache).view(bits).cpu()
        for n, slot in enumerate(slots.tolist()):
            if 0 <= slot < P * page:
                ref[slot // page, part, :, slot % page] = t[n]
    got, at = kv.cpu(), kv.view(cache).float().isnan().cpu()
    assert torch.equal(at, ref.view(cache).float().isnan())
    assert torch.equal(got[~at], ref[~at])


@pytest.mark.parametrize("scale", [1.0, 0.3, 0.0107421875, 3.0, 1e-30, 2.0 ** -127, 1e38, 3e38, 0.0])
def test_append_e4m3_rounds_the_exact_quotient(m, scale):
    """Quotients at and beside every midpoint of two e4m3 numbers, around its
    smallest and largest ones, and with scales whose reciprocal is no normal
    number: the bits of the quotient rounded to fp32 and then to e4m3."""
    H, D, page = 2, 64, 16
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    codes = codes[~codes.isnan()].unique()
    mid = torch.cat([(codes[1:] + codes[:-1]) / 2, codes, torch.tensor([448.0, 464.0, 480.0, 1e4, 2.0 ** -11, 2.0 ** -40], dtype=torch.float64)])
    x = (mid * scale).float()
    near = [x]
    for toward in (float("inf"), -float("inf")):
        y = x
        for _ in range(4):
            y = torch.nextafter(y, torch.tensor(toward))
            near.append(y)
    x = torch.cat(near)
    x = torch.cat([x, -x, torch.tensor([0.0, -0.0, float("inf"), -float("inf"), float("nan")])])
    N = -(-x.numel() // (H * D))
    x = torch.nn.functional.pad(x, (0, N * H * D - x.numel())).view(N, H * D).cuda()
    P = -(-N // page)
    kv = torch.zeros((P, 2, H, page, D), dtype=torch.uint8, device="cuda")
    sc = torch.full((H,), scale, device="cuda")
    m.moe_kv_append(_desc(m, kv, (sc, sc)), x, x, torch.arange(N, dtype=torch.int32, device="cuda"), N)
    want = (x / sc[0]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(N, H, D)
    for part in range(2):
        got = torch.stack([kv[n // page, part, :, n % page] for n in range(N)])
        nan = want.float().isnan()
        assert torch.equal(got.view(torch.float8_e4m3fn).float().isnan(), nan)
        assert torch.equal(got[~nan], want.view(torch.uint8)[~nan])


# ------------------------------------------------------------ attention
def _attend_case(m, lens, Hq, H, D, page, q_type, cache, window=0, seed=0, split=False, pad=0, P=None, spread=1.0, table_pad=2):
    """Runs one call on a cache whose every number behind the lengths is NaN,
    and whose table entries behind the blocks name no page."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B = len(lens)
    nb = [-(-max(0, n) // page) for n in lens]
    P = P or sum(nb) + 2
    wide = max(nb + [0]) + table_pad
    table = torch.full((B, wide), 2 ** 30, dtype=torch.int32, device="cuda")
    pages = torch.randperm(P, generator=g, device="cuda", dtype=torch.int32).tolist()
    for b, n in enumerate(nb):
        for j in range(n):
            table[b, j] = pages.pop()
    f8 = cache == torch.float8_e4m3fn
    shape = (2, P, H, page, D) if split else (P, 2, H, page, D)
    kv = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    k, v = (kv[0], kv[1]) if split else (kv[:, 0], kv[:, 1])
    sc = tuple(0.01 + 0.01 * torch.rand(H, generator=g, device="cuda") for _ in range(2)) if f8 else (None, None)
    for b, n in enumerate(lens):
        if n > 0:
            at = torch.arange(n, device="cuda")
            pg, off = table[b].long()[at // page], at % page
            for part in (k, v):
                x = torch.randn((n, H, D), generator=g, device="cuda") * spread
                part[pg, :, off] = (x / 0.015).clamp(-E4M3_MAX, E4M3_MAX).bfloat16() if f8 else x.bfloat16()
    kv = kv.to(cache)
    q = torch.randn((B, Hq * D + pad), generator=g, device="cuda").to(q_type)[:, : Hq * D].view(B, Hq, D)
    out = torch.full((B, Hq * D + pad), 5.0, dtype=q_type, device="cuda")
    lse = torch.full((B, Hq), 5.0, device="cuda")
    seq = _ints(list(lens))
    desc = _desc(m, kv, sc, split)
    ws = torch.full((m.moe_paged_attention_workspace_bytes(desc, B, Hq),), 255, dtype=torch.uint8, device="cuda")
    return dict(kv=kv, sc=sc, q=q, out=out, o=out[:, : Hq * D].view(B, Hq, D), lse=lse, seq=seq, table=table, desc=desc, ws=ws, lens=lens,
                Hq=Hq, H=H, D=D, page=page, window=window, split=split, scale=D ** -0.5)


def _call(m, c, stream=None):
    m.moe_paged_attention(c["desc"], c["q"], len(c["lens"]), c["Hq"], c["seq"], c["table"], c["table"].shape[1], c["scale"], c["o"],
                          c["ws"], lse=c["lse"], window=c["window"], stream=stream)


def _check(c, skip=()):
    """The formula in 64 bits.  Bounds: with dx the error of a score (fp32
    sums of D products, each within 2^-22 of exact, and the exponent's
    argument in fp32), a weight is within 2 dx + 2^-20 of exact relative to
    the weights' sum, so out within that times max |v| -- and with a 16-bit
    result, whose weights keep 11 bits (2^-12 after rounding), 2^-12 max |v|
    more and half a unit of bf16 -- and lse within dx + 2^-20 (1 + |lse|)."""
    kv, D, G, page = c["kv"], c["D"], c["Hq"] // c["H"], c["page"]
    k, v = (kv[0], kv[1]) if c["split"] else (kv[:, 0], kv[:, 1])
    out, lse = c["o"].double(), c["lse"].double()
    for b, n in enumerate(c["lens"]):
        if b in skip:
            assert out[b].isnan().all() and lse[b].isnan().all()
            continue
        if n <= 0:
            assert (out[b] == 0).all() and (lse[b] == -float("inf")).all()
            continue
        at = torch.arange(max(0, n - c["window"]) if c["window"] else 0, n, device="cuda")
        pg, off = c["table"][b].long()[at // page], at % page
        for h in range(c["H"]):
            kk, vv = k[pg, h, off].double(), v[pg, h, off].double()
            if c["sc"][0] is not None:
                kk, vv = kk * c["sc"][0][h].double(), vv * c["sc"][1][h].double()
            rows = slice(h * G, (h + 1) * G)
            q = c["q"][b, rows].double()
            x = c["scale"] * (q @ kk.T)
            size = c["scale"] * (q.abs() @ kk.abs().T).amax(1, keepdim=True)
            dx = 2.0 ** -22 * size + 2.0 ** -22 * x.abs().amax(1, keepdim=True)
            ref, ref_l = torch.softmax(x, 1) @ vv, torch.logsumexp(x, 1)
            tol = (2 * dx + 2.0 ** -20) * vv.abs().amax()
            if c["q"].dtype == torch.bfloat16:
                tol = tol + 2.0 ** -12 * vv.abs().amax() + 2.0 ** -8 * ref.abs()
            err = (out[b, rows] - ref).abs()
            assert (err <= tol).all(), (b, h, n, float((err - tol).max()), float((err / tol).max()))
            err = (lse[b, rows] - ref_l).abs()
            tol = dx[:, 0] + 2.0 ** -20 * (1 + ref_l.abs())
            assert (err <= tol).all(), (b, h, n, "lse", float((err / tol).max()))


TYPES = [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float8_e4m3fn),
         (torch.float32, torch.float8_e4m3fn)]


@pytest.mark.parametrize("q,cache", TYPES)
@pytest.mark.parametrize("Hq,H,D,page", [
    (1, 1, 64, 16), (8, 2, 128, 16), (16, 2, 256, 32), (12, 12, 80, 24), (7, 1, 96, 8), (32, 2, 64, 64), (24, 2, 192, 16),
    (20, 1, 128, 1), (6, 2, 16, 5), (33, 1, 48, 128), (10, 1, 256, 100), (9, 1, 112, 7)])
def test_attention_against_the_formula(m, q, cache, Hq, H, D, page):
    """Head sizes and groups of every kind; lengths of none, one, and around
    the ends of pages and tiles; short rows beside long ones."""
    lens = [0, 1, page, page + 1, 2, 15, 16, 17, 63, 64, 65, 129, 700, -3, 1, 0, 1999]
    c = _attend_case(m, lens, Hq, H, D, page, q, cache, seed=Hq * D + page)
    _call(m, c)
    _check(c)


@pytest.mark.parametrize("q,cache", TYPES)
@pytest.mark.parametrize("window", [1, 5, 16, 100, 1000, 5000])
def test_attention_window(m, q, cache, window):
    c = _attend_case(m, [0, 1, 4, 5, 6, 100, 101, 999, 1000, 1001, 3001], 8, 2, 128, 16, q, cache, window=window, seed=window)
    _call(m, c)
    _check(c)


@pytest.mark.parametrize("q,cache", TYPES)
@pytest.mark.parametrize("lens,Hq,H,D,page", [
    ([20011], 8, 8, 128, 16), ([20011], 16, 1, 64, 64), ([9000, 1, 30001], 32, 2, 256, 24), ([1] * 300, 4, 2, 64, 16),
    (list(range(0, 400, 3)), 6, 1, 80, 16), ([12007] * 5, 40, 2, 128, 256)])
def test_attention_split_and_joined(m, q, cache, lens, Hq, H, D, page):
    """Few long rows and many short ones: the split over the length."""
    c = _attend_case(m, lens, Hq, H, D, page, q, cache, seed=len(lens))
    _call(m, c)
    _check(c)


def test_attention_strides_and_a_cache_of_two_arrays(m):
    for q in (torch.float32, torch.bfloat16):
        c = _attend_case(m, [33, 0, 500], 8, 2, 64, 16, q, torch.bfloat16, split=True, pad=24, seed=5)
        assert c["q"].stride(0) == 8 * 64 + 24
        _call(m, c)
        _check(c)
        assert (c["out"][:, 8 * 64:] == 5.0).all()          # between the rows


@pytest.mark.parametrize("q,cache", TYPES)
def test_attention_of_large_scores(m, q, cache):
    """Scores in the hundreds: the running maximum moves, weights underflow."""
    c = _attend_case(m, [1, 40, 2000, 7001], 8, 2, 128, 16, q, cache, spread=1.5, seed=8)
    c["scale"] = 4.0
    _call(m, c)
    _check(c)


def test_attention_never_reads_through_a_bad_page_or_past_the_table(m):
    for q, cache in TYPES:
        c = _attend_case(m, [100, 3000, 64, 50, 17], 8, 2, 64, 16, q, cache, seed=2)
        c["table"][1, 77] = c["desc"].n_pages                # a page that is not
        c["table"][3, 0] = -1
        c["lens"][2] = c["table"].shape[1] * 16 + 1          # longer than its row
        c["seq"][2] = c["lens"][2]
        _call(m, c)
        _check(c, skip=(1, 2, 3))
        c["window"] = 500                                    # the bad page of row 1 is out of the window
        c["lens"][2] = 64
        c["seq"][2] = 64
        _call(m, c)
        _check(c, skip=(3,))


@pytest.mark.parametrize("q", [torch.bfloat16, torch.float32])
def test_attention_of_scales_of_zero_and_below(m, q):
    """Key scales of 0 (every weight alike) and below 0, and a value scale of
    0, with tiles that are partly masked."""
    c = _attend_case(m, [1, 5, 100, 333], 8, 4, 64, 16, q, torch.float8_e4m3fn, window=77, seed=3)
    c["sc"][0][0], c["sc"][0][1], c["sc"][1][2] = 0.0, -0.02, 0.0
    _call(m, c)
    _check(c)


def test_attention_without_lse_and_of_no_rows(m):
    c = _attend_case(m, [70, 3], 4, 2, 64, 16, torch.bfloat16, torch.bfloat16)
    _call(m, c)
    want, c["out"][:] = c["o"].clone(), 0
    m.moe_paged_attention(c["desc"], c["q"], 2, 4, c["seq"], c["table"], c["table"].shape[1], c["scale"], c["o"], c["ws"])
    assert torch.equal(c["o"], want)
    m.moe_paged_attention(c["desc"], c["q"][:0], 0, 4, c["seq"], c["table"], c["table"].shape[1], c["scale"], c["o"][:0], c["ws"])


def test_attention_gives_the_same_bits_again_and_on_another_stream(m):
    for q, cache in TYPES:
        c = _attend_case(m, [5000, 1, 0, 333, 12000], 16, 2, 128, 16, q, cache, seed=4)
        _call(m, c)
        want = c["o"].clone(), c["lse"].clone()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        for stream in (None, s, s):
            c["out"].zero_()
            c["ws"].fill_(17)
            torch.cuda.synchronize()
            _call(m, c, stream)
            torch.cuda.synchronize()
            assert torch.equal(c["o"], want[0]) and torch.equal(c["lse"], want[1])


def test_attention_in_a_graph_follows_the_lengths(m):
    """Captured once, replayed with other lengths and another table."""
    c = _attend_case(m, [900, 17, 0], 8, 2, 64, 16, torch.bfloat16, torch.bfloat16, seed=6)
    _call(m, c)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _call(m, c)
    for lens in ([900, 17, 0], [33, 17, 0], [900, 1, 0]):
        c["seq"].copy_(_ints(lens))
        c["lens"] = lens
        g.replay()
        torch.cuda.synchronize()
        _check(c)


@pytest.mark.parametrize("cache", [torch.bfloat16, torch.float8_e4m3fn])
def test_cache_offsets_past_32_bits(m, cache):
    """A cache of some 9 GB: pages whose numbers stand past 2^32 bytes and,
    in 16 bits, past 2^32 numbers."""
    H, page, D = 8, 64, 128
    elt = 2 if cache == torch.bfloat16 else 1
    P = (9 << 30) // (2 * H * page * D * elt)
    kv = torch.empty((P, 2, H, page, D), dtype=cache, device="cuda")
    ids = [P - 1, P // 2 + 1, 0, P - 7]
    n = 3 * page + 9
    slots = _ints([ids[t // page] * page + t % page for t in range(n)])
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((n, H, D), generator=g, device="cuda") for _ in range(2))
    sc = (None, None) if elt == 2 else tuple(torch.full((H,), 0.01, device="cuda") for _ in range(2))
    desc = _desc(m, kv, sc)
    m.moe_kv_append(desc, k, v, slots, n)
    for part, x, s in ((0, k, sc[0]), (1, v, sc[1])):
        got = torch.stack([kv[ids[t // page], part, :, t % page].float() for t in range(n)])
        x = x if s is None else (x / s[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        assert torch.equal(got, x.to(cache).float())
    table = _ints([ids])
    q = torch.randn((1, 16, D), generator=g, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((1, 16), device="cuda")
    c = dict(kv=kv, sc=sc, q=q, o=out, lse=lse, seq=_ints([n]), table=table, desc=desc, lens=[n], Hq=16, H=H, D=D, page=page, window=0,
             split=False, scale=D ** -0.5,
             ws=torch.empty(m.moe_paged_attention_workspace_bytes(desc, 1, 16), dtype=torch.uint8, device="cuda"))
    _call(m, c)
    _check(c)


def test_plan_append_attend_together(m):
    """Requests that grow from nothing, token by token and in prompts, with
    pages that come back: the attention over the cache equals the one over
    the keys as they were given."""
    R, H, Hq, D, page, P, mb, cap = 5, 2, 6, 64, 8, 60, 20, 64
    kv = torch.full((P, 2, H, page, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    desc = _desc(m, kv)
    z = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    table, ring = torch.full((R, mb), -1, dtype=torch.int32, device="cuda"), torch.arange(P, dtype=torch.int32, device="cuda")
    seq, pool, first, slots, places, status = z(R), _ints([0, P]), z(R + 1), z(cap), z(cap), z(1)
    keys = [[] for _ in range(R)]
    g = torch.Generator(device="cuda").manual_seed(3)
    rng = np.random.default_rng(3)
    ws = torch.empty(m.moe_paged_attention_workspace_bytes(desc, R, Hq), dtype=torch.uint8, device="cuda")
    for step in range(20):
        new = [int(rng.integers(5, 13)) if not keys[r] else 1 for r in range(R)]
        if step % 6 == 5:
            new[step % R] = -1
        seq_out, pool_out = z(R), z(2)
        m.moe_kv_plan(seq, _ints(new), R, table, mb, page, ring, P, pool, seq_out, first, slots, places, cap, pool_out, status)
        seq, pool = seq_out, pool_out
        k, v = (torch.randn((cap, H, D), generator=g, device="cuda").bfloat16() for _ in range(2))
        m.moe_kv_append(desc, k, v, slots, cap)
        i = 0
        for r in range(R):
            if new[r] < 0:
                keys[r] = []
            for _ in range(max(0, new[r])):
                keys[r].append((k[i], v[i]))
                i += 1
        q = torch.randn((R, Hq, D), generator=g, device="cuda").bfloat16()
        out, lse = torch.empty_like(q), torch.empty((R, Hq), device="cuda")
        m.moe_paged_attention(desc, q, R, Hq, seq, table, mb, D ** -0.5, out, ws, lse=lse)
        assert status.tolist() == [0] and seq.tolist() == [len(x) for x in keys]
        for r in range(R):
            if not keys[r]:
                assert (out[r] == 0).all()
                continue
            kk = torch.stack([x[0] for x in keys[r]]).double().transpose(0, 1).repeat_interleave(Hq // H, 0)
            vv = torch.stack([x[1] for x in keys[r]]).double().transpose(0, 1).repeat_interleave(Hq // H, 0)
            x = torch.einsum("hd,hnd->hn", q[r].double(), kk) * D ** -0.5
            ref = torch.einsum("hn,hnd->hd", torch.softmax(x, 1), vv)
            # bf16's half unit, and 2^-12 + 2^-18 of the largest value for the weights and scores
            tol = 2.0 ** -8 * ref.abs() + (2.0 ** -12 + 2.0 ** -18) * vv.abs().amax()
            assert ((out[r].double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("cache", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("Hq", [1, 8, 12, 16, 20])
def test_attention_weights_keep_sixteen_bits(m, cache, Hq):
    """Two tokens of nearly one score and of opposite values: the result is
    small beside the values, so what counts is the weights' rounding and not
    the result's own.  Bound: as above, with 2^-16 for the weights (2^-17 each
    where they are rounded to 16 bits, and the sum of them as much)."""
    c = _attend_case(m, [2, 2, 2], Hq, 1, 64, 16, torch.bfloat16, cache, seed=Hq)
    c["scale"] = 1.0
    c["q"].zero_()
    c["q"][:, :, 0] = (2.0 ** -6 * (1 + torch.arange(3 * Hq, device="cuda") / (2.0 * Hq))).view(3, Hq).bfloat16()
    one, most = (1.0, 4.0) if cache == torch.bfloat16 else (64.0, 448.0)
    for b in range(3):
        page = c["kv"][int(c["table"][b, 0])].view(2, 1, 16, 64)
        rows = torch.zeros((2, 2, 64), device="cuda")
        rows[0, 0, 0] = one
        rows[1, 0], rows[1, 1] = most, -most
        page.view(torch.uint8)[:, 0, :2] = rows.to(cache).view(torch.uint8)
    _call(m, c)
    D, G = 64, Hq
    for b in range(3):
        p = int(c["table"][b, 0])
        k, v = c["kv"][p, 0, 0, :2].double(), c["kv"][p, 1, 0, :2].double()
        if c["sc"][0] is not None:
            k, v = k * c["sc"][0].double(), v * c["sc"][1].double()
        x = c["q"][b].double() @ k.T
        ref = torch.softmax(x, 1) @ v
        dx = 2.0 ** -21 * x.abs().amax(1, keepdim=True)
        tol = (2 * dx + 2.0 ** -20 + 2.0 ** -16) * v.abs().amax() + 2.0 ** -8 * ref.abs()
        err = (c["o"][b].double() - ref).abs()
        assert (err <= tol).all(), float((err / tol).max())


def test_plan_of_arrays_that_stand_side_by_side(m):
    """All eleven in one allocation, none overlapping: nothing is refused."""
    R, mb, page, P, cap = 5, 4, 8, 30, 40
    sizes = dict(seq=R, new=R, table=R * mb, ring=P, pool=2, so=R, fi=R + 1, sl=cap, pl=cap, po=2, st=1)
    slab, at = torch.full((sum(sizes.values()),), 9, dtype=torch.int32, device="cuda"), 0
    a = {}
    for k, n in sizes.items():
        a[k], at = slab[at: at + n], at + n
    a["seq"].copy_(_ints([0, 8, 3, 0, 31]))
    a["new"].copy_(_ints([9, 1, 0, 4, 1]))
    a["table"].copy_(_ints([-1] * 4 + [7, -1, -1, -1] + [8, -1, -1, -1] + [-1] * 4 + [1, 2, 3, 4]))
    a["ring"].copy_(torch.arange(P, dtype=torch.int32, device="cuda"))
    a["pool"].copy_(_ints([10, 12]))
    m.moe_kv_plan(a["seq"], a["new"], R, a["table"], mb, page, a["ring"], P, a["pool"], a["so"], a["fi"], a["sl"], a["pl"], cap, a["po"],
                  a["st"])
    assert a["st"].tolist() == [0] and a["so"].tolist() == [9, 9, 3, 4, 32] and a["fi"].tolist() == [0, 9, 10, 10, 14, 15]
    assert a["po"].tolist() == [14, 8]
    assert a["sl"].tolist() == list(range(80, 89)) + [96, 104, 105, 106, 107, 39] + [-1] * 25
    assert a["pl"].tolist() == list(range(9)) + [8, 0, 1, 2, 3, 31] + [0] * 25
    assert a["table"].tolist() == [10, 11, -1, -1, 7, 12, -1, -1, 8, -1, -1, -1, 13, -1, -1, -1, 1, 2, 3, 4]


@pytest.mark.parametrize("cap", [2 ** 31 - 1, 2 ** 31 - 70000])
def test_plan_with_room_for_all_the_slots_there_can_be(m, cap):
    """Slots and places of almost 2^31 entries (17 GB): a step that fits and
    one that does not, every entry written and nothing beside them."""
    slots, places = (torch.full((cap + 2,), 9, dtype=torch.int32, device="cuda") for _ in range(2))
    table, ring = _ints([[7, -1], [3, 5]]), torch.arange(12, dtype=torch.int32, device="cuda")
    so, fi, po, st = (_ints([8] * n) for n in (2, 3, 2, 1))
    for new, status, want in (([9, 2], 0, [63, 0, 1, 2, 3, 4, 5, 6, 7, 41, 42]), ([9, 9], 5, [])):
        at = [7, 8, 9, 10, 11, 12, 13, 14, 15, 9, 10] if want else []
        m.moe_kv_plan(_ints([7, 9]), _ints(new), 2, table, 2, 8, ring, 12, _ints([0, 4]), so, fi, slots[1:], places[1:], cap, po, st)
        assert st.tolist() == [status]
        for got, first, rest in ((slots, want, -1), (places, at, 0)):
            assert got[1: 1 + len(first)].tolist() == first
            assert int(got[0]) == 9 and int(got[-1]) == 9
            low, high = torch.aminmax(got[1 + len(first): cap + 1])
            assert int(low) == rest and int(high) == rest
        slots.fill_(9)
        places.fill_(9)


_PLAN_ALONE = """
import sys, torch
from int4_expert_gemv_gb300 import moe as m
R, page, n_pages, cap = int(sys.argv[1]), 16, 20000, 5000
i32 = lambda n, v=0: torch.full((n,), v, dtype=torch.int32, device="cuda")
table, ring = i32(R * 2, -1), torch.arange(n_pages, dtype=torch.int32, device="cuda")
seq, new = i32(R), i32(R, 1)
so, fi, sl, pl, po, st = i32(R), i32(R + 1), i32(cap), i32(cap), i32(2), i32(1, 9)
pool = torch.tensor([0, n_pages], dtype=torch.int32, device="cuda")
m.moe_kv_plan(seq, new, R, table, 2, page, ring, n_pages, pool, so, fi, sl, pl, cap, po, st)
at = torch.arange(R, dtype=torch.int32, device="cuda")
assert st.tolist() == [0] and torch.equal(sl[:R], at * page) and torch.equal(table.view(R, 2)[:, 0], at)
assert po.tolist() == [R, n_pages - R] and torch.equal(fi[:R], at) and int(fi[R]) == R and (so == 1).all()
"""


@pytest.mark.parametrize("R", [1024, 1025, 4010, 4052, 4053, 4095, 4096])
def test_plan_of_any_count_is_the_first_call_of_a_process(m, R):
    """The shared memory of a call does not go by what larger calls before it
    have asked for: each count in a process of its own."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _PLAN_ALONE, str(R)], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


# ------------------------------------------------------------ calls that fill the GPU
class _PlanAt(Plan):
    """A plan whose slots and places begin `at` numbers behind an aligned address."""
    at = 0

    def call(self, m, new):
        d, R, at = self.dev, self.R, self.at
        fill = lambda n: torch.full((n,), 12345, dtype=torch.int32, device="cuda")  # noqa: E731
        o = dict(seq=fill(R), first=fill(R + 1), slots=fill(self.cap + at + 5), places=fill(self.cap + at + 5), pool=fill(2), status=fill(1))
        m.moe_kv_plan(d["seq"], _ints(list(new)), R, d["table"], self.mb, self.page, d["ring"], self.P, d["pool"],
                      o["seq"], o["first"], o["slots"][at:], o["places"][at:], self.cap, o["pool"], o["status"])
        for k in ("slots", "places"):
            assert (o[k][:at] == 12345).all() and (o[k][at + self.cap:] == 12345).all()
            o[k] = o[k][at: at + self.cap]
        got = {k: v.cpu().numpy() for k, v in o.items()}
        d["seq"], d["pool"] = o["seq"], o["pool"]
        return got


@pytest.mark.parametrize("at", [0, 1, 4])
@pytest.mark.parametrize("R,max_blocks,page,n_pages,cap", [
    (3, 4000, 16, 9000, 100003), (7, 3000, 24, 20000, 65537), (300, 60, 16, 15000, 120002), (1500, 12, 64, 14000, 400001), (2, 60000, 1, 90000, 90000)])
def test_plan_of_prompts(m, at, R, max_blocks, page, n_pages, cap):
    """Room for more new tokens than the grid has threads: four a thread,
    odd counts, requests and pages that end within a thread's four."""
    p = _PlanAt(R, max_blocks, page, n_pages, cap, seed=R + at)
    p.at = at
    p.upload()
    most, seen = cap // R, []
    for step in range(5):
        new = p.rng.integers(0, max(2, 2 * most // 3), R)
        new = np.where(p.rng.random(R) < 0.3, p.rng.integers(0, 4, R), new)
        new = np.where((p.rng.random(R) < 0.2) | (p.seq + new > max_blocks * page), -1, new)
        if step == 3:
            new[0] = cap                                 # more than there is
        seen.append(_same_step(m, p, new))
    assert 0 in seen and 5 in seen


@pytest.mark.parametrize("x", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cache", [torch.bfloat16, torch.float8_e4m3fn])
def test_append_of_a_prompt(m, x, cache):
    """More chunks than the grid has threads, and an odd count of tokens."""
    N, H, page, D = 7003, 8, 24, 128
    g = torch.Generator(device="cuda").manual_seed(N)
    qkv = (2 * torch.randn((N, 3 * H * D + 8), generator=g, device="cuda")).to(x)
    k, v = qkv[:, 8: 8 + H * D], qkv[:, 8 + 2 * H * D:]
    sc = (None, None) if cache == torch.bfloat16 else tuple(0.01 + 0.01 * torch.rand(H, generator=g, device="cuda") for _ in range(2))
    bits = torch.int16 if cache == torch.bfloat16 else torch.uint8
    P = N // page + 9
    kv = torch.full((P, 2, H, page, D), 77, dtype=bits, device="cuda")
    slots = torch.randperm(P * page, generator=g, device="cuda", dtype=torch.int32)[:N].clone()
    slots[N // 2:: 41] = -1
    slots[3:: 97] = P * page
    ref = kv.clone()
    ok = (slots >= 0) & (slots < P * page)
    at = slots[ok].long()
    for part, (t, s) in enumerate(((k, sc[0]), (v, sc[1]))):
        t = t[ok].reshape(-1, H, D).float()
        if s is not None:
            t = (t / s[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        ref[at // page, part, :, at % page] = t.to(cache).view(bits)
    m.moe_kv_append(_desc(m, kv, sc), k, v, slots, N)
    assert torch.equal(kv, ref)


def test_append_of_more_chunks_than_32_bits_count(m):
    """4.2 million tokens of 16 heads of 256 (34 GB; keys and values are one
    array): those around the 2^31st chunk have slots."""
    H, D, page = 16, 256, 16
    span = (2 ** 31 - 1) // (H * D // 8)
    N = span + 1003
    x = torch.empty((N, H * D), dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, span - 2, span - 1, span, span + 1, N - 2, N - 1]
    g = torch.Generator(device="cuda").manual_seed(0)
    for r in rows:
        x[r] = torch.randn(H * D, generator=g, device="cuda").bfloat16()
    slots = torch.full((N,), -1, dtype=torch.int32, device="cuda")
    for i, r in enumerate(rows):
        slots[r] = 3 * i + 1
    kv = torch.zeros((3, 2, H, page, D), dtype=torch.bfloat16, device="cuda")
    ref = kv.clone()
    for i, r in enumerate(rows):
        ref[(3 * i + 1) // page, :, :, (3 * i + 1) % page] = x[r].view(H, D)
    m.moe_kv_append(_desc(m, kv), x, x, slots, N)
    assert torch.equal(kv, ref)


def _resident(q, cache):
    """CTAs of heads of 128 that are on the GPU at once."""
    two = q == torch.bfloat16 and cache == torch.bfloat16
    return torch.cuda.get_device_properties(0).multi_processor_count * (2 if two else 3)


@pytest.mark.parametrize("q,cache", TYPES)
def test_attention_of_a_batch_of_one_length(m, q, cache):
    """As many rows as there are CTAs, or a few less, of one length: the rows
    turn out to be best left whole, and the joins have nothing to do."""
    ctas = _resident(q, cache)
    for lens in ([1000] * (ctas * 9 // 80), [1000] * (ctas * 9 // 80 - 2) + [0, 1], [1024] * (ctas // 8)):
        c = _attend_case(m, lens, 32, 8, 128, 16, q, cache, seed=len(lens))
        c["ws"].fill_(85)
        _call(m, c)
        _check(c)
    n = len(lens)                                        # bad pages and lengths among them
    c["table"][2, 5], c["table"][n - 1, 0] = c["desc"].n_pages, -1
    c["lens"] = list(c["lens"])
    c["lens"][4] = c["table"].shape[1] * 16 + 1
    c["seq"][4] = c["lens"][4]
    _call(m, c)
    _check(c, skip=(2, 4, n - 1))


@pytest.mark.parametrize("q,cache", TYPES)
def test_attention_of_more_rows_than_ctas_left_whole(m, q, cache):
    """Nearly as many long rows as CTAs and some short and empty ones, so that
    there are more rows than CTAs but no more work than whole rows take."""
    ctas = _resident(q, cache)
    n = ctas * 93 // 800
    lens = [1000] * n + [40] * (ctas // 8 - n + 3) + [0, -1]
    c = _attend_case(m, lens, 32, 8, 128, 16, q, cache, seed=3)
    c["ws"].fill_(85)
    _call(m, c)
    _check(c)


@pytest.mark.parametrize("page", [16, 24])
@pytest.mark.parametrize("q,cache", TYPES)
def test_attention_of_more_rows_than_ctas_cut(m, q, cache, page):
    """64 ragged requests of 8 key heads, an ordinary batch: rows cut between
    CTAs and told by the CTA of their first part; then with bad pages."""
    rng = np.random.default_rng(4)
    lens = [int(n) for n in rng.integers(1, 2500, 64)]
    lens[7], lens[20], lens[63], lens[0] = 0, 9001, 1, 2500
    c = _attend_case(m, lens, 32, 8, 128, page, q, cache, seed=11)
    c["ws"].fill_(85)
    _call(m, c)
    _check(c)
    want = c["o"].clone(), c["lse"].clone()
    c["ws"].fill_(170)
    c["out"].zero_()
    _call(m, c)
    assert torch.equal(c["o"], want[0]) and torch.equal(c["lse"], want[1])
    c["window"] = 777
    _call(m, c)
    _check(c)
    c["window"] = 0
    c["table"][20, 200], c["table"][0, 3] = -1, 2 ** 31 - 1
    _call(m, c)
    _check(c, skip=(0, 20))


def test_attention_of_many_rows_with_more_heads_than_a_tile(m):
    """33 and 20 heads to a key head: tiles of 16 and a rest, more of them
    than CTAs."""
    for q, cache in TYPES:
        for Hq, H, D in ((66, 2, 64), (80, 4, 128), (40, 2, 256)):
            rng = np.random.default_rng(Hq)
            lens = [int(n) for n in rng.integers(0, 900, 90)]
            c = _attend_case(m, lens, Hq, H, D, 16, q, cache, seed=Hq)
            _call(m, c)
            _check(c)


def test_attention_keeps_a_bad_number_to_its_own_row(m):
    """NaN among the keys or values in sight: NaN for the heads that read it,
    and for nobody else."""
    for q, cache in TYPES:
        c = _attend_case(m, [300, 40, 1200, 17], 8, 2, 64, 16, q, cache, seed=21)
        kv = c["kv"].view(torch.int16 if cache == torch.bfloat16 else torch.uint8)
        nan = 0x7fc0 if cache == torch.bfloat16 else 0x7f
        kv[int(c["table"][2, 50]), 0, 1, 3, 5] = nan     # a key of request 2, key head 1
        kv[int(c["table"][3, 1]), 1, 0, 0, 9] = nan      # a value of request 3, key head 0
        _call(m, c)
        assert c["o"][2, 4:].isnan().all() and c["lse"][2, 4:].isnan().all()
        assert c["o"][3, :4, 9].isnan().all() and not c["lse"][3].isnan().any()
        assert int(c["o"].isnan().sum()) == 4 * 64 + 4
        clean = _attend_case(m, [300, 40, 1200, 17], 8, 2, 64, 16, q, cache, seed=21)
        _call(m, clean)
        ok = ~c["o"].isnan()
        assert torch.equal(c["o"][ok], clean["o"][ok])
