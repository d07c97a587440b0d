"""A decoder layer's steps over a paged cache (needs a GPU): plan, append,
attention, scored route and expert FFN together, against the formulas in 64
bits over the keys and values as the steps made them."""
from dataclasses import replace

import numpy as np
import pytest
import torch

from int4_expert_gemv_gb300.configs import TINY
from test_gpu_scored_route import _rule

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,D,page,dtype", [(4, 2, 64, 16, torch.bfloat16), (6, 1, 80, 8, torch.float8_e4m3fn)])
def test_paged_decoder_steps(Hq, Hkv, D, page, dtype):
    from int4_expert_gemv_gb300 import build
    build.build()
    from int4_expert_gemv_gb300 import paged
    cfg = replace(TINY, seed=5)
    R = 5
    e4m3 = dtype == torch.float8_e4m3fn
    cache = paged.PagedCache(R, 24, page, Hkv, D, 8, 64, dtype, scale=0.02)
    dec = paged.PagedDecoder(paged.DeviceModel(cfg, heads=False), cache, Hq, n_group=4, keep_group=2)
    keys = [[] for _ in range(R)]
    g = torch.Generator(device="cuda").manual_seed(7)
    rng = np.random.default_rng(1)
    for step in range(40):
        new = [1 if rng.random() < 0.8 else 0 for _ in range(R)]
        if step % 9 == 8:
            new[int(rng.integers(R))] = -1
        rows = torch.tensor([r for r in range(R) if new[r] == 1], device="cuda", dtype=torch.int64)
        x = torch.randn((R, cfg.d), generator=g, device="cuda")
        out = dec.step(x, rows, torch.tensor(new, dtype=torch.int32, device="cuda"))
        for r in range(R):
            if new[r] == -1:
                keys[r] = []
        # the projections as the step makes them
        n = [len(keys[r]) + max(0, new[r]) for r in range(R)]
        assert int(cache.status[0]) == 0 and cache.seq_len.tolist() == n
        xn = (x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)).bfloat16()
        qkv = xn @ dec.w_qkv
        at = torch.tensor([max(0, i - 1) for i in n], device="cuda")
        q = paged.rotate(qkv[:, : Hq * D].view(R, Hq, D), at)
        k = paged.rotate(qkv[:, Hq * D: (Hq + Hkv) * D].view(R, Hkv, D), at)
        v = qkv[:, (Hq + Hkv) * D:].view(R, Hkv, D)
        if e4m3:
            k, v = (((t.float() / 0.02).clamp(-448, 448)).to(dtype).double() * float(cache.scales[0, 0]) for t in (k, v))
        for r in rows.tolist():
            keys[r].append((k[r].double(), v[r].double()))
        for r in range(R):
            if not keys[r]:
                assert (dec.attn[r] == 0).all()
                continue
            kk = torch.stack([t[0] for t in keys[r]]).transpose(0, 1).repeat_interleave(Hq // Hkv, 0)
            vv = torch.stack([t[1] for t in keys[r]]).transpose(0, 1).repeat_interleave(Hq // Hkv, 0)
            s = torch.einsum("hd,hnd->hn", q[r].double(), kk) * D ** -0.5
            ref = torch.einsum("hn,hnd->hd", torch.softmax(s, 1), vv)
            # half a unit of bf16; weights of 11 bits and scores in fp32
            tol = 2.0 ** -8 * ref.abs() + (2.0 ** -12 + 2.0 ** -18) * vv.abs().amax()
            assert ((dec.attn[r].double() - ref).abs() <= tol).all()
        # the route of the step's own logits, and the combination of its experts
        z, b = dec.logits.double().cpu().numpy(), dec.bias.double().cpu().numpy()
        for r in range(R):
            idx, w, margin = _rule(z[r], cfg.K, "sigmoid", 4, 2, 2, True, 2.5, b)
            if margin > 2.0 ** -20:
                assert dec.idx[r].tolist() == list(idx)
                assert np.abs(dec.w[r].double().cpu().numpy() - w).max() <= 2.0 ** -18 * w.max()
        ref = dec.hidden.double() + (dec.w.double()[:, :, None] * dec.y[:, : cfg.K].double()).sum(1)
        # K fused multiply-adds in fp32 onto the residual
        size = dec.hidden.double().abs() + (dec.w.double()[:, :, None] * dec.y[:, : cfg.K].double()).abs().sum(1)
        assert ((out.double() - ref).abs() <= 2.0 ** -22 * size).all()


def test_paged_run_reports(capsys):
    from int4_expert_gemv_gb300 import paged
    r = paged.run(TINY, 3, 50, 6, Hq=4, Hkv=2, D=64)
    assert r["requests"] == 3 and r["us_per_step"] > 0 and 3 * 32 <= r["cached_tokens"] <= 3 * 56


def test_paged_step_in_a_graph_goes_on_with_each_replay():
    """Captured once and replayed: the same steps as without a graph, bit for
    bit, from the lengths and free pages to the layer's result."""
    from int4_expert_gemv_gb300 import build
    build.build()
    from int4_expert_gemv_gb300 import paged
    cfg, R = replace(TINY, seed=5), 4
    model = paged.DeviceModel(cfg, heads=False)
    both = []
    for _ in range(2):
        cache = paged.PagedCache(R, 30, 4, 2, 64, 8, R)
        both.append((cache, paged.PagedDecoder(model, cache, 4, n_group=4, keep_group=2)))
    g = torch.Generator(device="cuda").manual_seed(3)
    xs = torch.randn((9, R, cfg.d), generator=g, device="cuda")
    rows, one = torch.arange(R, device="cuda"), torch.ones(R, dtype=torch.int32, device="cuda")
    x = xs[0].clone()
    want = []
    for t in range(9):
        cache, dec = both[0]
        out = dec.step(xs[t], rows, one).clone()
        want.append((out, cache.seq_len.clone(), cache.pool.clone(), cache.table.clone(), cache.slots.clone(), dec.attn.clone()))
    cache, dec = both[1]
    dec.step(x, rows, one)                               # the first step as it is, then the graph's
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dec.step(x, rows, one)
    for t in range(1, 9):
        x.copy_(xs[t])
        graph.replay()
        torch.cuda.synchronize()
        got = (dec.out, cache.seq_len, cache.pool, cache.table, cache.slots, dec.attn)
        assert cache.seq_len.tolist() == [t + 1] * R and cache.status.tolist() == [0]
        for a, b in zip(got, want[t]):
            assert torch.equal(a, b)


def test_paged_steps_without_room_are_told():
    from int4_expert_gemv_gb300 import build
    build.build()
    from int4_expert_gemv_gb300 import moe, paged
    cfg, R = replace(TINY, seed=5), 3
    cache = paged.PagedCache(R, 3, 2, 2, 64, 8, R)       # a page of two tokens for each, and no more
    dec = paged.PagedDecoder(paged.DeviceModel(cfg, heads=False), cache, 4, n_group=4, keep_group=2)
    x = torch.randn((R, cfg.d), device="cuda")
    rows = torch.arange(R, device="cuda")
    new = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for _ in range(2):
        dec.step(x, rows, new(1, 1, 1))
    cache.check()
    dec.step(x, rows, new(1, 1, 1))                      # does not fit
    dec.step(x, rows[:0], new(0, 0, -1))                 # does
    assert cache.status.tolist() == [0] and cache.seq_len.tolist() == [2, 2, 0]
    with pytest.raises(moe.MoEError) as e:
        cache.check()
    assert e.value.status == moe.MOE_ENOSPACE
    dec.step(x, rows[:1], new(1, 0, 0))
    cache.check()
    assert cache.seq_len.tolist() == [3, 2, 0]


@pytest.mark.parametrize("steps", [1, 2, 3, 4])
def test_paged_run_of_few_steps(steps):
    from int4_expert_gemv_gb300 import build
    build.build()
    from int4_expert_gemv_gb300 import paged
    r = paged.run(TINY, 2, 20, steps, Hq=4, Hkv=2, D=64)
    assert r["us_per_step"] > 0 and 2 * 11 + 2 * steps <= r["cached_tokens"] <= 2 * 20 + 2 * steps
