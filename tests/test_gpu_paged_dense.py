"""A decoder layer whose norms, projections and rotary embedding are in 8 bits
(needs a GPU): the steps' calls together, each against the formulas in 64 bits
on what the one before it left."""
from dataclasses import replace

import numpy as np
import pytest
import torch

from int4_expert_gemv_gb300.configs import TINY

pytestmark = pytest.mark.gpu


def _decoder(R, Hq, Hkv, D, page, dtype=torch.bfloat16, dense="e4m3"):
    from int4_expert_gemv_gb300 import build
    build.build()
    from int4_expert_gemv_gb300 import paged
    cfg = replace(TINY, seed=5)
    cache = paged.PagedCache(R, 8 * R, page, Hkv, D, 8, R, dtype, scale=0.02)
    return cfg, cache, paged.PagedDecoder(paged.DeviceModel(cfg, heads=False), cache, Hq, n_group=4, keep_group=2, dense=dense)


def _rows(x, scales):
    """Codes [R][n] with scales of 1 x 128 blocks, as numbers."""
    return x.double() * scales.double().repeat_interleave(128, 1)[:, : x.shape[1]]


def _weights(codes, scales):
    N, K = codes.shape
    return codes.double() * scales.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]


def _close(got, want, size, rel, bf16):
    tol = size * rel + (want.abs() * 2.0 ** -8 * (1 + 2.0 ** -7) if bf16 else 0)
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


@pytest.mark.parametrize("R,Hq,Hkv,D,page,dtype", [(5, 4, 2, 64, 16, torch.bfloat16), (70, 6, 1, 80, 8, torch.float8_e4m3fn), (1, 2, 2, 48, 16, torch.bfloat16)])
def test_dense_steps(R, Hq, Hkv, D, page, dtype):
    cfg, cache, dec = _decoder(R, Hq, Hkv, D, page, dtype)
    de, d = dec.dense, cfg.d
    g = torch.Generator(device="cuda").manual_seed(7)
    every, one = torch.arange(R, device="cuda"), torch.ones(R, dtype=torch.int32, device="cuda")
    keys = []
    for step in range(12):
        x = torch.randn((R, d), generator=g, device="cuda")
        out = dec.step(x, every, one)
        # the norm in 8 bits: half a step of a code, or of its smallest one, and the norm's fp32 (2^-18)
        xn = x.double() / torch.sqrt(x.double().square().mean(1, keepdim=True) + 1e-6)
        xc = _rows(de.x, de.x_scales)
        step_size = de.x_scales.double().repeat_interleave(128, 1)[:, :d]
        assert bool(((xc - xn).abs() <= xn.abs() * (2.0 ** -4 + 2.0 ** -17) + step_size * 2.0 ** -10).all())
        # the projection of those codes, rounded to bf16, then turned in fp32 from it and rounded again
        w = _weights(de.qkv_codes, de.qkv_scales)
        want, size = xc @ w.t(), xc.abs() @ w.abs().t()
        n = (Hq + Hkv) * D
        _close(de.qkv[:, n:], want[:, n:], size[:, n:], (128 + 2 + 2) * 2.0 ** -24, True)
        z = want[:, :n].view(R, Hq + Hkv, D)
        a, b = z[..., : D // 2], z[..., D // 2:]
        f = torch.exp(torch.arange(0, D, 2, device="cuda", dtype=torch.float64) * (-np.log(10000.0) / D)) * step
        c, s = torch.cos(f), torch.sin(f)
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
        pair = (a.abs() + b.abs()).repeat(1, 1, 2)
        sz = size[:, :n].view(R, Hq + Hkv, D)
        szp = (sz[..., : D // 2] + sz[..., D // 2:]).repeat(1, 1, 2)
        err = (de.qkv[:, :n].view(R, Hq + Hkv, D).double() - turned).abs()
        # (both roundings; the second's is of what the first has moved by up to 2^-8 of the pair)
        tol = pair * (2.0 ** -8 * (1 + 2.0 ** -8) + 2.0 ** -21) + szp * 132 * 2.0 ** -24 + turned.abs() * 2.0 ** -8 + pair * 2.0 ** -16
        assert bool((err <= tol).all())
        # the attention over the keys as the steps stored them
        k, v = de.qkv[:, Hq * D: n].view(R, Hkv, D), de.qkv[:, n:].view(R, Hkv, D)
        if dtype == torch.float8_e4m3fn:
            k, v = ((t.float() / 0.02).clamp(-448, 448).to(dtype).double() * float(cache.scales[0, 0]) for t in (k, v))
        keys.append((k.double().clone(), v.double().clone()))
        kk, vv = (torch.stack([t[i] for t in keys], 2).repeat_interleave(Hq // Hkv, 1) for i in (0, 1))      # [R][Hq][n][D]
        q = de.qkv[:, : Hq * D].view(R, Hq, D).double()
        p = torch.softmax(torch.einsum("rhd,rhnd->rhn", q, kk) * D ** -0.5, 2)
        ref = torch.einsum("rhn,rhnd->rhd", p, vv)
        tol = 2.0 ** -8 * ref.abs() + (2.0 ** -12 + 2.0 ** -18) * vv.abs().amax()
        assert bool(((dec.attn.double() - ref).abs() <= tol).all())
        # its codes, their projection, the residual stream and its norm
        ac, an = _rows(de.a, de.a_scales), dec.attn.double().flatten(1)
        step_size = de.a_scales.double().repeat_interleave(128, 1)[:, : Hq * D]
        assert bool(((ac - an).abs() <= an.abs() * (2.0 ** -4 + 2.0 ** -20) + step_size * 2.0 ** -10).all())
        w = _weights(de.out_codes, de.out_scales)
        _close(de.proj, ac @ w.t(), ac.abs() @ w.abs().t(), (128 + 2 + 5) * 2.0 ** -24, True)
        h = x.double() + de.proj.double()
        _close(dec.hidden, h, h.abs(), 2.0 ** -24, False)
        _close(de.hn, h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6), h.abs() * 0 + 1e-6, 1.0, True)
        assert bool(torch.isfinite(out).all())
    dec.check()


def test_dense_steps_are_near_those_in_bf16():
    """The same weights and inputs in 8 bits and in 16: weights and activations
    are each off by up to 2^-4 of themselves, at random, so a projection is by
    some 4 % of its own size; the residual stream stays exact."""
    R, Hq, Hkv, D = 33, 4, 2, 64
    outs = []
    for dense in ("bf16", "e4m3"):
        cfg, cache, dec = _decoder(R, Hq, Hkv, D, 16, dense=dense)
        g = torch.Generator(device="cuda").manual_seed(3)
        every, one = torch.arange(R, device="cuda"), torch.ones(R, dtype=torch.int32, device="cuda")
        for _ in range(5):
            x = torch.randn((R, cfg.d), generator=g, device="cuda")
            dec.step(x, every, one)
        outs.append((dec.hidden - x).double())
        dec.check()
    assert float((outs[0] - outs[1]).norm() / outs[0].norm()) < 0.15


def test_dense_step_captured_in_a_graph_goes_on_with_each_replay():
    R, Hq, Hkv, D, steps = 6, 4, 2, 64, 9
    x = torch.randn((steps, R, TINY.d), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    every, one = torch.arange(R, device="cuda"), torch.ones(R, dtype=torch.int32, device="cuda")
    _, _, eager = _decoder(R, Hq, Hkv, D, 16)
    want = [eager.step(x[t], every, one).clone() for t in range(steps)]
    _, cache, dec = _decoder(R, Hq, Hkv, D, 16)
    buf = x[0].clone()
    for t in range(2):
        buf.copy_(x[t])
        dec.step(buf, every, one)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dec.step(buf, every, one)
    for t in range(2, steps):
        buf.copy_(x[t])
        graph.replay()
        assert torch.equal(dec.out, want[t]), t
    assert cache.seq_len.tolist() == [steps] * R
    dec.check()


def test_dense_run_reports():
    from int4_expert_gemv_gb300 import paged
    r = paged.run(TINY, 3, 50, 6, Hq=4, Hkv=2, D=64, dense="e4m3")
    assert r["requests"] == 3 and r["us_per_step"] > 0 and 3 * 32 <= r["cached_tokens"] <= 3 * 56


def test_a_wait_that_runs_out_is_told():
    """A copy that never comes (the hook's): the call returns, its workspace says so, and the next calls run as ever."""
    from int4_expert_gemv_gb300 import build
    build.build()
    from int4_expert_gemv_gb300 import moe, paged
    for T in (1, 60, 300):
        w = torch.randn((256, 512), device="cuda")
        codes, scales, desc = paged.quantised(w)
        x = torch.randn((T, 512), device="cuda")
        xc, xs = torch.zeros((T, 512), dtype=torch.float8_e4m3fn, device="cuda"), torch.zeros((T, 4), device="cuda")
        moe.moe_quantise_e4m3(x, T, 512, xc, xs)
        ws = torch.zeros(moe.moe_scaled_product_workspace_bytes(desc, T), dtype=torch.uint8, device="cuda")
        out, ref = torch.zeros((T, 256), device="cuda"), torch.zeros((T, 256), device="cuda")
        moe.moe_scaled_product(desc, xc, xs, T, ref, ws)
        torch.cuda.synchronize()
        assert int(ws.view(torch.int32)[0]) == moe.MOE_OK
        try:
            moe.moe_debug_batched_waits(2_000_000, True)
            moe.moe_scaled_product(desc, xc, xs, T, out, ws)
            torch.cuda.synchronize()
        finally:
            moe.moe_debug_batched_waits(0, False)
        assert int(ws.view(torch.int32)[0]) == moe.MOE_ETIMEOUT
        ws.zero_()
        moe.moe_scaled_product(desc, xc, xs, T, out, ws)
        torch.cuda.synchronize()
        assert int(ws.view(torch.int32)[0]) == moe.MOE_OK and torch.equal(out, ref)


def test_a_decoder_tells_a_wait_that_ran_out():
    from int4_expert_gemv_gb300 import moe
    _, _, dec = _decoder(2, 4, 2, 64, 16)
    dec.check()
    dec.dense.ws[0] = moe.MOE_ETIMEOUT
    with pytest.raises(moe.MoEError):
        dec.check()
    dec.check()
