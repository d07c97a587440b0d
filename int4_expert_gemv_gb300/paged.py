"""A decoder layer around the expert FFN: paged key-value cache, attention of
one new token per request, routing by scores.

PagedCache holds one layer's pages and a batch's block tables and runs the
page plan of each step; PagedDecoder runs whole decode steps of one layer:

  plan      moe_kv_plan: pages, slots and places of the step's new tokens
  project   q, k, v of the normalised input (plain matrix products), turned by
            their places (rotary embedding)
  append    moe_kv_append: k and v into the cache
  attend    moe_paged_attention: every request over its own pages
  route     moe_prerouter_head with H = 0 (the layer's own router), then
            moe_scored_route (sigmoid scores, balance bias, groups)
  experts   moe_expert_ffn_int4, moe_combine_residual

The pages this framework follows predict the route a token ahead
(moe_prerouter_head, moe_topk_route); this is the layer of a model that routes
by scores instead, as far as the expert FFN's own calls go.  Weights are
seeded and random.

  python -m int4_expert_gemv_gb300.paged [--requests 64] [--length 4096] ...
runs steps of it and prints what a step takes.
"""
from __future__ import annotations

import torch

from . import moe
from .configs import ALL, MoEConfig
from .model import DeviceModel


class PagedCache:
    """Pages of one layer ([n_pages][2][Hkv][page][D]: a page's keys, then its
    values) and the block tables of R requests.  plan() is one scheduler step.
    The call does not write what it reads (lengths, free pages), so the new
    state is copied over the old one behind it: all addresses stay, and a
    captured step moves on with each replay."""

    def __init__(self, R: int, n_pages: int, page: int, Hkv: int, D: int, max_blocks: int,
                 max_new: int, dtype=torch.bfloat16, scale: float | None = None, device="cuda"):
        self.R, self.n_pages, self.page, self.max_blocks, self.max_new = R, n_pages, page, max_blocks, max_new
        i32 = dict(dtype=torch.int32, device=device)
        self.kv = torch.zeros((n_pages, 2, Hkv, page, D), dtype=dtype, device=device)
        e4m3 = dtype == torch.float8_e4m3fn
        self.scales = torch.full((2, Hkv), scale or 1.0, device=device) if e4m3 else None
        half = Hkv * page * D * self.kv.element_size()
        self.desc = moe.KVDesc(n_pages=n_pages, page=page, Hkv=Hkv, D=D,
                               dtype=moe.MOE_DTYPE_E4M3 if e4m3 else moe.MOE_DTYPE_BF16,
                               k=self.kv.data_ptr(), v=self.kv.data_ptr() + half, page_stride=2 * half,
                               k_scale=self.scales[0].data_ptr() if e4m3 else None,
                               v_scale=self.scales[1].data_ptr() if e4m3 else None)
        self.table = torch.full((R, max_blocks), -1, **i32)
        self.ring = torch.arange(n_pages, **i32)
        self._state, self._after = torch.zeros(R + 2, **i32), torch.zeros(R + 2, **i32)
        self.lengths, self.pool = self._state[:R], self._state[R:]   # pool: the first free page's place, their count
        self._lengths_after, self._pool_after = self._after[:R], self._after[R:]
        self.pool[1] = n_pages
        self.first = torch.zeros(R + 1, **i32)
        self.slots = torch.zeros(max_new, **i32)
        self.places = torch.zeros(max_new, **i32)
        self.status = torch.zeros(1, **i32)          # of the last plan
        self.worst = torch.zeros(1, **i32)           # of all plans since check()

    @property
    def seq_len(self) -> torch.Tensor:
        """Tokens of each request in the cache, those of the last plan included."""
        return self.lengths

    def plan(self, new_len: torch.Tensor, most: int | None = None) -> None:
        """new_len int32 [R] on the device: tokens that each request adds, -1
        for one that has ended; `most`: of all together, at most max_new (the
        places there are in `slots` and `places`, all of which the call
        writes).  A plan that does not fit changes nothing and gives no slots:
        self.status tells, and check() for all plans since the last check."""
        most = self.max_new if most is None else most
        if not 0 <= most <= self.max_new:
            raise ValueError(f"at most {most} new tokens in a cache with places for {self.max_new}")
        if (new_len.dtype != torch.int32 or new_len.numel() < self.R or not new_len.is_contiguous()
                or new_len.device != self.table.device):
            raise ValueError(f"new_len: int32 [{self.R}] on {self.table.device} needed, got {new_len.dtype} "
                             f"{tuple(new_len.shape)} on {new_len.device}")
        moe.moe_kv_plan(self.lengths, new_len, self.R, self.table, self.max_blocks, self.page,
                        self.ring, self.n_pages, self.pool, self._lengths_after, self.first,
                        self.slots, self.places, most, self._pool_after, self.status)
        self._state.copy_(self._after)
        torch.maximum(self.worst, self.status, out=self.worst)

    def check(self) -> None:
        """Waits for the GPU; raises MoEError if a plan since the last check did
        not fit (its tokens are in no slot, and steps over it ran on the keys
        that were there)."""
        worst = int(self.worst[0])
        self.worst.zero_()
        if worst != moe.MOE_OK:
            raise moe.MoEError(worst, "moe_kv_plan", "a step's tokens did not fit")

    def append(self, k: torch.Tensor, v: torch.Tensor) -> None:
        """k, v [N][Hkv * D] of the plan's new tokens, in order of requests."""
        n, row = k.shape[0], self.desc.Hkv * self.desc.D
        if n > self.max_new:
            raise ValueError(f"{n} tokens for {self.max_new} slots")
        if k.numel() != n * row or v.shape[0] != n or v.numel() != n * row:
            raise ValueError(f"k and v: [N][{row}] needed, got {tuple(k.shape)} and {tuple(v.shape)}")
        moe.moe_kv_append(self.desc, k, v, self.slots, n)


def rotate(x: torch.Tensor, places: torch.Tensor) -> torch.Tensor:
    """Rotary embedding: pairs (i, i + D/2) of x [T][H][D] turned by place * 10000^(-2i/D)."""
    D = x.shape[-1]
    freq = torch.exp(torch.arange(0, D, 2, device=x.device) * (-9.210340371976184 / D))
    angle = places[:, None].float() * freq
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    a, b = x[..., : D // 2].float(), x[..., D // 2:].float()
    return torch.cat([a * c - b * s, b * c + a * s], -1).to(x.dtype)


class PagedDecoder:
    """Decode steps of one layer over a batch of R requests (bf16 activations,
    fp32 residual stream)."""

    def __init__(self, model: DeviceModel, cache: PagedCache, Hq: int, layer: int = 0, seed: int = 0,
                 n_group: int = 8, keep_group: int = 4, factor: float = 2.5):
        self.m, self.cache, self.Hq = model, cache, Hq
        c, dev, R = model.cfg, model.device, cache.R
        self.cfg, self.ly = c, model.layers[layer]
        self.Hkv, self.D = cache.desc.Hkv, cache.desc.D
        g = torch.Generator(device=dev).manual_seed(seed)
        n = (Hq + 2 * self.Hkv) * self.D
        w = lambda i, o: (torch.randn((i, o), generator=g, device=dev) * i ** -0.5).bfloat16()  # noqa: E731
        self.w_qkv, self.w_out = w(c.d, n), w(Hq * self.D, c.d)
        self.bias = 0.02 * torch.randn(c.E, generator=g, device=dev)
        self.route = moe.RouteDesc(E=c.E, K=c.K, score=moe.MOE_SCORE_SIGMOID, n_group=n_group,
                                   keep_group=keep_group, group_best=min(2, c.E // n_group),
                                   renorm=1, factor=factor, bias=self.bias.data_ptr())
        f32, bf = dict(dtype=torch.float32, device=dev), dict(dtype=torch.bfloat16, device=dev)
        self.attn = torch.zeros((R, Hq, self.D), **bf)
        self.logits, self.w = torch.zeros((R, c.E), **f32), torch.zeros((R, c.K), **f32)
        self.idx = torch.zeros((R, c.K), dtype=torch.int32, device=dev)
        self.y = torch.zeros((R, c.slots, c.d), **f32)
        self.out, self.x_next = torch.zeros((R, c.d), **f32), torch.zeros((R, c.d), **f32)
        u8 = lambda b: torch.empty(max(256, b), dtype=torch.uint8, device=dev)  # noqa: E731
        self.attn_ws = u8(moe.moe_paged_attention_workspace_bytes(cache.desc, R, Hq))
        self.head_ws = u8(moe.moe_prerouter_head_workspace_bytes(self.ly["router_desc"], R))
        self.ffn_ws = u8(moe.moe_expert_ffn_workspace_bytes(self.ly["experts_desc"], R, c.K))

    def step(self, x: torch.Tensor, rows: torch.Tensor, new_len: torch.Tensor) -> torch.Tensor:
        """One token for each of the requests in `rows` (int64, ascending; the
        ones whose new_len is 1; at most the cache's max_new).  x fp32 [R][d]: the residual stream; the
        result is the layer's, valid in those rows.  Nothing here waits for
        the GPU, and a step captured in a graph can be replayed: each replay is
        one step more.  Whether all steps' tokens had room tells the cache's
        check(), to be asked before their results are used."""
        ca, c, R = self.cache, self.cfg, self.cache.R
        if rows.numel() > ca.max_new:
            raise ValueError(f"{rows.numel()} tokens in a step of a cache with places for {ca.max_new}")
        ca.plan(new_len, min(R, ca.max_new))
        xn = (x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)).bfloat16()
        qkv = xn @ self.w_qkv
        q = qkv[:, : self.Hq * self.D].view(R, self.Hq, self.D)
        at = (ca.seq_len - 1).clamp(min=0)
        q = rotate(q, at)
        k = rotate(qkv[:, self.Hq * self.D: (self.Hq + self.Hkv) * self.D].view(R, self.Hkv, self.D), at)
        ca.append(k[rows].flatten(1), qkv[rows, (self.Hq + self.Hkv) * self.D:])
        moe.moe_paged_attention(ca.desc, q, R, self.Hq, ca.seq_len, ca.table, ca.max_blocks,
                                self.D ** -0.5, self.attn, self.attn_ws)
        h = x + (self.attn.flatten(1) @ self.w_out).float()
        hn = (h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6)).bfloat16()
        moe.moe_prerouter_head(self.ly["router_desc"], hn, None, None, c.K, R, self.logits, self.head_ws)
        moe.moe_scored_route(self.route, self.logits, R, self.idx, self.w)
        moe.moe_expert_ffn_int4(self.ly["experts_desc"], hn, self.idx, R, c.K, self.y, self.ffn_ws)
        moe.moe_combine_residual(self.y, self.w, R, c.K, c.shared, c.d, h, self.out, self.x_next)
        self.hidden = h
        return self.out


def run(cfg: MoEConfig, R: int, length: int, steps: int, Hq: int = 16, Hkv: int = 2, D: int = 128,
        page: int = 16, dtype=torch.bfloat16) -> dict:
    """Requests of up to `length` cached tokens (random), `steps` decode steps
    of one layer, the first three of them untimed where there are more; the
    time of a step in microseconds."""
    if steps < 1:
        raise ValueError(f"steps={steps}")
    timed = max(1, steps - 3)
    model = DeviceModel(cfg, heads=False)
    blocks = (length + steps + 2 * page) // page
    cache = PagedCache(R, R * blocks, page, Hkv, D, blocks, max(R, R * length), dtype, scale=0.01)
    dec = PagedDecoder(model, cache, Hq)
    g = torch.Generator(device="cuda").manual_seed(1)
    have = torch.randint(length // 2 + 1, length + 1, (R,), generator=g, device="cuda", dtype=torch.int32)
    cache.plan(have)
    n = int(have.sum())
    for a in range(0, n, 8192):                       # the prompts' keys and values, a piece at a time
        b = min(n, a + 8192)
        kv = torch.randn((2, b - a, Hkv * D), generator=g, device="cuda").bfloat16()
        moe.moe_kv_append(cache.desc, kv[0], kv[1], cache.slots[a:b], b - a)
    x = torch.randn((R, cfg.d), generator=g, device="cuda")
    rows, one = torch.arange(R, device="cuda"), torch.ones(R, dtype=torch.int32, device="cuda")
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    for _ in range(steps - timed):
        dec.step(x, rows, one)
    ev[0].record()
    for _ in range(timed):
        x = dec.step(x, rows, one).clone()
    ev[1].record()
    torch.cuda.synchronize()
    cache.check()
    return {"requests": R, "cached_tokens": int(cache.seq_len.sum()),
            "us_per_step": ev[0].elapsed_time(ev[1]) * 1e3 / timed}


if __name__ == "__main__":
    import argparse
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--config", default="batched-T64")
    ap.add_argument("--requests", type=int, default=64)
    ap.add_argument("--length", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--e4m3", action="store_true", help="an 8-bit cache")
    a = ap.parse_args()
    print(run(ALL[a.config], a.requests, a.length, a.steps,
              dtype=torch.float8_e4m3fn if a.e4m3 else torch.bfloat16))
