"""The operators around the expert layer's decode step, as a user calls them: the page plan of a paged key-value cache,
the append of new keys and values, the attention of one new token per request, and the routing by scores.

listed() names the measured cases, draw() gives more of the same ranges, prepare() makes what a caller holds before the
call, run() is one pass, in plain torch or (own = True) through the framework, exact() the values in 64 bits."""
import math
import random

import torch

own = False

BF16, F32, E4M3 = "bf16", "f32", "e4m3"
TORCH = {BF16: torch.bfloat16, F32: torch.float32, E4M3: torch.float8_e4m3fn}
SIZE = {BF16: 2, F32: 4, E4M3: 1}
E4M3_MAX = 448.0


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one scheduler step of 256 running requests: most add one token, some wait, some have ended and give their pages back
        dict(name="plan-step-256", op="plan", R=256, length=8192, page=16, new=1, ended=0.05, waits=0.05, room=256, mix=11),
        # a step that admits long prompts beside running requests, hundreds of thousands of new tokens with their slots and places
        dict(name="plan-admit-4096", op="plan", R=4096, length=32768, page=64, new=256, ended=0.02, waits=0.3, room=1 << 20, mix=12),
        # the new rows of 64 decoding requests, cut out of their fused projections, into an 8-bit cache
        dict(name="append-64-e4m3", op="append", N=64, Hq=32, Hkv=8, D=128, page=16, x=BF16, cache=E4M3, pages=1024, mix=21),
        # a long prompt's rows into a 16-bit cache; the token count is odd
        dict(name="append-65521-bf16", op="append", N=65521, Hq=16, Hkv=8, D=128, page=64, x=BF16, cache=BF16, pages=1100, mix=22),
        # one token's route: only latency
        dict(name="route-1", op="route", T=1, E=256, K=8, score="sigmoid", bias=True, groups=8, keep=4, best=2, renorm=True, factor=2.5, x=F32, mix=31),
        # a batch over the wide layer's 512 experts, softmax scores renormalised over the kept ones, 16-bit logits
        dict(name="route-4096-softmax", op="route", T=4096, E=512, K=4, score="softmax", bias=False, groups=1, keep=1, best=1, renorm=True, factor=1.0, x=BF16, mix=32),
        # a long prompt's routes with balance bias and groups
        dict(name="route-65521", op="route", T=65521, E=256, K=8, score="sigmoid", bias=True, groups=8, keep=4, best=2, renorm=True, factor=2.5, x=F32, mix=33),
        # one request in fp32, two key heads of 256: the smallest call of a decoder, latency and the split over the length
        dict(name="attend-1x2011", op="attend", B=1, length=2011, ragged=False, Hq=16, Hkv=2, D=256, page=16, q=F32, cache=BF16, window=0, mix=41),
        # 64 requests of every length up to 8192, four query heads to a key head
        dict(name="attend-64-ragged", op="attend", B=64, length=8192, ragged=True, Hq=32, Hkv=8, D=128, page=16, q=BF16, cache=BF16, window=0, mix=42),
        # two long contexts: few rows, a long axis
        dict(name="attend-2x130977", op="attend", B=2, length=130977, ragged=False, Hq=64, Hkv=8, D=128, page=64, q=BF16, cache=BF16, window=0, mix=43),
        # a full batch over an 8-bit cache
        dict(name="attend-96-e4m3", op="attend", B=96, length=16384, ragged=True, Hq=32, Hkv=8, D=128, page=32, q=BF16, cache=E4M3, window=0, mix=44),
        # a sliding window, a head size and a page size that are no power of two, one query head to a key head
        dict(name="attend-29-window", op="attend", B=29, length=6001, ragged=True, Hq=12, Hkv=12, D=80, page=24, q=F32, cache=BF16, window=1000, mix=45),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        case = _draw(rng)
        sizes = [v for v in case.values() if isinstance(v, int) and not isinstance(v, bool)]
        sizes += [case[h] * case["D"] for h in ("Hq", "Hkv") if h in case]
        if 3 * 1024 not in sizes:
            return case


def _draw(rng):
    op = rng.choice(["plan", "append", "route", "route", "attend", "attend", "attend"])
    mix = rng.randrange(1, 1 << 20)
    if op == "plan":
        R = _log(rng, 1, 4096)
        new = _log(rng, 1, max(1, min(4096, 500000 // R)))
        length = _log(rng, 16, 32768)
        return dict(op=op, R=R, length=length, page=rng.choice([1 if R * length < 1 << 20 else 16, 8, 16, 24, 32, 64, 128]), new=new,
                    ended=rng.choice([0.0, 0.1]), waits=rng.choice([0.0, 0.3]), room=R * (2 * new - 1) + rng.randrange(0, 300), mix=mix)
    if op == "append":
        D, Hkv, G = rng.choice([64, 80, 96, 128, 192, 256]), rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 2, 4, 5, 8])
        cache = rng.choice([BF16, E4M3])
        N = _log(rng, 1, max(1, min(65521, (1 << 27) // (2 * Hkv * D))))
        page = rng.choice([8, 16, 24, 32, 64, 128])
        return dict(op=op, N=N, Hq=Hkv * G, Hkv=Hkv, D=D, page=page, x=rng.choice([BF16, F32]), cache=cache, pages=N // page + rng.randrange(2, 80), mix=mix)
    if op == "route":
        E = rng.choice([16, 60, 64, 128, 160, 256, 384, 512])
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0 and E // g >= 2])
        keep = rng.randrange(1, groups + 1)
        K = rng.randrange(1, min(16, keep * (E // groups)) + 1)
        T = _log(rng, 1, min(65521, (1 << 24) // E))
        return dict(op=op, T=T, E=E, K=K, score=rng.choice(["sigmoid", "softmax"]), bias=rng.random() < 0.6, groups=groups, keep=keep,
                    best=rng.choice([1, 2]), renorm=rng.random() < 0.7, factor=rng.choice([1.0, 2.5]), x=rng.choice([F32, BF16]), mix=mix)
    D, Hkv, G = rng.choice([64, 80, 96, 128, 128, 192, 256]), rng.choice([1, 2, 4, 8, 12]), rng.choice([1, 2, 3, 4, 6, 7, 8, 12, 16, 20])
    cache = rng.choice([BF16, BF16, E4M3])
    B = _log(rng, 1, 256)
    most = min(131071, (1 << (28 if G <= 8 else 27)) // (B * Hkv * D))  # numbers in the keys of the padded batch
    length = _log(rng, 1, max(1, most))
    window = _log(rng, 1, length) if rng.random() < 0.25 else 0
    return dict(op=op, B=B, length=length, ragged=rng.random() < 0.7, Hq=Hkv * G, Hkv=Hkv, D=D, page=rng.choice([8, 16, 16, 24, 32, 64, 128]),
                q=rng.choice([BF16, F32]), cache=cache, window=window, mix=mix)


def _lengths(case):
    """The requests' lengths: the same for every seed, as work() goes by them."""
    r = random.Random(case["mix"])
    B, L = case["B"], case["length"]
    if not case["ragged"]:
        return [L] * B
    n = [r.randint(1, L) for _ in range(B)]
    n[r.randrange(B)] = L
    if B > 4:
        n[-2] = 0  # a request that waits: an empty row
        n[-1] = 1
    return n


def _requests(case):
    """Lengths and new tokens of a scheduler step; -1 new tokens: the request has ended."""
    r = random.Random(case["mix"])
    seq, new, room = [], [], case["room"]
    for _ in range(case["R"]):
        seq.append(r.randint(0, case["length"]))
        x = r.random()
        if x < case["ended"]:
            new.append(-1)
        elif x < case["ended"] + case["waits"]:
            new.append(0)
        else:
            new.append(min(room, r.randint(1, 2 * case["new"] - 1)))
            room -= new[-1]
    return seq, new


def _blocks(n, page):
    return -(-n // page)


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"plan": _prepare_plan, "append": _prepare_append, "route": _prepare_route, "attend": _prepare_attend}[case["op"]](case, g)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _prepare_plan(case, g):
    seq, new = _requests(case)
    page, R = case["page"], case["R"]
    have = [_blocks(s, page) for s in seq]
    after = [_blocks(s + max(n, 0), page) for s, n in zip(seq, new)]
    width = max(1, max(after))
    need = sum(a - h for a, h in zip(after, have))
    pages = sum(have) + need + 77
    perm = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)
    table = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
    held = sum(have)
    table[torch.arange(width, device="cuda")[None, :] < _ints(have)[:, None]] = perm[:held]
    free = pages - held
    head = pages - free // 2  # the ring's free part wraps round its end
    ring = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    ring[(head + torch.arange(free, device="cuda")) % pages] = perm[held:]
    room, dev = case["room"], dict(dtype=torch.int32, device="cuda")
    return dict(case=case, seq=_ints(seq), new=_ints(new), table=table, ring=ring, pool=_ints([head % pages, free]), pages=pages,
                seq_out=torch.empty(R, **dev), first=torch.empty(R + 1, **dev), slots=torch.empty(room, **dev), places=torch.empty(room, **dev),
                pool_out=torch.empty(2, **dev), status=torch.empty(1, **dev))


def _scales(case, g):
    if case["cache"] != E4M3:
        return None, None
    k = (4.0 / E4M3_MAX) * (0.75 + 0.5 * torch.rand(case["Hkv"], generator=g, device="cuda"))
    v = (4.0 / E4M3_MAX) * (0.75 + 0.5 * torch.rand(case["Hkv"], generator=g, device="cuda"))
    return k, v


def _cache(case, pages, g):
    """A pool of pages, each [2][Hkv][page][D]: keys, then values. In 8 bits the numbers are in units of a scale per head."""
    kv = torch.empty((pages, 2, case["Hkv"], case["page"], case["D"]), dtype=torch.bfloat16, device="cuda")
    kv.normal_(generator=g)
    if case["cache"] == E4M3:
        kv = kv.mul_(E4M3_MAX / 4.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return kv


def _prepare_append(case, g):
    N, Hq, Hkv, D, page, pages = (case[k] for k in ("N", "Hq", "Hkv", "D", "page", "pages"))
    qkv = torch.randn((N, (Hq + 2 * Hkv) * D), generator=g, device="cuda").to(TORCH[case["x"]])
    ks, vs = _scales(case, g)
    kv = _cache(case, pages, g)
    slots = torch.randperm(pages * page, generator=g, device="cuda", dtype=torch.int32)[:N].clone()
    slots[N // 2 :: 97] = -1  # padding
    return dict(case=case, qkv=qkv, k=qkv[:, Hq * D : (Hq + Hkv) * D], v=qkv[:, (Hq + Hkv) * D :], slots=slots, kv=kv, ks=ks, vs=vs)


def _prepare_route(case, g):
    T, E = case["T"], case["E"]
    z = 1.5 * torch.randn((T, E), generator=g, device="cuda")
    bias = 0.05 * torch.randn(E, generator=g, device="cuda") if case["bias"] else None
    z = z.to(TORCH[case["x"]])
    for _ in range(20):  # rows with a choice that 32 bits cannot settle are drawn again; equal logits stay and go by index
        near = _undecided(case, z, bias)
        n = int(near.sum())
        if not n:
            break
        z[near] = (1.5 * torch.randn((n, E), generator=g, device="cuda")).to(z.dtype)
    dev = dict(device="cuda")
    return dict(case=case, z=z, bias=bias, idx=torch.empty((T, case["K"]), dtype=torch.int32, **dev), w=torch.empty((T, case["K"]), **dev))


def _undecided(case, z, bias):
    """Rows in which two neighbours of an order that counts are nearer than 32-bit scores tell apart, but not equal."""
    T, E, n = case["T"], case["E"], case["groups"]
    z = z.double()
    c = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.softmax(z, 1)
    if bias is not None:
        c = c + bias.double()
    size = c.abs().amax(1, keepdim=True)
    gap = lambda x: x[:, :-1] - x[:, 1:]  # noqa: E731
    near = lambda d: ((d > 0) & (d < 2e-6 * size)).any(1)  # noqa: E731
    bad = torch.zeros(T, dtype=torch.bool, device=z.device)
    if n > 1:
        s = c.view(T, n, E // n).sort(2, descending=True).values[:, :, : case["best"]].sum(2).sort(1, descending=True)
        bad |= near(gap(s.values))
        off = torch.ones((T, n), dtype=torch.bool, device=z.device).scatter_(1, s.indices[:, : case["keep"]], False)
        c = c.view(T, n, E // n).masked_fill(off[:, :, None], -9.0).view(T, E)
    top = c.sort(1, descending=True).values[:, : case["K"] + 1]
    return bad | near(gap(top))


def _prepare_attend(case, g):
    n = _lengths(case)
    B, page = case["B"], case["page"]
    nb = [_blocks(x, page) for x in n]
    width, pages = max(1, max(nb)), sum(nb) + 5
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    perm = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)
    table[torch.arange(width, device="cuda")[None, :] < _ints(nb)[:, None]] = perm[: sum(nb)]
    ks, vs = _scales(case, g)
    kv = _cache(case, pages, g)
    q = torch.randn((B, case["Hq"], case["D"]), generator=g, device="cuda").to(TORCH[case["q"]])
    return dict(case=case, q=q, kv=kv, ks=ks, vs=vs, table=table, seq=_ints(n), scale=case["D"] ** -0.5,
                out=torch.empty_like(q), lse=torch.empty((B, case["Hq"]), device="cuda"))


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"plan": _own_plan, "append": _own_append, "route": _own_route, "attend": _own_attend}[op](state)
    return {"plan": _plain_plan, "append": _plain_append, "route": _plain_route, "attend": _plain_attend}[op](state)


def _plain_plan(s):
    case, page, room = s["case"], s["case"]["page"], s["case"]["room"]
    seq, new, table, ring, P = s["seq"].long(), s["new"].long(), s["table"], s["ring"], s["pages"]
    head, free = s["pool"][0].long(), s["pool"][1].long()
    add = new.clamp(min=0)
    have = (seq + page - 1) // page
    need = (seq + add + page - 1) // page - have
    gone = torch.where(new < 0, have, 0)
    before = lambda x: torch.cumsum(x, 0) - x  # noqa: E731
    of = lambda x: torch.repeat_interleave(torch.arange(case["R"], device=x.device), x)  # noqa: E731
    # new blocks out of the ring, ended requests' pages behind its free part
    r = of(need)
    j = torch.arange(len(r), device=r.device)
    table[r, have[r] + j - before(need)[r]] = ring[(head + j) % P]
    r = of(gone)
    j = torch.arange(len(r), device=r.device)
    ring[(head + free + j) % P] = table[r, j - before(gone)[r]]
    # slots and places of the new tokens
    r = of(add)
    n = len(r)
    at = seq[r] + torch.arange(n, device=r.device) - before(add)[r]
    slots = torch.full((room,), -1, dtype=torch.int32, device=r.device)
    places = torch.zeros(room, dtype=torch.int32, device=r.device)
    slots[:n] = table[r, at // page] * page + (at % page).int()
    places[:n] = at.int()
    first = torch.cat([torch.zeros_like(add[:1]), torch.cumsum(add, 0)])
    used = need.sum()
    pool = torch.stack([(head + used) % P, free - used + gone.sum()])
    return dict(table=table, ring=ring, seq=torch.where(new < 0, 0, seq + add).int(), first=first.int(), slots=slots, places=places,
                pool=pool.int(), status=torch.zeros_like(s["status"]))


def _plain_append(s):
    case, kv = s["case"], s["kv"]
    N, Hkv, D, page = s["case"]["N"], case["Hkv"], case["D"], case["page"]
    keep = s["slots"] >= 0
    at = s["slots"][keep].long()

    def stored(x, scale):
        x = x.reshape(N, Hkv, D)[keep].float()
        return x.to(kv.dtype) if scale is None else (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(kv.dtype)

    bits = kv.view(torch.uint8) if kv.dtype == torch.float8_e4m3fn else kv
    bits[at // page, 0, :, at % page] = stored(s["k"], s["ks"]).view(bits.dtype)
    bits[at // page, 1, :, at % page] = stored(s["v"], s["vs"]).view(bits.dtype)
    return kv


def _plain_route(s):
    case, T, E, n, K = s["case"], s["case"]["T"], s["case"]["E"], s["case"]["groups"], s["case"]["K"]
    z = s["z"].float()
    if case["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-z))
    else:
        e = torch.exp(z - z.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    c = score if s["bias"] is None else score + s["bias"]
    if n > 1:
        best = c.view(T, n, E // n).sort(2, descending=True).values[:, :, : case["best"]].sum(2)
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, : case["keep"]]
        off = torch.ones((T, n), dtype=torch.bool, device=z.device).scatter_(1, kept, False)
        c = c.view(T, n, E // n).masked_fill(off[:, :, None], -math.inf).view(T, E)
    idx = c.sort(dim=1, descending=True, stable=True).indices[:, :K]
    w = score.gather(1, idx)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return dict(idx=idx.int(), w=w * case["factor"])


def _plain_attend(s):
    case, B, Hq, Hkv, D = s["case"], s["case"]["B"], s["case"]["Hq"], s["case"]["Hkv"], s["case"]["D"]
    pages = s["kv"][s["table"].clamp(min=0)]  # [B, blocks, 2, Hkv, page, D]
    L = pages.shape[1] * case["page"]
    k = pages[:, :, 0].transpose(1, 2).reshape(B, Hkv, L, D).float()
    v = pages[:, :, 1].transpose(1, 2).reshape(B, Hkv, L, D).float()
    del pages
    if s["ks"] is not None:
        k, v = k * s["ks"][:, None, None], v * s["vs"][:, None, None]
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    at, n = torch.arange(L, device=q.device), s["seq"][:, None]
    seen = (at < n) if not case["window"] else (at < n) & (at >= n - case["window"])
    seen = seen[:, None, None, :]
    m = x.masked_fill(~seen, -math.inf).amax(3, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.where(seen, torch.exp(x - m), 0.0)
    total = p.sum(3, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    lse = m + torch.log(total)  # an empty row: minus infinity
    return dict(out=out.view(B, Hq, D).to(s["q"].dtype), lse=lse.view(B, Hq))


# ---------------------------------------------------------------- the framework's calls
def _kv_desc(moe, s):
    case, kv = s["case"], s["kv"]
    half = case["Hkv"] * case["page"] * case["D"] * SIZE[case["cache"]]
    at = lambda x: None if x is None else x.data_ptr()  # noqa: E731
    kind = moe.MOE_DTYPE_E4M3 if case["cache"] == E4M3 else moe.MOE_DTYPE_BF16
    return moe.KVDesc(n_pages=kv.shape[0], page=case["page"], Hkv=case["Hkv"], D=case["D"], dtype=kind, k=kv.data_ptr(),
                      v=kv.data_ptr() + half, page_stride=2 * half, k_scale=at(s["ks"]), v_scale=at(s["vs"]))


def _own_plan(s):
    from int4_expert_gemv_gb300 import moe
    c = s["case"]
    moe.moe_kv_plan(s["seq"], s["new"], c["R"], s["table"], s["table"].shape[1], c["page"], s["ring"], s["pages"], s["pool"], s["seq_out"],
                    s["first"], s["slots"], s["places"], c["room"], s["pool_out"], s["status"])
    return dict(table=s["table"], ring=s["ring"], seq=s["seq_out"], first=s["first"], slots=s["slots"], places=s["places"], pool=s["pool_out"],
                status=s["status"])


def _own_append(s):
    from int4_expert_gemv_gb300 import moe
    if "desc" not in s:
        s["desc"] = _kv_desc(moe, s)
    moe.moe_kv_append(s["desc"], s["k"], s["v"], s["slots"], s["case"]["N"])
    return s["kv"]


def _own_route(s):
    from int4_expert_gemv_gb300 import moe
    c = s["case"]
    if "desc" not in s:
        kind = moe.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else moe.MOE_SCORE_SOFTMAX
        s["desc"] = moe.RouteDesc(E=c["E"], K=c["K"], score=kind, n_group=c["groups"], keep_group=c["keep"], group_best=c["best"],
                                  renorm=int(c["renorm"]), factor=c["factor"], bias=None if s["bias"] is None else s["bias"].data_ptr())
    moe.moe_scored_route(s["desc"], s["z"], c["T"], s["idx"], s["w"])
    return dict(idx=s["idx"], w=s["w"])


def _own_attend(s):
    from int4_expert_gemv_gb300 import moe
    c = s["case"]
    if "desc" not in s:
        s["desc"] = _kv_desc(moe, s)
        s["ws"] = torch.empty(moe.moe_paged_attention_workspace_bytes(s["desc"], c["B"], c["Hq"]), dtype=torch.uint8, device="cuda")
    moe.moe_paged_attention(s["desc"], s["q"], c["B"], c["Hq"], s["seq"], s["table"], s["table"].shape[1], s["scale"], s["out"], s["ws"],
                            lse=s["lse"], window=c["window"])
    return dict(out=s["out"], lse=s["lse"])


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "plan":
        seq, new = _requests(case)
        page = case["page"]
        need = sum(_blocks(s + n, page) - _blocks(s, page) for s, n in zip(seq, new) if n > 0)
        gone = sum(_blocks(s, page) for s, n in zip(seq, new) if n < 0)
        part = sum(s % page != 0 for s, n in zip(seq, new) if n > 0)  # pages that new tokens fill up
        return {"bytes": 4 * (4 * case["R"] + 2 * case["room"] + 2 * need + 2 * gone + part), "flops": sum(n for n in new if n > 0)}
    if case["op"] == "append":
        n = 2 * case["N"] * case["Hkv"] * case["D"]
        return {"bytes": n * (SIZE[case["x"]] + SIZE[case["cache"]]) + 4 * case["N"], "flops": n if case["cache"] == E4M3 else 0}
    if case["op"] == "route":
        n = case["T"] * case["E"]
        return {"bytes": n * SIZE[case["x"]] + 8 * case["T"] * case["K"] + 4 * case["E"] * case["bias"], "flops": 4 * n}
    seen = sum(min(n, case["window"] or n) for n in _lengths(case))
    rows = case["B"] * case["Hq"]
    return {"bytes": seen * 2 * case["Hkv"] * case["D"] * SIZE[case["cache"]] + 2 * rows * case["D"] * SIZE[case["q"]] + 4 * rows
            + 4 * _blocks(seen, case["page"]), "flops": 4 * seen * case["Hq"] * case["D"]}


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    if case["op"] == "route":
        return _exact_route(case, prepare(case, seed))
    if case["op"] == "attend":
        return _exact_attend(case, prepare(case, seed))
    if case["op"] == "append":
        return _exact_append(case, prepare(case, seed))
    return None  # whole numbers


def _exact_append(case, s):
    """Head by head: the pool with the rows that have a slot in their places, before they are rounded to the cache's type."""
    kv, D = s["kv"].double(), case["D"]
    rows = torch.nonzero(s["slots"] != -1)[:, 0]
    page = torch.div(s["slots"][rows].long(), case["page"], rounding_mode="floor")
    inside = s["slots"][rows].long() - page * case["page"]
    for part, (x, scale) in enumerate([(s["k"], s["ks"]), (s["v"], s["vs"])]):
        for h in range(case["Hkv"]):
            new = x[rows, h * D : (h + 1) * D].double()
            if scale is not None:
                new = torch.clip(new / scale[h].double(), -E4M3_MAX, E4M3_MAX)
            kv[page, part, h, inside] = new
    return kv


def _exact_route(case, s):
    """Expert by expert of a row's choice: the best of what is left, K times."""
    T, E, n = case["T"], case["E"], case["groups"]
    z = s["z"].double()
    score = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
    left = score + (s["bias"].double() if s["bias"] is not None else 0.0)
    rows = torch.arange(T, device=z.device)
    first = lambda x: (x == x.amax(1, keepdim=True)).int().argmax(1)  # noqa: E731  the lowest index of the largest
    if n > 1:
        per = left.view(T, n, E // n)
        total = torch.topk(per, case["best"], dim=2).values.sum(2)
        allowed = torch.zeros((T, n), dtype=torch.bool, device=z.device)
        for _ in range(case["keep"]):
            i = first(total)
            allowed[rows, i] = True
            total[rows, i] = -math.inf
        left = torch.where(allowed[:, :, None], per, -math.inf).reshape(T, E)
    w = []
    for _ in range(case["K"]):
        i = first(left)
        w.append(score[rows, i])
        left[rows, i] = -math.inf
    w = torch.stack(w, 1)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return dict(idx=None, w=case["factor"] * w)


def _exact_attend(case, s):
    """Request by request, over the keys that it sees and no others."""
    B, Hq, Hkv, D, page = (case[k] for k in ("B", "Hq", "Hkv", "D", "page"))
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(case)):
        if n == 0:
            continue
        at = torch.arange(max(0, n - case["window"]) if case["window"] else 0, n, device="cuda")
        pages, inside = s["table"][b].long()[at // page], at % page
        for h in range(Hkv):
            k, v = s["kv"][pages, 0, h, inside].double(), s["kv"][pages, 1, h, inside].double()
            if s["ks"] is not None:
                k, v = k * s["ks"][h].double(), v * s["vs"][h].double()
            rows = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            x = s["scale"] * (s["q"][b, rows].double() @ k.T)
            lse[b, rows] = torch.logsumexp(x, 1)
            out[b, rows] = torch.softmax(x, 1) @ v
    return dict(out=out, lse=lse)
