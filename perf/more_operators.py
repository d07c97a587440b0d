"""The dense half of a decoder layer in 8-bit floating point, as a user calls it: the root-mean-square norm with the
residual's addition and an output in 8 bits, the quantisation of rows and of weights by blocks, the matrix product of
such numbers with a scale for each block of 128, and the rotary embedding of queries and keys.

listed() names the measured cases, draw() gives more of the same ranges, prepare() makes what a caller holds before the
call, run() is one pass, in plain torch or (own = True) through the framework, exact() the values in 64 bits."""
import math

import torch

own = False

BF16, F32, E4M3 = "bf16", "f32", "e4m3"
TORCH = {BF16: torch.bfloat16, F32: torch.float32, E4M3: torch.float8_e4m3fn}
SIZE = {BF16: 2, F32: 4, E4M3: 1}
E4M3_MAX = 448.0
LEAST = 2.0 ** -100  # the smallest scale
BLOCK = 128


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token's last norm: only latency
        dict(name="norm-1", op="norm", T=1, d=2048, x=F32, res="", weight=F32, y=BF16, pow2=False),
        # a decode step of 64 requests: the projection added to the fp32 residual stream, the next projection's input in 8 bits
        dict(name="norm-64-e4m3", op="norm", T=64, d=2048, x=BF16, res=F32, weight=BF16, y=E4M3, pow2=False),
        # a long prompt of the wide layer, 16-bit residual, scales that are powers of two
        dict(name="norm-8191-e4m3", op="norm", T=8191, d=4096, x=BF16, res=BF16, weight=BF16, y=E4M3, pow2=True),
        # the attention's outputs of a long prompt, a scale for each row's 128 numbers
        dict(name="quant-16381-rows", op="quant", rows=16381, cols=4096, block=1, x=BF16, pow2=False),
        # weights of a projection, laid out once: a scale for 128 x 128 numbers, sizes that are no multiple of it
        dict(name="quant-2500-weights", op="quant", rows=2500, cols=2000, block=128, x=F32, pow2=False),
        # one token through the fused query, key and value projection of the 2048-wide layer (20 heads of 128)
        dict(name="product-1", op="product", T=1, N=2560, K=2048, out=BF16, pow2=False),
        # 64 requests through the wide layer's (40 heads of 128), fp32 out
        dict(name="product-64", op="product", T=64, N=5120, K=4096, out=F32, pow2=False),
        # a prompt's piece; no size is a multiple of a tile
        dict(name="product-505", op="product", T=505, N=5000, K=4000, out=BF16, pow2=True),
        # a long prompt
        dict(name="product-8190", op="product", T=8190, N=5120, K=4096, out=BF16, pow2=False),
        # one token far into a long context, two key heads, fp32
        dict(name="rotary-1", op="rotary", T=1, Hq=16, Hk=2, D=128, rot=128, first=0, layout="half", scaling="none", x=F32, far=1 << 20, inplace=False),
        # a decode step: 64 requests, interleaved pairs in the last part of each head, scaled for a long context, in place
        dict(name="rotary-64-part", op="rotary", T=64, Hq=64, Hk=1, D=192, rot=64, first=128, layout="interleaved", scaling="yarn", x=BF16, far=131072, inplace=True),
        # a long prompt's queries and keys
        dict(name="rotary-16381", op="rotary", T=16381, Hq=32, Hk=8, D=128, rot=128, first=0, layout="half", scaling="bands", x=BF16, far=131072, inplace=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "quant", "product", "product", "product", "rotary", "rotary"])
    if op == "norm":
        d = _log(rng, 64, 16384)
        d = rng.choice([d, d, d // 8 * 8, -(-d // 128) * 128])
        return dict(op=op, T=_log(rng, 1, max(1, min(16384, (1 << 25) // d))), d=d, x=rng.choice([BF16, BF16, F32]), res=rng.choice(["", BF16, F32]),
                    weight=rng.choice(["", BF16, F32]), y=rng.choice([E4M3, E4M3, BF16, F32]), pow2=rng.random() < 0.4)
    if op == "quant":
        cols = _log(rng, 64, 16384)
        cols = rng.choice([cols, cols // 8 * 8, -(-cols // 128) * 128])
        block = rng.choice([1, 1, 128])
        return dict(op=op, rows=_log(rng, 1, max(1, (1 << 25) // cols)), cols=cols, block=block, x=rng.choice([BF16, F32]), pow2=rng.random() < 0.4)
    if op == "product":
        N, K = _log(rng, 64, 8192), _log(rng, 64, 16384)
        if rng.random() < 0.6:
            N, K = -(-N // 128) * 128, -(-K // 128) * 128
        T = _log(rng, 1, max(1, min(16384, (1 << 37) // (N * K))))
        return dict(op=op, T=T, N=N, K=K, out=rng.choice([BF16, BF16, F32]), pow2=rng.random() < 0.4)
    D = rng.choice([64, 80, 96, 128, 128, 192, 256])
    rot = rng.choice([D, D, D // 2, D // 4, 2 * rng.randrange(1, D // 2 + 1)])
    first = rng.choice([0, 0, D - rot])
    Hk = rng.choice([1, 2, 4, 8])
    Hq = Hk * rng.choice([1, 2, 3, 4, 7, 8])
    T = _log(rng, 1, max(1, min(16384, (1 << 26) // ((Hq + Hk) * D))))
    return dict(op=op, T=T, Hq=Hq, Hk=Hk, D=D, rot=rot, first=first, layout=rng.choice(["half", "interleaved"]),
                scaling=rng.choice(["none", "linear", "base", "yarn", "bands"]), x=rng.choice([BF16, F32]), far=_log(rng, 16, 1 << 20), inplace=rng.random() < 0.5)


def _up(n, m):
    return -(-n // m) * m


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"norm": _prepare_norm, "quant": _prepare_quant, "product": _prepare_product, "rotary": _prepare_rotary}[case["op"]](case, g)


def _rows(T, n, dtype, fill=None):
    """[T][n] with its rows on 16-byte boundaries."""
    x = torch.empty((T, _up(n, 16)), dtype=dtype, device="cuda")[:, :n]
    if fill is not None:
        x.copy_(fill)
    return x


def _randn(T, n, g, wide=()):
    x = torch.randn((T, n), generator=g, device="cuda")
    for c in wide:  # channels that are far larger than the others, as activations have them
        if c < n:
            x[:, c] *= 30.0
    return x


def _prepare_norm(case, g):
    T, d = case["T"], case["d"]
    x = _rows(T, d, TORCH[case["x"]], _randn(T, d, g))
    res = _rows(T, d, TORCH[case["res"]], 3.0 * _randn(T, d, g, (5, 1111))) if case["res"] else None
    w = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(TORCH[case["weight"]]) if case["weight"] else None
    e4m3 = case["y"] == E4M3
    return dict(case=case, x=x, res=res, w=w, sum=_rows(T, d, res.dtype) if case["res"] else None, y=_rows(T, d, TORCH[case["y"]]),
                scales=torch.empty((T, -(-d // BLOCK)), device="cuda") if e4m3 else None)


def _prepare_quant(case, g):
    R, n = case["rows"], case["cols"]
    x = _randn(R, n, g, (5, 1111)) if case["block"] == 1 else 0.02 * _randn(R, n, g)
    return dict(case=case, x=_rows(R, n, TORCH[case["x"]], x), codes=_rows(R, n, torch.float8_e4m3fn),
                scales=torch.empty((-(-R // case["block"]), -(-n // BLOCK)), device="cuda"))


def _prepare_product(case, g):
    T, N, K = case["T"], case["N"], case["K"]
    a, sa = _quantise(_randn(T, K, g, (5, 1111)), 1, case["pow2"])
    w, sw = _quantise(0.02 * _randn(N, K, g), BLOCK, case["pow2"])
    return dict(case=case, a=_rows(T, K, a.dtype, a), sa=sa.contiguous(), w=_rows(N, K, w.dtype, w), sw=sw.contiguous(), out=_rows(T, N, TORCH[case["out"]]))


#: base of the frequencies, and what the scalings for long contexts go by: the factor, the length of the training, the two borders
BASE, FACTOR, TRAINED = 500000.0, 8.0, 8192
BORDERS = {"yarn": (1.0, 32.0), "bands": (1.0, 4.0)}


def _amplitude(case):
    """What the scaling adds to the products' size; 1 in place, where pass follows pass on the same numbers."""
    return 0.1 * math.log(FACTOR) + 1.0 if case["scaling"] == "yarn" and not case["inplace"] else 1.0


def _freqs(case):
    """Radians a place, pair by pair."""
    rot, kind = case["rot"], case["scaling"]
    base = BASE * FACTOR ** (rot / (rot - 2)) if kind == "base" and rot > 2 else BASE
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if kind == "linear":
        return [x / FACTOR for x in f]
    if kind == "yarn":
        at = lambda turns: rot * math.log(TRAINED / (turns * 2 * math.pi)) / (2 * math.log(BASE))  # noqa: E731  the pair that turns so often within the training's length
        low, high = max(math.floor(at(BORDERS[kind][1])), 0), min(math.ceil(at(BORDERS[kind][0])), rot - 1)
        ramp = [min(1.0, max(0.0, (i - low) / max(high - low, 0.001))) for i in range(rot // 2)]
        return [x * (1 - r) + x / FACTOR * r for x, r in zip(f, ramp)]
    if kind == "bands":
        lo, hi = BORDERS[kind]
        keep = [min(1.0, max(0.0, (TRAINED * x / (2 * math.pi) - lo) / (hi - lo))) for x in f]
        return [x * k + x / FACTOR * (1 - k) for x, k in zip(f, keep)]
    return f


def _prepare_rotary(case, g):
    T, Hq, Hk, D = (case[k] for k in ("T", "Hq", "Hk", "D"))
    qkv = torch.randn((T, (Hq + 2 * Hk) * D), generator=g, device="cuda").to(TORCH[case["x"]])
    places = torch.randint(0, case["far"], (T,), generator=g, device="cuda", dtype=torch.int32)
    s = dict(case=case, qkv=qkv, q=qkv[:, : Hq * D], k=qkv[:, Hq * D : (Hq + Hk) * D], places=places, freq=torch.tensor(_freqs(case), dtype=torch.float64, device="cuda"))
    if case["inplace"]:  # queries and keys turn where they stand, pass after pass
        return dict(s, q_out=s["q"], k_out=s["k"])
    return dict(s, q_out=torch.empty((T, Hq * D), dtype=qkv.dtype, device="cuda"), k_out=torch.empty((T, Hk * D), dtype=qkv.dtype, device="cuda"))


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "quant": _own_quant, "product": _own_product, "rotary": _own_rotary}[op](state)
    return {"norm": _plain_norm, "quant": _plain_quant, "product": _plain_product, "rotary": _plain_rotary}[op](state)


def _quantise(x, rows, pow2):
    """x [R][n] fp32 by blocks of `rows` x 128 numbers: their values in units of the block's scale as e4m3, and the scales."""
    R, n = x.shape
    RB, NB = -(-R // rows), -(-n // BLOCK)
    full = torch.nn.functional.pad(x, (0, NB * BLOCK - n, 0, RB * rows - R)).view(RB, rows, NB, BLOCK)
    scale = (full.abs().amax((1, 3)) / E4M3_MAX).clamp(min=LEAST)
    if pow2:
        m, e = torch.frexp(scale)
        scale = torch.ldexp(torch.ones_like(scale), e - (m == 0.5).int())
    codes = (full / scale[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes.reshape(RB * rows, NB * BLOCK)[:R, :n], scale


def _plain_norm(s):
    case, h = s["case"], s["x"].float()
    out = {}
    if s["res"] is not None:
        h = h + s["res"].float()
        out["sum"] = h.to(s["res"].dtype)
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6)
    if s["w"] is not None:
        y = y * s["w"].float()
    if case["y"] == E4M3:
        out["codes"], out["scales"] = _quantise(y, 1, case["pow2"])
    else:
        out["y"] = y.to(TORCH[case["y"]])
    return out


def _plain_quant(s):
    codes, scales = _quantise(s["x"].float(), s["case"]["block"], s["case"]["pow2"])
    return dict(codes=codes, scales=scales)


def _plain_product(s):
    K, N = s["case"]["K"], s["case"]["N"]
    wide = lambda x, n: torch.repeat_interleave(x, BLOCK, 1)[:, :n]  # noqa: E731  a scale for each number
    a = s["a"].float() * wide(s["sa"], K)
    w = s["w"].float() * torch.repeat_interleave(wide(s["sw"], K), BLOCK, 0)[:N]
    return dict(out=torch.mm(a, w.t()).to(s["out"].dtype))


def _turned(x, H, case, c, s):
    D, rot, first = case["D"], case["rot"], case["first"]
    x = x.unflatten(1, (H, D))
    part = x[..., first : first + rot].float()
    if case["layout"] == "half":
        a, b = part[..., : rot // 2], part[..., rot // 2 :]
        part = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([x[..., :first], part.to(x.dtype), x[..., first + rot :]], -1).flatten(1)


def _plain_rotary(st):
    case = st["case"]
    angle = st["places"].double()[:, None] * st["freq"]  # in 64 bits: far places times frequencies near 1
    c, s = ((_amplitude(case) * f(angle)).float()[:, None] for f in (torch.cos, torch.sin))
    q, k = _turned(st["q"], case["Hq"], case, c, s), _turned(st["k"], case["Hk"], case, c, s)
    st["q_out"].copy_(q)
    st["k_out"].copy_(k)
    return dict(q=st["q_out"], k=st["k_out"])


def _own_norm(s):
    from int4_expert_gemv_gb300 import moe
    c = s["case"]
    if "desc" not in s:
        s["desc"] = moe.NormDesc(d=c["d"], eps=1e-6, weight=None if s["w"] is None else s["w"].data_ptr(),
                                 w_dtype=moe.MOE_DTYPE_BF16 if c["weight"] == BF16 else moe.MOE_DTYPE_F32, pow2=int(c["pow2"]))
    moe.moe_add_rms_norm(s["desc"], s["x"], c["T"], s["y"], res=s["res"], sum=s["sum"], scales=s["scales"])
    out = {} if s["res"] is None else dict(sum=s["sum"])
    return dict(out, codes=s["y"], scales=s["scales"]) if c["y"] == E4M3 else dict(out, y=s["y"])


def _own_quant(s):
    from int4_expert_gemv_gb300 import moe
    c = s["case"]
    moe.moe_quantise_e4m3(s["x"], c["rows"], c["cols"], s["codes"], s["scales"], block_rows=c["block"], pow2=c["pow2"])
    return dict(codes=s["codes"], scales=s["scales"])


def _own_product(s):
    from int4_expert_gemv_gb300 import moe
    c = s["case"]
    if "desc" not in s:
        s["desc"] = moe.ScaledMatrixDesc(N=c["N"], K=c["K"], w=s["w"].data_ptr(), w_stride=s["w"].stride(0), scales=s["sw"].data_ptr(),
                                         scale_stride=s["sw"].stride(0))
        s["ws"] = torch.zeros(moe.moe_scaled_product_workspace_bytes(s["desc"], c["T"]), dtype=torch.uint8, device="cuda")
    moe.moe_scaled_product(s["desc"], s["a"], s["sa"], c["T"], s["out"], s["ws"])
    return dict(out=s["out"])


def _own_rotary(s):
    from int4_expert_gemv_gb300 import moe
    c = s["case"]
    if "desc" not in s:
        kind = dict(none=moe.MOE_ROTARY_PLAIN, linear=moe.MOE_ROTARY_LINEAR, base=moe.MOE_ROTARY_BASE, yarn=moe.MOE_ROTARY_YARN, bands=moe.MOE_ROTARY_BANDS)[c["scaling"]]
        low, high = BORDERS.get(c["scaling"], (0.0, 0.0))
        s["desc"] = moe.RotaryDesc(D=c["D"], rot=c["rot"], first=c["first"], layout=moe.MOE_ROTARY_HALF if c["layout"] == "half" else moe.MOE_ROTARY_INTERLEAVED,
                                   scaling=kind, trained=TRAINED, base=BASE, factor=FACTOR, low=low, high=high, amplitude=_amplitude(c))
        s["turns"] = torch.empty(c["rot"] // 2, dtype=torch.int64, device="cuda")
        moe.moe_rotary_table(s["desc"], s["turns"])
    moe.moe_rotary(s["desc"], s["turns"], s["places"], c["T"], s["q"], c["Hq"], s["q_out"], s["k"], c["Hk"], s["k_out"])
    return dict(q=s["q_out"], k=s["k_out"])


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "norm":
        n = case["T"] * case["d"]
        b = n * (SIZE[case["x"]] + 2 * (SIZE[case["res"]] if case["res"] else 0) + SIZE[case["y"]]) + (SIZE[case["weight"]] * case["d"] if case["weight"] else 0)
        return {"bytes": b + (4 * case["T"] * -(-case["d"] // BLOCK) if case["y"] == E4M3 else 0), "flops": 6 * n}
    if case["op"] == "quant":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (SIZE[case["x"]] + 1) + 4 * -(-case["rows"] // case["block"]) * -(-case["cols"] // BLOCK), "flops": 2 * n}
    if case["op"] == "product":
        T, N, K = case["T"], case["N"], case["K"]
        return {"bytes": T * K + N * K + T * N * SIZE[case["out"]] + 4 * (T + -(-N // BLOCK)) * -(-K // BLOCK), "flops": 2 * T * N * K}
    heads = case["T"] * (case["Hq"] + case["Hk"])
    n = case["rot"] if case["inplace"] else case["D"]  # in place, what does not turn stays
    return {"bytes": 2 * heads * n * SIZE[case["x"]] + 4 * case["T"], "flops": 3 * heads * case["rot"]}


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "quant": _exact_quant, "product": _exact_product, "rotary": _exact_rotary}[case["op"]](case, s)


def _exact_blocks(x, rows, pow2):
    """Block column by block column; the values in units of their scale, before they are rounded to 8 bits."""
    R, n = x.shape
    values, scales = torch.empty_like(x), []
    group = torch.arange(R, device=x.device) // rows
    for a in range(0, n, BLOCK):
        most = x[:, a : a + BLOCK].abs().amax(1)
        top = torch.zeros(-(-R // rows), dtype=x.dtype, device=x.device).scatter_reduce(0, group, most, "amax")
        top = torch.maximum(top / E4M3_MAX, torch.full_like(top, LEAST))
        if pow2:
            top = torch.exp2(torch.ceil(torch.log2(top)))
        scales.append(top)
        values[:, a : a + BLOCK] = x[:, a : a + BLOCK] / top[group][:, None]
    return values, torch.stack(scales, 1)


def _exact_norm(case, s):
    h = s["x"].double()
    out = {}
    if s["res"] is not None:
        h = h + s["res"].double()
        out["sum"] = h
    y = h / torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / case["d"] + 1e-6)
    if s["w"] is not None:
        y = s["w"].double() * y
    if case["y"] == E4M3:
        out["codes"], out["scales"] = _exact_blocks(y, 1, case["pow2"])
    else:
        out["y"] = y
    return out


def _exact_quant(case, s):
    codes, scales = _exact_blocks(s["x"].double(), case["block"], case["pow2"])
    return dict(codes=codes, scales=scales)


def _exact_product(case, s):
    """Block of K by block of K: the block's sum, then its two scales."""
    T, N, K = case["T"], case["N"], case["K"]
    out = torch.zeros((T, N), dtype=torch.float64, device="cuda")
    rows = torch.arange(N, device="cuda") // BLOCK
    for b in range(-(-K // BLOCK)):
        a = s["a"][:, b * BLOCK : (b + 1) * BLOCK].double()
        w = s["w"][:, b * BLOCK : (b + 1) * BLOCK].double()
        out += (a @ w.t()) * s["sa"][:, b].double()[:, None] * s["sw"][:, b].double()[rows]
    return dict(out=out)


def _exact_rotary(case, s):
    """Each pair as a complex number, times amplitude * exp(i * place * frequency)."""
    D, rot, first = case["D"], case["rot"], case["first"]
    by = _amplitude(case) * torch.exp(1j * torch.outer(s["places"].double(), s["freq"]))[:, None]
    pair = torch.arange(rot // 2, device="cuda")
    i, j = (pair, pair + rot // 2) if case["layout"] == "half" else (2 * pair, 2 * pair + 1)
    out = {}
    for name, H in (("q", case["Hq"]), ("k", case["Hk"])):
        x = s[name].double().unflatten(1, (H, D))
        z = torch.complex(x[..., first + i], x[..., first + j]) * by
        x[..., first + i], x[..., first + j] = z.real, z.imag
        out[name] = x.flatten(1)
    return out
