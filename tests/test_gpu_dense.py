"""The add-and-norm, the quantisation by blocks, the block-scaled product and
the rotary embedding on the GPU, against plain forms in 64 bits."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
NAN_CODE = 0x7F


@pytest.fixture(scope="module")
def m():
    from int4_expert_gemv_gb300 import build
    build.build()
    from int4_expert_gemv_gb300 import moe
    moe.lib()
    return moe


def _values():
    """The 128 codes without a sign as numbers (the last is NaN)."""
    c = np.arange(128)
    e, f = c >> 3, c & 7
    v = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))
    v[127] = np.nan
    return v


VALUES = _values()


def _round(x):
    """Codes of numbers within +-448, to nearest, ties to the even code."""
    a = np.abs(x)
    hi = np.clip(np.searchsorted(VALUES[:127], a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = VALUES[hi] - a, a - VALUES[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def _number(codes):
    """Codes' values; the codes as bytes."""
    c = codes.view(torch.uint8).cpu().numpy()
    return np.where(c & 128, -1.0, 1.0) * VALUES[c & 127]


def _rows(T, n, dtype, fill=None, pad=16, canary=None):
    """[T][n] within wider rows; canary: what stands in the padding, as a byte."""
    wide = torch.empty((T + 2, (n + 15) // 16 * 16 + pad), dtype=dtype, device="cuda")
    wide.view(torch.uint8).fill_(0xEE if canary is None else canary)
    x = wide[1:T + 1, :n]
    if fill is not None:
        x.copy_(fill)
    x.wide = wide
    return x


def _untouched(x, canary=0xEE):
    """The padding around x is as it was."""
    T, n = x.shape
    raw = x.wide.view(torch.uint8)
    size = x.wide.element_size()
    assert bool((raw[0] == canary).all()) and bool((raw[T + 1] == canary).all())
    assert bool((raw[1:T + 1, n * size:] == canary).all())


def _codes(T, n):
    x = _rows(T, n, torch.uint8)
    return x


# ---------------------------------------------------------------- quantise
def _quantised(x, rows, pow2):
    """Codes and scales by the rule: x fp32 on the host."""
    R, n = x.shape
    RB, NB = -(-R // rows), -(-n // 128)
    full = np.zeros((RB * rows, NB * 128), np.float32)
    full[:R, :n] = x
    t = full.reshape(RB, rows, NB, 128)
    top = np.abs(t).max(axis=(1, 3))
    scale = np.maximum(top / np.float32(448.0), np.float32(2.0 ** -100)).astype(np.float32)
    if pow2:
        f, e = np.frexp(scale)
        scale = np.ldexp(np.float32(1.0), e - (f == 0.5)).astype(np.float32)
    q = (t / scale[:, None, :, None]).astype(np.float32)
    return _round(np.clip(q, -448, 448).astype(np.float64)).reshape(RB * rows, NB * 128)[:R, :n], scale


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("R,n", [(1, 1), (1, 128), (3, 127), (2, 129), (5, 257), (129, 300), (300, 2048), (257, 1001), (1, 40000), (1500, 384)])
def test_quantise_is_exact(m, R, n, rows, pow2, dtype):
    g = torch.Generator(device="cuda").manual_seed(R * 1000 + n)
    x = torch.randn((R, n), generator=g, device="cuda") * torch.exp(4 * torch.randn((R, 1), generator=g, device="cuda"))
    x[:, ::7] *= 1e-3                                          # numbers that end below the codes' normal ones
    x[R // 2] = 0.0
    x = _rows(R, n, dtype, x)
    codes, scales = _codes(R, n), _rows(-(-R // rows), -(-n // 128), F32)
    m.moe_quantise_e4m3(x, R, n, codes, scales, block_rows=rows, pow2=pow2)
    want, scale = _quantised(x.float().cpu().numpy(), rows, pow2)
    assert np.array_equal(scales.cpu().numpy(), scale)
    got = codes.cpu().numpy()
    assert np.array_equal(got, want), np.argwhere(got != want)[:5]
    _untouched(codes)
    _untouched(scales)


def test_quantise_settles_ties_and_borders(m):
    """Quotients on the middle between two codes, and next to it: sizes that
    are multiples of a scale which fp32 does not invert exactly."""
    mids = 0.5 * (VALUES[:126] + VALUES[1:127])
    rows = []
    for a in (1.0, 3.0, 5.0, 7.0, 11.0, 13.0, 27.0):
        s = np.float32(a)
        for near in (0, 1, -1):
            v = (mids * float(s)).astype(np.float32)
            v = v if near == 0 else np.nextafter(v, np.float32(np.inf if near > 0 else 0.0)).astype(np.float32)
            row = np.zeros(128, np.float32)
            row[:126], row[126], row[127] = v, 448 * s, -448 * s
            rows.append(row)
    x = np.stack(rows)
    codes, scales = torch.zeros((len(x), 128), dtype=torch.uint8, device="cuda"), torch.zeros((len(x), 1), device="cuda")
    m.moe_quantise_e4m3(torch.from_numpy(x).cuda(), len(x), 128, codes, scales)
    want, scale = _quantised(x, 1, False)
    assert np.array_equal(scales.cpu().numpy(), scale) and np.array_equal(codes.cpu().numpy(), want)


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_quantise_of_what_is_not_finite(m, bad, rows):
    x = torch.ones((200, 500), device="cuda")
    x[130, 200] = bad
    codes, scales = torch.zeros((200, 512), dtype=torch.uint8, device="cuda")[:, :500], torch.zeros((200, 4), device="cuda")
    m.moe_quantise_e4m3(x, 200, 500, codes, scales, block_rows=rows)
    nan = torch.isnan(scales[: -(-200 // rows)])
    want = torch.zeros_like(nan)
    want[130 // rows, 1] = True
    assert torch.equal(nan, want)
    hit = torch.zeros((200, 500), dtype=torch.bool, device="cuda")
    hit[(128 if rows == 128 else 130):(200 if rows == 128 else 131), 128:256] = True
    assert bool(((codes & 127) == NAN_CODE)[hit].all()) and bool((codes[~hit] == 0x7E).all())


def test_quantise_extremes_of_fp32(m):
    """The largest and the smallest numbers: no scale overflows or vanishes."""
    x = torch.zeros((4, 128), device="cuda")
    x[0, 3], x[1, 5], x[2, 7], x[3, 9] = 3.4028234e38, 1e-45, 2.0 ** -126, -1e-30
    for pow2 in (False, True):
        codes, scales = torch.zeros((4, 128), dtype=torch.uint8, device="cuda"), torch.zeros((4, 1), device="cuda")
        m.moe_quantise_e4m3(x, 4, 128, codes, scales, pow2=pow2)
        want, scale = _quantised(x.cpu().numpy(), 1, pow2)
        assert np.array_equal(scales.cpu().numpy(), scale) and np.array_equal(codes.cpu().numpy(), want)


# ---------------------------------------------------------------- norm
# fp32 arithmetic of the norm, relative to the result: h 2^-24; the sum of
# squares at most 64 additions in a thread and 10 across the CTA, and twice h's
# error, half of it after the root: 38 2^-24; three divisions and roots and two
# products: 5 2^-24.
NORM = 48 * 2.0 ** -24


def _norm(x, res, w, eps):
    h = x.double().cpu() + (0 if res is None else res.double().cpu())
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + eps)
    return h.numpy(), (y if w is None else y * w.double().cpu()).numpy()


@pytest.mark.parametrize("x_type,res_type,w_type", [(BF16, F32, BF16), (BF16, BF16, F32), (F32, None, None), (F32, F32, F32), (F32, BF16, BF16),
                                                    (BF16, None, BF16)])
@pytest.mark.parametrize("y_type", [F32, BF16, E4M3])
@pytest.mark.parametrize("T,d", [(1, 1), (1, 8), (3, 100), (5, 256), (2, 257), (7, 512), (4, 513), (3, 2048), (2, 2050), (3, 4096), (2, 8200), (2, 16384),
                                 (1, 32768), (400, 1000), (2, 32763)])
def test_norm(m, T, d, x_type, res_type, w_type, y_type):
    g = torch.Generator(device="cuda").manual_seed(T * 100 + d)
    x = _rows(T, d, x_type, torch.randn((T, d), generator=g, device="cuda"))
    res = None if res_type is None else _rows(T, d, res_type, 3 * torch.randn((T, d), generator=g, device="cuda"))
    w = None if w_type is None else (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(w_type)
    s = None if res is None else _rows(T, d, res_type)
    y = _rows(T, d, torch.uint8 if y_type == E4M3 else y_type)
    scales = _rows(T, -(-d // 128), F32) if y_type == E4M3 else None
    nd = m.NormDesc(d=d, eps=1e-6, weight=None if w is None else w.data_ptr(), w_dtype=1 if w_type == BF16 else 0, pow2=0)
    m.moe_add_rms_norm(nd, x, T, y, res=res, sum=s, scales=scales)
    h, want = _norm(x, res, w, 1e-6)
    if s is not None:
        err = np.abs(s.double().cpu().numpy() - h)
        assert (err <= np.abs(h) * (2.0 ** -24 if res_type == F32 else 2.0 ** -8 + 2.0 ** -23)).all()
        _untouched(s)
    if y_type == E4M3:
        sc = scales.double().cpu().numpy()
        wide = np.repeat(sc, 128, 1)[:, :d]
        top = np.maximum.reduceat(np.abs(want), np.arange(0, d, 128), axis=1)
        assert (np.abs(sc - top / 448) <= sc * (NORM + 2.0 ** -23)).all()
        # half a step of the code, a quotient rounded to fp32, the norm's own error
        assert (np.abs(_number(y) * wide - want) <= np.abs(want) * (2.0 ** -4 + 2 * NORM) + wide * 2.0 ** -10).all()
        _untouched(scales)
    else:
        tol = NORM + (2.0 ** -8 if y_type == BF16 else 0.0)
        assert (np.abs(y.double().cpu().numpy() - want) <= np.abs(want) * tol * (1 + 2.0 ** -7) + 1e-40).all()
    _untouched(y)


@pytest.mark.parametrize("T,d", [(3, 300), (9, 2048)])
def test_norm_scales_that_are_powers_of_two(m, T, d):
    g = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn((T, d), generator=g, device="cuda")[:, :d // 8 * 8].contiguous()
    d = x.shape[1]
    y, scales = _codes(T, d), torch.zeros((T, -(-d // 128)), device="cuda")
    m.moe_add_rms_norm(m.NormDesc(d=d, eps=0.0, weight=None, w_dtype=0, pow2=1), x, T, y, scales=scales)
    _, want = _norm(x, None, None, 0.0)
    sc = scales.double().cpu().numpy()
    f, _ = np.frexp(sc)
    assert (f == 0.5).all()
    top = np.maximum.reduceat(np.abs(want), np.arange(0, d, 128), axis=1)
    assert (top <= 448 * sc * (1 + NORM)).all() and (top > 224 * sc * (1 - NORM)).all()
    wide = np.repeat(sc, 128, 1)[:, :d]
    assert (np.abs(_number(y) * wide - want) <= np.abs(want) * (2.0 ** -4 + 2 * NORM) + wide * 2.0 ** -10).all()


@pytest.mark.parametrize("d", [200, 2048, 5000, 20000])
@pytest.mark.parametrize("what", ["sum is res", "sum is x", "y is x", "both"])
def test_norm_in_place(m, d, what):
    T = 5
    g = torch.Generator(device="cuda").manual_seed(d)
    x, res = torch.randn((T, d), generator=g, device="cuda"), torch.randn((T, d), generator=g, device="cuda")
    nd = m.NormDesc(d=d, eps=1e-6, weight=None, w_dtype=0, pow2=0)
    y, s = torch.empty_like(x), torch.empty_like(x)
    m.moe_add_rms_norm(nd, x, T, y, res=res, sum=s)
    x2, res2 = x.clone(), res.clone()
    s2 = res2 if what in ("sum is res", "both") else x2 if what == "sum is x" else torch.empty_like(x)
    y2 = x2 if what in ("y is x", "both") else torch.empty_like(x)
    m.moe_add_rms_norm(nd, x2, T, y2, res=res2, sum=s2)
    assert torch.equal(y, y2) and torch.equal(s, s2)


def test_norm_of_unusual_rows(m):
    """NaN, infinities and zeros stay in their rows; far sizes."""
    T, d = 6, 1024
    x = torch.ones((T, d), device="cuda")
    x[0, 17], x[1, 900], x[2] = math.nan, math.inf, 0.0
    x[3] *= 1e-25
    x[4] *= 1e15
    nd = m.NormDesc(d=d, eps=1e-6, weight=None, w_dtype=0, pow2=0)
    y = torch.empty_like(x)
    m.moe_add_rms_norm(nd, x, T, y)
    assert bool(torch.isnan(y[0]).all())
    assert bool(torch.isnan(y[1, 900])) and int((y[1] == 0).sum()) == d - 1
    assert bool((y[2] == 0).all())
    assert torch.allclose(y[3], torch.full((d,), 1e-22, device="cuda"), rtol=1e-5) and torch.allclose(y[4:], torch.ones((2, d), device="cuda"), rtol=1e-5)
    c, s = torch.zeros((T, d), dtype=E4M3, device="cuda"), torch.zeros((T, d // 128), device="cuda")
    m.moe_add_rms_norm(nd, x, T, c, scales=s)
    assert bool(torch.isnan(c[0].float()).all()) and bool(torch.isnan(s[0]).all())
    assert bool((s[2] == 2.0 ** -100).all()) and bool((c[2].float() == 0).all())
    assert bool((c[4:].float() == 448).all()) and not bool(torch.isnan(s[2:]).any())
    m.moe_add_rms_norm(m.NormDesc(d=d, eps=0.0, weight=None, w_dtype=0, pow2=0), x, T, y)      # 0 / 0
    assert bool(torch.isnan(y[2]).all())


# ---------------------------------------------------------------- product
def _matrix(m, w, K, scales):
    N = w.shape[0]
    return m.ScaledMatrixDesc(N=N, K=K, w=w.data_ptr(), w_stride=w.stride(0), scales=scales.data_ptr(), scale_stride=scales.stride(0))


def _product_inputs(T, N, K, seed, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    KB = -(-K // 128)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x = (100 * rnd(T, K)).clamp(-448, 448).to(E4M3)
    w = (100 * rnd(N, K)).clamp(-448, 448).to(E4M3)
    sx = 0.01 * torch.exp(spread * rnd(T, KB))
    sw = 0.001 * torch.exp(spread * rnd(-(-N // 128), KB))
    return x, w, sx, sw


def _put(x, K, canary=0x7F):
    """Codes in wider rows whose padding is NaN."""
    r = _rows(x.shape[0], K, torch.uint8, x.view(torch.uint8), canary=canary)
    return r


def _product(x, w, sx, sw, K):
    """The product and the sum of its terms' sizes."""
    cols = torch.arange(K, device="cuda") // 128
    a = x.double() * sx.double()[:, cols]
    b = w.double() * sw.double()[:, cols][torch.arange(w.shape[0], device="cuda") // 128]
    return a @ b.t(), a.abs() @ b.abs().t()


def _product_tol(K):
    """A block's 128 products and their sum, the product of two scales, the
    block's product with it, the sum over the blocks."""
    return (128 + 2 + -(-K // 128)) * 2.0 ** -24


def _check_product(m, T, N, K, out_type, seed=0, spread=1.0, x=None, w=None, sx=None, sw=None):
    if x is None:
        x, w, sx, sw = _product_inputs(T, N, K, seed, spread)
    xr, wr = _put(x, K), _put(w, K)
    out = _rows(T, N, out_type)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    wd = _matrix(m, wr, K, sw)
    assert m.moe_scaled_product_workspace_bytes(wd, T) <= 256
    m.moe_scaled_product(wd, xr, sx, T, out, ws)
    want, size = _product(x, w, sx, sw, K)
    tol = size * _product_tol(K)
    if out_type == BF16:
        tol = tol + want.abs() * 2.0 ** -8 * (1 + 2.0 ** -8)
    err = (out.double() - want).abs()
    assert bool((err <= tol).all()), (float((err / size.clamp(min=1e-300)).max()), torch.nonzero(err > tol)[:5].tolist())
    assert int(ws.view(torch.int32)[0]) == 0
    _untouched(out)
    return out


@pytest.mark.parametrize("out_type", [F32, BF16])
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 100, 128, 129, 255, 257])
@pytest.mark.parametrize("N,K", [(128, 128), (1, 1), (100, 33), (130, 129), (257, 500), (384, 1000), (640, 2048)])
def test_product(m, T, N, K, out_type):
    _check_product(m, T, N, K, out_type, seed=T + N + K)


@pytest.mark.parametrize("T,N,K,out_type", [
    (1, 2560, 2048, BF16), (1, 5120, 4096, F32), (1, 100, 16384, F32), (3, 8192, 1024, BF16), (40, 2048, 7168, F32), (64, 5120, 4096, BF16),
    (200, 2560, 2048, BF16), (300, 5000, 4000, F32), (500, 5001, 600, BF16), (513, 1100, 3000, BF16), (1000, 4096, 1024, F32), (1025, 2560, 2176, BF16), (2048, 2048, 2048, F32),
    (3000, 1300, 500, BF16), (4097, 640, 256, F32), (1, 70000, 128, BF16), (70000, 16, 128, F32), (5, 16, 65536, F32), (600, 300, 20000, F32)])
def test_product_of_larger_sizes(m, T, N, K, out_type):
    _check_product(m, T, N, K, out_type, seed=T + N + K)


@pytest.mark.parametrize("T", [1, 20, 100, 300, 600])
def test_product_of_whole_numbers_is_exact(m, T):
    """Codes and scales whose sums fp32 holds: equal to the last bit, and blocks of far sizes meet their own scales."""
    N, K = 700, 900
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randint(-8, 9, (T, K), generator=g, device="cuda").float().to(E4M3)
    w = torch.randint(-8, 9, (N, K), generator=g, device="cuda").float().to(E4M3)
    sx = torch.exp2(torch.randint(0, 4, (T, 8), generator=g, device="cuda").float())
    sw = torch.exp2(torch.randint(-2, 2, (6, 8), generator=g, device="cuda").float())
    out = _check_product(m, T, N, K, F32, x=x, w=w, sx=sx, sw=sw)
    assert torch.equal(out.double(), _product(x, w, sx, sw, K)[0])


@pytest.mark.parametrize("T", [1, 30, 130, 700])
def test_product_of_far_scales(m, T):
    """Block scales over many orders: each block's sum is held in fp32 on its own."""
    _check_product(m, T, 300, 2000, F32, seed=T, spread=6.0)


@pytest.mark.parametrize("T", [1, 33, 200, 600])
def test_product_keeps_nan_in_its_row_and_column(m, T):
    N, K = 300, 640
    x, w, sx, sw = _product_inputs(T, N, K, 5)
    x, w = x.view(torch.uint8).clone(), w.view(torch.uint8).clone()
    t, n = T // 2, 222
    x[t, 333], w[n, 100] = NAN_CODE, NAN_CODE | 128
    out, ws = torch.empty((T, 304), device="cuda")[:, :N], torch.zeros(256, dtype=torch.uint8, device="cuda")
    m.moe_scaled_product(_matrix(m, w, K, sw), x, sx, T, out, ws)
    want = torch.zeros((T, N), dtype=torch.bool, device="cuda")
    want[t], want[:, n] = True, True
    assert torch.equal(torch.isnan(out), want)


def test_product_twice_gives_the_same_bits(m):
    for T, N, K in ((1, 2560, 2048), (50, 1000, 4000), (500, 2500, 4096)):
        x, w, sx, sw = _product_inputs(T, N, K, 1)
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        outs = []
        for _ in range(3):
            out = torch.zeros((T, N), device="cuda")
            m.moe_scaled_product(_matrix(m, w, K, sw), x, sx, T, out, ws)
            outs.append(out)
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_products_on_two_streams_and_in_graphs_share_a_workspace(m):
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    jobs = []
    for i, (T, N, K) in enumerate([(1, 2560, 2048), (64, 2048, 2048), (700, 2500, 2048), (5, 640, 8192)]):
        x, w, sx, sw = _product_inputs(T, N, K, i)
        jobs.append((T, x, sx, w, sw, _matrix(m, w, K, sw), torch.zeros((T, N), device="cuda"), _product(x, w, sx, sw, K)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(5):
        for st, (T, x, sx, w, sw, wd, out, _) in zip(streams, jobs):
            m.moe_scaled_product(wd, x, sx, T, out, ws, stream=st)
    torch.cuda.synchronize()
    graphs = []
    for T, x, sx, w, sw, wd, out, (want, size) in jobs:
        assert bool(((out.double() - want).abs() <= size * _product_tol(x.shape[1])).all())
        out.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.moe_scaled_product(wd, x, sx, T, out, ws)
        graphs.append(g)
    for _ in range(3):
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for T, x, sx, w, sw, wd, out, (want, size) in jobs:
        assert bool(((out.double() - want).abs() <= size * _product_tol(x.shape[1])).all())
    assert int(ws.view(torch.int32)[0]) == 0


# ---------------------------------------------------------------- rotary
KINDS = ["PLAIN", "LINEAR", "BASE", "YARN", "BANDS"]


def _freqs(rot, kind, base=10000.0, factor=4.0, trained=4096, low=1.0, high=32.0):
    i = np.arange(rot // 2)
    b = base * factor ** (rot / (rot - 2)) if kind == "BASE" and rot > 2 else base
    f = b ** (-2.0 * i / rot)
    if kind == "LINEAR":
        return f / factor
    turns = trained * f / (2 * np.pi)
    if kind == "BANDS":
        keep = np.clip((turns - low) / (high - low), 0, 1)
        return f * keep + f / factor * (1 - keep)
    if kind == "YARN":
        pair = lambda n: rot * np.log(trained / (n * 2 * np.pi)) / (2 * np.log(base))  # noqa: E731
        a, z = max(np.floor(pair(high)), 0), min(np.ceil(pair(low)), rot - 1)
        ramp = np.clip((i - a) / max(z - a, 0.001), 0, 1)
        return f * (1 - ramp) + f / factor * ramp
    return f


def _desc(m, D, rot, first, layout, kind, amplitude=1.0):
    return m.RotaryDesc(D=D, rot=rot, first=first, layout=m.MOE_ROTARY_HALF if layout == "half" else m.MOE_ROTARY_INTERLEAVED,
                        scaling=KINDS.index(kind), trained=4096, base=10000.0, factor=4.0, low=1.0, high=32.0, amplitude=amplitude)


def _turn(x, H, D, rot, first, layout, angle, amplitude):
    """x [T][H * D] turned, in 64 bits, and the size |a| + |b| of each number's pair (0 where none turns)."""
    x = x.double().cpu().numpy().reshape(-1, H, D)
    out, size = x.copy(), np.zeros_like(x)
    p = np.arange(rot // 2)
    i, j = (first + p, first + p + rot // 2) if layout == "half" else (first + 2 * p, first + 2 * p + 1)
    c, s = np.cos(angle)[:, None] * amplitude, np.sin(angle)[:, None] * amplitude
    a, b = x[..., i], x[..., j]
    out[..., i], out[..., j] = a * c - b * s, b * c + a * s
    size[..., i] = size[..., j] = (np.abs(a) + np.abs(b)) * abs(amplitude)
    return out.reshape(len(x), -1), size.reshape(len(x), -1)


# cosine and sine: what is left of the angle within a quarter rounded to fp32 (2^-24 of at most pi / 4), the
# functions' two steps (2^-22), their product with the amplitude (2^-24); a product, and an fma: 2^-23.
TURN = 2.0 ** -21


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,Hq,Hk,D,rot,first,kind,amplitude", [
    (1, 1, 0, 2, 2, 0, "PLAIN", 1.0), (1, 16, 2, 128, 128, 0, "PLAIN", 1.0), (5, 4, 4, 64, 32, 0, "LINEAR", 1.0), (33, 3, 1, 80, 80, 0, "BASE", 1.3),
    (7, 8, 1, 192, 64, 128, "YARN", 1.1386), (64, 5, 2, 96, 48, 16, "BANDS", 1.0), (9, 2, 1, 50, 30, 7, "YARN", -0.5), (2, 1, 3, 1024, 1024, 0, "PLAIN", 1.0),
    (300, 0, 2, 128, 64, 64, "BANDS", 2.0), (1000, 6, 2, 128, 128, 0, "LINEAR", 1.0), (3, 130, 1, 256, 256, 0, "YARN", 1.0), (4, 2, 2, 72, 24, 8, "PLAIN", 1.0)])
@pytest.mark.parametrize("inplace", [False, True])
def test_rotary(m, T, Hq, Hk, D, rot, first, kind, amplitude, layout, dtype, inplace):
    g = torch.Generator(device="cuda").manual_seed(T + D)
    n = (Hq + 2 * Hk) * D
    qkv = torch.randn((T, n), generator=g, device="cuda").to(dtype)
    places = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda", dtype=torch.int32)
    places[0] = 0 if T > 1 else 987654
    rd = _desc(m, D, rot, first, layout, kind, amplitude)
    turns = torch.zeros(rot // 2, dtype=torch.int64, device="cuda")
    m.moe_rotary_table(rd, turns)
    before = qkv.clone()
    q, k = qkv[:, : Hq * D] if Hq else None, qkv[:, Hq * D:(Hq + Hk) * D] if Hk else None
    qo = q if inplace else torch.full((T, Hq * D), 7.0, dtype=dtype, device="cuda") if Hq else None
    ko = k if inplace else torch.full((T, Hk * D), 7.0, dtype=dtype, device="cuda") if Hk else None
    m.moe_rotary(rd, turns, places, T, q, Hq, qo, k, Hk, ko)
    angle = places.cpu().numpy().astype(np.float64)[:, None] * _freqs(rot, kind)
    for H, o, at in ((Hq, qo, 0), (Hk, ko, Hq * D)):
        if not H:
            continue
        want, size = _turn(before[:, at:at + H * D], H, D, rot, first, layout, angle, amplitude)
        tol = size * TURN + (np.abs(want) * 2.0 ** -8 * (1 + 2.0 ** -8) * (size > 0) if dtype == BF16 else 0)
        err = np.abs(o.double().cpu().numpy() - want)
        assert (err <= tol).all(), (err - tol).max()
    assert torch.equal(qkv[:, (Hq + Hk) * D:], before[:, (Hq + Hk) * D:])
    if not inplace:
        assert torch.equal(qkv, before)


def test_rotary_of_far_and_negative_places(m):
    """Places up to the ends of 32 bits: the angle in whole numbers, against whole numbers in Python."""
    D, T = 128, 8
    places = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, -(2 ** 20) - 7, 999_999_937]
    rd = _desc(m, D, D, 0, "half", "PLAIN")
    turns = torch.zeros(D // 2, dtype=torch.int64, device="cuda")
    m.moe_rotary_table(rd, turns)
    F = [int(v) % 2 ** 64 for v in turns.cpu().tolist()]
    exact = [10000.0 ** (-2.0 * i / D) / (2 * math.pi) * 2.0 ** 64 for i in range(D // 2)]
    assert all(abs(a - b) <= 2.0 ** -50 * b + 1 for a, b in zip(F, exact))            # a few steps of fp64
    x = torch.randn((T, D), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    out = torch.empty_like(x)
    m.moe_rotary(rd, turns, torch.tensor(places, dtype=torch.int32, device="cuda"), T, x, 1, out)
    angle = np.array([[(p * f) % 2 ** 64 / 2.0 ** 64 * 2 * math.pi for f in F] for p in places])
    want, size = _turn(x, 1, D, D, 0, "half", angle, 1.0)
    assert (np.abs(out.double().cpu().numpy() - want) <= size * TURN).all()


def test_rotary_back_and_forth_in_a_graph(m):
    """Turned by its places and back by their opposites; captured and replayed."""
    T, H, D = 50, 4, 64
    x = torch.randn((T, H * D), device="cuda")
    places = torch.arange(T, dtype=torch.int32, device="cuda") * 1001
    rd = _desc(m, D, 64, 0, "interleaved", "PLAIN")
    turns = torch.zeros(32, dtype=torch.int64, device="cuda")
    m.moe_rotary_table(rd, turns)
    a, b = torch.empty_like(x), torch.empty_like(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    back = -places
    with torch.cuda.graph(g):
        m.moe_rotary(rd, turns, places, T, x, H, a)
        m.moe_rotary(rd, turns, back, T, a, H, b)
    g.replay()
    # each way at most TURN of |a| + |b|, which is at most sqrt 2 of the pair's length
    length = torch.sqrt(x.view(T, H, D // 2, 2).double().square().sum(-1, keepdim=True)).expand(-1, -1, -1, 2).reshape(T, -1)
    assert bool(((b.double() - x.double()).abs() <= 4 * TURN * length).all())
    assert not torch.equal(a, x)


def test_rotary_of_unaligned_tokens(m):
    """Tokens and starts off 16-byte boundaries: the same numbers, one at a time."""
    T, H, D = 6, 3, 64
    for dtype in (F32, BF16):
        buf = torch.randn(T * (H * D + 3) + 5, device="cuda").to(dtype)
        x = torch.as_strided(buf, (T, H * D), (H * D + 3, 1), 5)
        y = x.contiguous()
        places = torch.arange(T, dtype=torch.int32, device="cuda") * 77
        for layout in ("half", "interleaved"):
            rd = _desc(m, D, 32, 16, layout, "PLAIN")
            turns = torch.zeros(16, dtype=torch.int64, device="cuda")
            m.moe_rotary_table(rd, turns)
            a, b = torch.zeros((T, H * D), dtype=dtype, device="cuda"), torch.zeros((T, H * D), dtype=dtype, device="cuda")
            m.moe_rotary(rd, turns, places, T, x, H, a)
            m.moe_rotary(rd, turns, places, T, y, H, b)
            assert torch.equal(a, b)


FIRST_CALLS = """
import torch
from int4_expert_gemv_gb300 import moe, paged
T, d = %d, 512
x, places = torch.randn((T, d), device="cuda"), torch.arange(T, dtype=torch.int32, device="cuda")
w = torch.randn((300, d), device="cuda")
codes, scales = torch.zeros((300, d), dtype=torch.uint8, device="cuda"), torch.zeros((3, 4), device="cuda")
desc = moe.ScaledMatrixDesc(N=300, K=d, w=codes.data_ptr(), w_stride=d, scales=scales.data_ptr(), scale_stride=4)
xc, xs = torch.zeros((T, d), dtype=torch.uint8, device="cuda"), torch.zeros((T, 4), device="cuda")
out, ws = torch.zeros((T, 304), device="cuda")[:, :300], torch.zeros(256, dtype=torch.uint8, device="cuda")
rd = moe.RotaryDesc(D=64, rot=64, first=0, layout=0, scaling=0, base=10000.0, amplitude=1.0)
turns, turned = torch.zeros(32, dtype=torch.int64, device="cuda"), torch.zeros((T, d), device="cuda")
def calls():
    moe.moe_quantise_e4m3(w, 300, d, codes, scales, block_rows=128)
    moe.moe_add_rms_norm(moe.NormDesc(d=d, eps=1e-6, weight=None, w_dtype=0, pow2=0), x, T, xc, scales=xs)
    moe.moe_scaled_product(desc, xc, xs, T, out, ws)
    moe.moe_rotary_table(rd, turns)
    moe.moe_rotary(rd, turns, places, T, x, 8, turned)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    calls()
g.replay()
got = out.clone(), turned.clone()
out.zero_(), turned.zero_()
calls()
torch.cuda.synchronize()
assert torch.equal(got[0], out) and torch.equal(got[1], turned) and float(out.abs().sum()) > 0 and int(ws.view(torch.int32)[0]) == 0
print("same")
"""


@pytest.mark.parametrize("T", [1, 300])
def test_first_calls_of_a_process_may_be_captured(T):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS % T], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
