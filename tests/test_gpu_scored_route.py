"""Routing by scores on the GPU (needs a GPU) against the rule in 64 bits."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    from int4_expert_gemv_gb300 import build
    build.build()
    from int4_expert_gemv_gb300 import moe
    moe.lib()
    return moe


def _route(m, z, K, score="softmax", n_group=1, keep=1, best=1, renorm=True, factor=1.0, bias=None):
    T, E = z.shape
    rd = m.RouteDesc(E=E, K=K, score=m.MOE_SCORE_SIGMOID if score == "sigmoid" else m.MOE_SCORE_SOFTMAX, n_group=n_group,
                     keep_group=keep, group_best=best, renorm=int(renorm), factor=factor,
                     bias=None if bias is None else bias.data_ptr())
    idx = torch.full((T, K), -9, dtype=torch.int32, device="cuda")
    w = torch.full((T, K), 9.0, device="cuda")
    m.moe_scored_route(rd, z, T, idx, w)
    return idx.cpu().numpy(), w.cpu().double().numpy()


def _rule(z, K, score, n_group, keep, best, renorm, factor, bias):
    """(idx, w, margin) of one token in 64 bits; margin: the smallest
    difference between a choice that was made and the next unequal one (equal
    ones go by their index)."""
    E = len(z)
    on = np.isfinite(z) | (z == np.inf)
    s = np.zeros(E)
    with np.errstate(over="ignore"):
        if score == "sigmoid":
            s[on] = 1.0 / (1.0 + np.exp(-z[on]))
        elif on.any():
            top = z[on].max()
            e = np.where(z[on] == top, 1.0, np.exp(np.where(z[on] == top, 0.0, z[on]) - np.where(z[on] == top, 0.0, top)))
            s[on] = e / e.sum()
    c = np.where(on, s + (0.0 if bias is None else bias), -np.inf)
    gs = E // n_group
    margin = np.inf

    def order(v, n):
        nonlocal margin
        o = np.argsort(-v, kind="stable")
        for i in range(n):
            below = v[o[i:]][v[o[i:]] < v[o[i]]]
            if len(below) and np.isfinite(below[0]):
                margin = min(margin, v[o[i]] - below[0])
        return o[:n]

    allowed = np.ones(E, bool)
    if keep < n_group:
        g = np.array([np.sort(c[j * gs:(j + 1) * gs])[::-1][:best].sum() for j in range(n_group)])
        kept = order(g, keep)
        allowed = np.isin(np.arange(E) // gs, kept)
    cand = np.flatnonzero(allowed)
    idx = cand[order(c[cand], K)]
    w = s[idx]
    if renorm:
        w = w / w.sum() if w.sum() > 0 else np.zeros(K)
    return idx, factor * w, margin


def _check(m, z, K, **kw):
    """Indices equal wherever the 64-bit rule's margin exceeds 2^-20 (scores
    are at most 1, and fp32's exp, quotient and sums of up to 1024 terms keep
    them within 2^-21 of exact); weights within 2^-18 relative (a score, the
    sum of at most 16, a quotient) and the choices unequal otherwise."""
    bias = kw.get("bias")
    idx, w = _route(m, z, K, **kw)
    zz = z.double().cpu().numpy()
    b = None if bias is None else bias.double().cpu().numpy()
    full = dict(score="softmax", n_group=1, keep=1, best=1, renorm=True, factor=1.0)
    full.update({k: v for k, v in kw.items() if k != "bias"})
    decided = 0
    for t in range(len(zz)):
        ref, rw, margin = _rule(zz[t], K, bias=b, **full)
        assert len(set(idx[t])) == K and (0 <= idx[t]).all() and (idx[t] < zz.shape[1]).all()
        if margin > 2.0 ** -20:
            decided += 1
            assert np.array_equal(idx[t], ref), (t, idx[t], ref, margin)
            assert (np.abs(w[t] - rw) <= 2.0 ** -18 * np.abs(rw) + 1e-37).all(), (t, w[t], rw)
    return decided


SHAPES = [  # E, K, n_group, keep, best
    (1, 1, 1, 1, 1), (16, 2, 1, 1, 1), (60, 4, 4, 2, 2), (64, 16, 8, 3, 2), (256, 8, 8, 4, 2), (256, 8, 1, 1, 1), (512, 4, 1, 1, 1),
    (160, 6, 8, 3, 1), (384, 8, 8, 8, 2), (1024, 16, 32, 5, 2), (1020, 3, 17, 2, 2), (96, 5, 3, 2, 2), (33, 7, 1, 1, 1), (32, 1, 32, 1, 1),
    (1024, 16, 1, 1, 1)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K,n_group,keep,best", SHAPES)
def test_scored_route_against_the_rule(m, score, E, K, n_group, keep, best):
    g = torch.Generator(device="cuda").manual_seed(E + K)
    z = 1.5 * torch.randn((67, E), generator=g, device="cuda")
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    kw = dict(score=score, n_group=n_group, keep=keep, best=best)
    n = 0
    for x in (z, z.bfloat16()):
        n += _check(m, x, K, **kw)
        n += _check(m, x, K, bias=bias, renorm=False, factor=2.5, **kw)
    assert n >= 200                                      # of 268: near-ties are rare


def test_scored_route_ties_go_by_index(m):
    z = torch.zeros((9, 64), device="cuda")
    z[1, 40], z[2, ::2], z[3, 63], z[4] = 1.0, 2.0, -1.0, float("-inf")
    z[5, 10:] = -0.0
    for score in ("softmax", "sigmoid"):
        for kw in (dict(), dict(n_group=8, keep=2, best=2), dict(n_group=4, keep=3, best=1)):
            assert _check(m, z, 5, score=score, **kw) == 9
    zero = torch.zeros(64, device="cuda")
    zero[::3] = -0.0                                     # a bias of -0 changes nothing
    idx, _ = _route(m, z[:1], 5, score="sigmoid", bias=zero)
    assert idx[0].tolist() == [0, 1, 2, 3, 4]
    idx, _ = _route(m, z[:1], 5, score="sigmoid", bias=zero - 0.5)   # choices of 0: +0 and -0 are one
    assert idx[0].tolist() == [0, 1, 2, 3, 4]


def test_scored_route_experts_that_are_off(m):
    """-inf and NaN logits come after everything that is on and weigh 0; +inf
    shares the mass; rows with nothing on get valid indices and zeros."""
    inf, nan = float("inf"), float("nan")
    g = torch.Generator(device="cuda").manual_seed(0)
    z = torch.randn((8, 64), generator=g, device="cuda")
    z[0, ::2] = -inf
    z[1, 5:] = nan
    z[2, :] = -inf
    z[3, :] = nan
    z[4, 7], z[4, 50] = inf, inf
    z[5, :62] = torch.finfo(torch.float32).min
    z[6, 1:] = -inf
    z[7, 8:16], z[7, 20] = nan, inf
    for score in ("softmax", "sigmoid"):
        for kw in (dict(), dict(n_group=8, keep=3, best=2)):
            idx, w = _route(m, z, 6, score=score, **kw)
            assert np.isfinite(w).all() and (w >= 0).all()
            full = dict(n_group=1, keep=1, best=1, renorm=True, factor=1.0, bias=None)
            full.update(kw)
            for t in range(8):
                ref, rw, margin = _rule(z[t].double().cpu().numpy(), 6, score, **full)
                assert len(set(idx[t])) == 6 and (0 <= idx[t]).all() and (idx[t] < 64).all()
                if margin > 2.0 ** -20:
                    assert np.array_equal(idx[t], ref), (score, kw, t, idx[t], ref)
                    assert (np.abs(w[t] - rw) <= 2.0 ** -18 * rw + 1e-37).all()
    bias = torch.full((64,), 10.0, device="cuda")        # a bias does not bring them back
    idx, w = _route(m, z[6:7], 3, score="sigmoid", bias=bias)
    assert idx[0].tolist() == [0, 1, 2] and w[0, 0] == 1.0 and (w[0, 1:] == 0).all()


def test_scored_route_rows_of_a_wider_tensor(m):
    g = torch.Generator(device="cuda").manual_seed(1)
    for dt in (torch.float32, torch.bfloat16):
        wide = torch.randn((50, 131), generator=g, device="cuda").to(dt)
        z = wide[:, 3:63]                                # neither aligned nor contiguous
        assert _check(m, z, 4, score="sigmoid", n_group=4, keep=2, best=2) > 40


def test_scored_route_equals_topk_route_and_repeats(m):
    """Softmax scores, no groups, renormalised: the framework's first route."""
    g = torch.Generator(device="cuda").manual_seed(2)
    z = torch.randn((300, 256), generator=g, device="cuda")
    idx, w = _route(m, z, 4)
    i2, w2 = torch.empty((300, 4), dtype=torch.int32, device="cuda"), torch.empty((300, 4), device="cuda")
    m.moe_topk_route(z, 300, 256, 4, i2, w2)
    near = (torch.sort(z, 1, descending=True).values[:, :5].diff(dim=1).abs() < 1e-5).any(1).cpu().numpy()
    assert near.sum() < 5
    assert np.array_equal(idx[~near], i2.cpu().numpy()[~near])
    assert np.abs(w - w2.cpu().double().numpy())[~near].max() <= 2.0 ** -19
    again = _route(m, z, 4)
    assert np.array_equal(idx, again[0]) and np.array_equal(w, again[1])


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [0.0, 100.0, -100.0, 1000.0, -1000.0, 20000.0])
def test_scored_route_softmax_ignores_an_offset(m, offset, dt):
    """Softmax of logits far from zero: weights that are not renormalised,
    with and without a bias, within the same bounds."""
    g = torch.Generator(device="cuda").manual_seed(17)
    z = (1.5 * torch.randn((200, 256), generator=g, device="cuda") + offset).to(dt)
    bias = 0.01 * torch.randn(256, generator=g, device="cuda")
    n = 0
    for kw in (dict(), dict(bias=bias), dict(n_group=8, keep=3, best=2, bias=bias)):
        n += _check(m, z, 6, renorm=False, factor=2.5, **kw)
    assert n >= 400                                      # of 600


def _every_row(m, z, K, bias=None, **kw):
    """All rows' choices equal to the rule's, whatever the margin."""
    idx, w = _route(m, z, K, bias=bias, **kw)
    full = dict(score="softmax", n_group=1, keep=1, best=1, renorm=True, factor=1.0)
    full.update(kw)
    b = None if bias is None else bias.double().cpu().numpy()
    for t, row in enumerate(z.double().cpu().numpy()):
        ref, rw, _ = _rule(row, K, bias=b, **full)
        assert np.array_equal(idx[t], ref), (kw, t, idx[t], ref)
        assert (np.abs(w[t] - rw) <= 2.0 ** -18 * np.abs(rw) + 1e-37).all(), (kw, t, w[t], rw)


@pytest.mark.parametrize("T", [1, 6])
def test_scored_route_without_a_bias_goes_by_the_logits(m, T):
    """Scores that 32 bits cannot hold or tell apart (e^-100 beside 1, the
    sigmoids of -95 and -96): the order is the logits'."""
    E = 64
    g = torch.Generator(device="cuda").manual_seed(5)
    perm = torch.stack([torch.randperm(E, generator=g, device="cuda") for _ in range(T)])
    far = (torch.arange(E, device="cuda") - 200.0)[perm]
    far[:, 0] = 100.0                                    # one expert far above all others
    low = (-90.0 - 0.25 * torch.arange(E, device="cuda"))[perm]
    near = (20.0 + 0.0625 * torch.arange(E, device="cuda"))[perm]          # beside 1 by e^-20 and less
    for z in (far, low, far.bfloat16(), low.bfloat16()):
        for score in ("softmax", "sigmoid"):
            _every_row(m, z, 5, score=score)
            _every_row(m, z, 5, score=score, n_group=4, keep=2, best=1)
            _every_row(m, z, 5, score=score, n_group=4, keep=2, best=2)
            _every_row(m, z, 5, score=score, renorm=False, factor=2.5)
    for z in (near, near.bfloat16()):
        _every_row(m, z, 5, score="sigmoid")
        _every_row(m, z, 5, score="softmax")


def test_scored_route_equals_topk_route_of_wide_logits(m):
    g = torch.Generator(device="cuda").manual_seed(6)
    z = 120.0 * torch.randn((300, 256), generator=g, device="cuda")
    idx, w = _route(m, z, 8)
    i2, w2 = torch.empty((300, 8), dtype=torch.int32, device="cuda"), torch.empty((300, 8), device="cuda")
    m.moe_topk_route(z, 300, 256, 8, i2, w2)
    assert np.array_equal(idx, i2.cpu().numpy())
    assert np.abs(w - w2.cpu().double().numpy()).max() <= 2.0 ** -19


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scored_route_takes_the_lowest_number_before_what_is_off(m, score):
    """A logit or a bias of the type's lowest value is a number: its expert
    comes after all others and before those that are off."""
    low, inf = torch.finfo(torch.float32).min, float("inf")
    z = torch.zeros((2, 16), device="cuda")
    z[0, :12] = -inf
    z[0, 12:15] = low                                    # three at the lowest, one (15) above
    z[1, :5] = float("nan")
    z[1, 5:15] = -1.0
    z[1, 9] = low
    idx, w = _route(m, z, 6, score=score)
    assert idx[0].tolist() == [15, 12, 13, 14, 0, 1]
    assert idx[1].tolist() == [15, 5, 6, 7, 8, 10]
    assert w[0, 0] == 1.0 and (w[0, 4:] == 0).all()
    z = torch.zeros((1, 16), device="cuda")
    z[0, :4] = -inf
    bias = torch.full((16,), low, device="cuda")
    bias[7] = 0.0
    idx, w = _route(m, z, 14, score=score, bias=bias)
    assert idx[0].tolist() == [7, 4, 5, 6] + list(range(8, 16)) + [0, 1]
    assert np.abs(w[0, :12] - 1 / 12).max() <= 2.0 ** -18 and (w[0, 12:] == 0).all()


@pytest.mark.parametrize("T", [2 ** 31 - 1, 2 ** 31 - 16])
def test_scored_route_of_all_the_tokens_there_can_be(m, T):
    """One or two experts: idx and w of every token, and
    nothing behind them (21 GB and more)."""
    E = 1 if T % 2 else 2
    wide = torch.empty((T, E), dtype=torch.bfloat16, device="cuda")
    wide.fill_(0.5)
    if E == 2:
        wide[::3, 1] = 0.75
    idx = torch.full((T + 3,), -9, dtype=torch.int32, device="cuda")
    w = torch.full((T + 3,), 9.0, device="cuda")
    rd = m.RouteDesc(E=E, K=1, score=m.MOE_SCORE_SIGMOID, n_group=1, keep_group=1, group_best=1, renorm=1, factor=0.5, bias=None)
    m.moe_scored_route(rd, wide, T, idx, w)
    assert idx[T:].tolist() == [-9] * 3 and w[T:].tolist() == [9.0] * 3
    for a in range(0, T, 1 << 28):
        b = min(T, a + (1 << 28))
        want = (torch.arange(a, b, device="cuda") % 3 == 0).int() if E == 2 else torch.zeros(b - a, dtype=torch.int32, device="cuda")
        assert torch.equal(idx[a:b], want)
        assert bool((w[a:b] == 0.5).all())


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scored_route_of_rows_with_nothing_on(m, score, renorm):
    z = torch.full((5, 40), float("-inf"), device="cuda")
    z[1], z[2, ::2], z[3, 11] = float("nan"), float("nan"), 0.25
    for bias in (None, torch.linspace(-1, 1, 40, device="cuda")):
        idx, w = _route(m, z, 3, score=score, renorm=renorm, bias=bias)
        assert idx[[0, 1, 2, 4]].tolist() == [[0, 1, 2]] * 4 and idx[3].tolist() == [11, 0, 1]
        assert (w[[0, 1, 2, 4]] == 0).all() and (w[3, 1:] == 0).all()
        want = 1.0 if renorm or score == "softmax" else 1 / (1 + np.exp(-0.25))
        assert abs(w[3, 0] - want) <= 2.0 ** -18


def _rule_rows(z, K, score, n_group, keep, best, renorm, factor, bias):
    """_rule for all rows at once, on the device: (idx, w, margin)."""
    T, E = z.shape
    z = z.double()
    inf = float("inf")
    on = z > -inf                                        # not -inf, not NaN
    z0 = torch.where(on, z, -inf)
    if score == "sigmoid":
        s = torch.sigmoid(z0)
    else:
        top = z0.amax(1, keepdim=True)
        e = torch.where(z0 == top, 1.0, torch.exp(z0 - torch.where(top.isinf(), 0.0, top)))
        e = torch.where(on & ~((top == inf) & (z0 < inf)), e, 0.0)
        s = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    c = torch.where(on, s + (0.0 if bias is None else bias.double()), -inf)
    margin = torch.full((T,), inf, dtype=torch.float64, device=z.device)

    def order(v, n):
        nonlocal margin
        o = v.sort(dim=1, descending=True, stable=True)
        d = o.values[:, :-1] - o.values[:, 1:]
        counts = (torch.arange(d.shape[1], device=z.device) < n) | (o.values[:, :-1] == o.values[:, n - 1: n])
        if d.shape[1]:
            margin = torch.minimum(margin, torch.where(counts & (d > 0) & d.isfinite(), d, inf).amin(1))
        return o.indices[:, :n]

    if keep < n_group:
        g = c.view(T, n_group, E // n_group).sort(2, descending=True).values[:, :, :best].sum(2)
        kept = torch.zeros((T, n_group), dtype=torch.bool, device=z.device).scatter_(1, order(g, keep), True)
        kept = kept.repeat_interleave(E // n_group, 1)
        # the dropped ones behind those that are off
        key = torch.where(c == -inf, -1e300, c)
        idx = order(torch.where(kept, key, -inf), K)
    else:
        idx = order(torch.where(c == -inf, -1e300, c), K)
    w = s.gather(1, idx)
    if renorm:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return idx, factor * w, margin


def _check_many(m, z, K, **kw):
    """_check's bounds over a batch that fills the GPU."""
    idx, w = _route(m, z, K, **kw)
    full = dict(score="softmax", n_group=1, keep=1, best=1, renorm=True, factor=1.0, bias=None)
    full.update(kw)
    ref, rw, margin = (x.cpu().numpy() for x in _rule_rows(z, K, **full))
    one = np.sort(idx, 1)
    assert (one[:, 1:] != one[:, :-1]).all() and (one >= 0).all() and (one < z.shape[1]).all()
    sure = margin > 2.0 ** -20
    wrong = np.flatnonzero(sure & (idx != ref).any(1))
    assert not len(wrong), (len(wrong), wrong[0], idx[wrong[0]], ref[wrong[0]], margin[wrong[0]])
    off = np.flatnonzero(sure & (np.abs(w - rw) > 2.0 ** -18 * np.abs(rw) + 1e-37).any(1))
    assert not len(off), (len(off), off[0], w[off[0]], rw[off[0]])
    return int(sure.sum())


MANY = 6007      # above 32 tokens an SM: eight lanes a token whatever the width; a part of a block and of a warp at the end


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K,n_group,keep,best", SHAPES + [(1023, 16, 31, 9, 2), (640, 12, 32, 11, 1), (1024, 1, 16, 16, 1)])
def test_scored_route_of_many_tokens(m, score, E, K, n_group, keep, best):
    g = torch.Generator(device="cuda").manual_seed(E * 31 + K)
    z = 1.5 * torch.randn((MANY, E), generator=g, device="cuda")
    z[::7, E // 2:] = z[::7, : E - E // 2]               # equal logits
    z[5::11, : max(0, E // 3)] = float("-inf")
    z[6::13, E - E // 4:] = float("nan")
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    kw = dict(score=score, n_group=n_group, keep=keep, best=best)
    n = 0
    for x in (z, z.bfloat16()):
        n += _check_many(m, x, K, **kw)
        n += _check_many(m, x, K, bias=bias, renorm=False, factor=2.5, **kw)
    assert n >= 0.7 * 4 * MANY


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scored_route_of_many_tokens_answers_as_of_few(m, score):
    """Rows of ties, infinities, NaN, lowest numbers and far logits: the same
    choices in a batch that fills the GPU as in one of a few tokens."""
    inf, nan, low = float("inf"), float("nan"), torch.finfo(torch.float32).min
    g = torch.Generator(device="cuda").manual_seed(9)
    z = torch.randn((16, 96), generator=g, device="cuda")
    z[0], z[1], z[2, ::2], z[3] = 0.0, -inf, nan, nan
    z[4, 7], z[4, 50] = inf, inf
    z[5, :90], z[6, 1:], z[7, ::3] = low, -inf, -inf
    z[7, 1::3] = low
    z[8] = torch.arange(96, device="cuda") - 300.0
    z[8, 0] = 200.0
    z[9] = -90.0 - 0.5 * torch.arange(96, device="cuda")
    z[10] = 30.0 + torch.arange(96, device="cuda")
    z[11, 40:], z[12, 8:16], z[12, 20] = 5.0, nan, inf
    many = z.repeat(400, 1)
    bias = 0.25 * torch.randn(96, generator=g, device="cuda")
    bias[::5] = low
    for kw in (dict(), dict(n_group=12, keep=3, best=2), dict(n_group=4, keep=2, best=1), dict(n_group=32, keep=5, best=2)):
        for b in (None, bias):
            for renorm in (True, False):
                a = _route(m, z, 6, score=score, bias=b, renorm=renorm, **kw)
                c = _route(m, many, 6, score=score, bias=b, renorm=renorm, **kw)
                assert np.array_equal(np.tile(a[0], (400, 1)), c[0])
                # sums over a row in another order: 96 terms in fp32
                assert (np.abs(np.tile(a[1], (400, 1)) - c[1]) <= 2.0 ** -19 * np.abs(c[1])).all()


def test_scored_route_of_many_rows_of_a_wider_tensor(m):
    g = torch.Generator(device="cuda").manual_seed(12)
    for dt in (torch.float32, torch.bfloat16):
        wide = torch.randn((MANY, 131), generator=g, device="cuda").to(dt)
        for kw in (dict(n_group=4, keep=2, best=2), dict(n_group=12, keep=5, best=2), dict()):
            assert _check_many(m, wide[:, 3:63], 4, score="sigmoid", **kw) > 0.7 * MANY
