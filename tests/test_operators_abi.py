"""Refusals and sizes of the paged cache's calls and of the scored route,
without a GPU: a rejected call never reaches the device, an empty one
returns before it touches a pointer."""
import ctypes as C

import pytest

from int4_expert_gemv_gb300 import build as nbuild

AT = 1 << 20          # a well aligned address that is never read


@pytest.fixture(scope="module")
def m():
    nbuild.build()
    from int4_expert_gemv_gb300 import moe
    moe.lib()
    return moe


def _kv(m, **kw):
    a = dict(n_pages=100, page=16, Hkv=2, D=128, dtype=m.MOE_DTYPE_BF16, k=AT, v=AT, page_stride=2 * 16 * 128 * 2, k_scale=None,
             v_scale=None)
    a.update(kw)
    return m.KVDesc(**a)


BAD_KV = [dict(n_pages=0), dict(page=0), dict(page=65537), dict(Hkv=0), dict(D=0), dict(D=24), dict(D=272), dict(dtype=0), dict(dtype=7),
          dict(k=None), dict(v=None), dict(k=AT + 8), dict(v=AT + 2), dict(page_stride=2 * 16 * 128 * 2 - 16),
          dict(page_stride=2 * 16 * 128 * 2 + 8), dict(k_scale=AT), dict(v_scale=AT), dict(dtype=2, k_scale=AT + 2)]


# ------------------------------------------------------------ attention
def _attend(m, kv, **kw):
    a = dict(q=AT, q_dtype=1, q_stride=8 * 128, B=3, Hq=8, seq=AT, table=AT, max_blocks=4, scale=0.1, window=0, out=AT, out_stride=8 * 128,
             lse=AT, ws=AT, ws_bytes=1 << 40)
    a.update(kw)
    return m.lib().moe_paged_attention(None if kv is None else C.byref(kv), a["q"], a["q_dtype"], a["q_stride"], a["B"], a["Hq"], a["seq"],
                                       a["table"], a["max_blocks"], a["scale"], a["window"], a["out"], a["out_stride"], a["lse"], a["ws"],
                                       a["ws_bytes"], None)


@pytest.mark.parametrize("kw", BAD_KV)
def test_calls_reject_a_bad_cache(m, kw):
    assert _attend(m, _kv(m, **kw)) == m.MOE_EINVAL
    assert m.last_error() != ""
    assert _append(m, _kv(m, **kw)) == m.MOE_EINVAL


def test_calls_reject_a_missing_or_too_large_cache(m):
    assert _attend(m, None) == m.MOE_EINVAL and _append(m, None) == m.MOE_EINVAL
    big = _kv(m, n_pages=1 << 27)
    assert _attend(m, big) == m.MOE_EUNSUPPORTED and _append(m, big) == m.MOE_EUNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(B=65537), dict(Hq=0), dict(Hq=7), dict(Hq=65538), dict(max_blocks=0), dict(window=-1), dict(q_dtype=2), dict(scale=0.0),
    dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None), dict(q=AT + 4), dict(out=None), dict(out=AT + 8),
    dict(seq=None), dict(seq=AT + 2), dict(table=None), dict(table=AT + 1), dict(lse=AT + 2), dict(q_stride=8 * 128 - 8),
    dict(out_stride=8 * 128 - 8), dict(q_stride=8 * 128 + 4), dict(out_stride=8 * 128 + 1)])
def test_attention_rejects_bad_arguments(m, kw):
    assert _attend(m, _kv(m), **kw) == m.MOE_EINVAL
    assert m.last_error() != ""


def test_attention_workspace(m):
    kv = _kv(m)
    need = m.moe_paged_attention_workspace_bytes(kv, 3, 8)
    assert need > 0
    assert m.lib().moe_paged_attention_workspace_bytes(None, 3, 8) == 0
    assert m.moe_paged_attention_workspace_bytes(kv, 3, 7) == 0
    assert _attend(m, kv, ws=None) == m.MOE_ENOSPACE
    assert _attend(m, kv, ws_bytes=need - 1) == m.MOE_ENOSPACE
    assert _attend(m, kv, ws=AT + 128) == m.MOE_ENOSPACE


def test_empty_calls_are_no_ops(m):
    assert _attend(m, _kv(m), B=0, q=None, out=None, seq=None, table=None, ws=None) == m.MOE_OK
    assert _append(m, _kv(m), N=0, k=None, v=None, slots=None) == m.MOE_OK
    assert _route(m, _rd(m), T=0, z=None, idx=None, w=None) == m.MOE_OK


# ------------------------------------------------------------ append
def _append(m, kv, **kw):
    a = dict(k=AT, ks=256, v=AT, vs=256, dt=1, slots=AT, N=5)
    a.update(kw)
    return m.lib().moe_kv_append(None if kv is None else C.byref(kv), a["k"], a["ks"], a["v"], a["vs"], a["dt"], a["slots"], a["N"], None)


@pytest.mark.parametrize("kw", [dict(N=-1), dict(dt=2), dict(k=None), dict(v=None), dict(slots=None), dict(k=AT + 4), dict(v=AT + 8),
                                dict(slots=AT + 2), dict(ks=248), dict(vs=255), dict(ks=260), dict(dt=0, vs=258)])
def test_append_rejects_bad_arguments(m, kw):
    assert _append(m, _kv(m), **kw) == m.MOE_EINVAL
    assert m.last_error() != ""


# ------------------------------------------------------------ plan
def _plan(m, **kw):
    names = ["seq", "new", "R", "table", "mb", "page", "ring", "P", "pool", "seq_out", "first", "slots", "places", "cap", "pool_out", "status"]
    a = dict.fromkeys(names, AT)
    a.update(R=4, mb=8, page=16, P=100, cap=64, seq=AT + 64, new=AT + 128, pool=AT + 256)
    a.update(kw)
    return m.lib().moe_kv_plan(*[a[n] for n in names], None)


@pytest.mark.parametrize("kw", [
    dict(R=-1), dict(cap=-1), dict(mb=0), dict(page=0), dict(page=65537), dict(P=0), dict(seq=None), dict(new=None), dict(table=None),
    dict(ring=None), dict(pool=None), dict(seq_out=None), dict(first=None), dict(slots=None), dict(places=None), dict(pool_out=None),
    dict(status=None), dict(seq=AT + 1), dict(slots=AT + 2), dict(status=AT + 3), dict(seq=AT), dict(pool=AT), dict(new=AT)])
def test_plan_rejects_bad_arguments(m, kw):
    assert _plan(m, **kw) == m.MOE_EINVAL
    assert m.last_error() != ""


def test_plan_refuses_sizes_it_has_no_kernel_for(m):
    assert _plan(m, R=16385) == m.MOE_EUNSUPPORTED
    assert _plan(m, P=1 << 27) == m.MOE_EUNSUPPORTED


# ------------------------------------------------------------ route
def _rd(m, **kw):
    a = dict(E=64, K=4, score=1, n_group=8, keep_group=4, group_best=2, renorm=1, factor=1.0, bias=None)
    a.update(kw)
    return m.RouteDesc(**a)


def _route(m, rd, **kw):
    a = dict(z=AT, dt=0, stride=64, T=3, idx=AT, w=AT)
    a.update(kw)
    return m.lib().moe_scored_route(None if rd is None else C.byref(rd), a["z"], a["dt"], a["stride"], a["T"], a["idx"], a["w"], None)


@pytest.mark.parametrize("rd,kw", [
    (dict(E=0), {}), (dict(E=1025, n_group=1, keep_group=1), {}), (dict(K=0), {}), (dict(K=17), {}), (dict(K=9, keep_group=1), {}),
    (dict(score=2), {}), (dict(n_group=0), {}), (dict(n_group=7), {}), (dict(n_group=64, keep_group=64, group_best=1), {}),
    (dict(keep_group=0), {}), (dict(keep_group=9), {}), (dict(group_best=0), {}), (dict(group_best=3), {}),
    (dict(E=32, n_group=32, keep_group=8), {}), (dict(bias=AT + 2), {}), ({}, dict(T=-1)), ({}, dict(dt=2)), ({}, dict(z=None)),
    ({}, dict(idx=None)), ({}, dict(w=None)), ({}, dict(z=AT + 2)), ({}, dict(idx=AT + 2)), ({}, dict(w=AT + 1)), ({}, dict(stride=63)),
    ({}, dict(dt=1, z=AT + 1))])
def test_scored_route_rejects_bad_arguments(m, rd, kw):
    assert _route(m, _rd(m, **rd), **kw) == m.MOE_EINVAL
    assert m.last_error() != ""


def test_scored_route_needs_a_descriptor(m):
    assert _route(m, None) == m.MOE_EINVAL


# ------------------------------------------------------------ the binding
def test_binding_refuses_types_and_rows_it_cannot_pass_on(m):
    import torch
    kv, x = _kv(m), torch.zeros((3, 8, 128))
    with pytest.raises(TypeError):
        m.moe_paged_attention(kv, x, 3, 8, AT, AT, 4, 0.1, x.bfloat16(), AT)
    with pytest.raises(TypeError):
        m.moe_paged_attention(kv, x.half(), 3, 8, AT, AT, 4, 0.1, x.half(), AT)
    with pytest.raises(TypeError):
        m.moe_kv_append(kv, x, x.bfloat16(), AT, 3)
    with pytest.raises(ValueError):
        m.moe_kv_append(kv, x.transpose(1, 2), x, AT, 3, stream=0)
    with pytest.raises(TypeError):
        m.moe_scored_route(_rd(m), x[:, 0].half(), 3, AT, AT, stream=0)
    with pytest.raises(m.MoEError) as e:
        m.moe_paged_attention(kv, x, 3, 7, AT, AT, 4, 0.1, x, AT, stream=0)
    assert e.value.status == m.MOE_EINVAL


# ------------------------------------------------------------ the plan's arrays
_PLAN_R, _PLAN_MB, _PLAN_P, _PLAN_CAP = 6, 5, 40, 50
_PLAN_ARRAYS = dict(seq=("seq_len", _PLAN_R), new=("new_len", _PLAN_R), table=("block_table", _PLAN_R * _PLAN_MB), ring=("ring", _PLAN_P),
                    pool=("pool", 2), seq_out=("seq_out", _PLAN_R), first=("first", _PLAN_R + 1), slots=("slots", _PLAN_CAP),
                    places=("places", _PLAN_CAP), pool_out=("pool_out", 2), status=("status", 1))
_READ = ["seq", "new", "table", "ring", "pool"]
_PAIRS = [(w, r) for w in ("seq_out", "first", "slots", "places", "pool_out", "status") for r in _READ]
_PAIRS += [("ring", r) for r in ("seq", "new", "table", "pool")] + [("table", r) for r in ("seq", "new", "pool")]


@pytest.mark.parametrize("w,r", _PAIRS)
def test_plan_rejects_an_array_that_overlaps_what_is_read(m, w, r):
    """All arrays apart but two: the same address, the last number of one in
    the first place of the other, and the reverse."""
    base = {n: AT + 4096 * i for i, n in enumerate(_PLAN_ARRAYS)}
    nw, nr = _PLAN_ARRAYS[w][1], _PLAN_ARRAYS[r][1]
    for at in (base[r], base[r] + 4 * (nr - 1), base[r] - 4 * (nw - 1)):
        a = dict(base, R=_PLAN_R, mb=_PLAN_MB, P=_PLAN_P, cap=_PLAN_CAP)
        a[w] = at
        assert _plan(m, **a) == m.MOE_EINVAL
        said = m.last_error()
        assert "overlaps" in said and _PLAN_ARRAYS[w][0] in said and _PLAN_ARRAYS[r][0] in said, said


@pytest.mark.parametrize("what", [b"0123456789abcdef", "0123456789abcdef", 1.0, bytearray(16), [1, 2], object()])
def test_binding_takes_tensors_and_addresses_and_nothing_else(m, what):
    """ctypes would pass bytes and text on as addresses of the host."""
    import torch
    x, rd, kv = torch.zeros((3, 64)), _rd(m), _kv(m)
    with pytest.raises(AttributeError):
        m.moe_topk_route(what, 0, 64, 4, AT, AT, stream=0)
    with pytest.raises(AttributeError):
        m.moe_scored_route(rd, x, 0, what, AT, stream=0)
    with pytest.raises(AttributeError):
        m.moe_kv_append(kv, x, x, what, 0, stream=0)
    m.moe_scored_route(rd, x, 0, None, AT, stream=0)
