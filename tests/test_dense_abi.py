"""Refusals of the add-and-norm, the quantisation, the block-scaled product and
the rotary embedding, without a GPU: a rejected call never reaches the device,
an empty one returns before it touches a pointer."""
import ctypes as C

import pytest

from int4_expert_gemv_gb300 import build as nbuild

AT = 1 << 20          # a well aligned address that is never read
FAR = 1 << 32         # others, far from it and from each other
F32, BF16, E4M3 = 0, 1, 2


@pytest.fixture(scope="module")
def m():
    nbuild.build()
    from int4_expert_gemv_gb300 import moe
    moe.lib()
    return moe


def at(i):
    return i * FAR


# ------------------------------------------------------------ norm
def _norm(m, desc=None, **kw):
    d = dict(d=256, eps=1e-6, weight=at(9), w_dtype=BF16, pow2=0)
    d.update(desc or {})
    a = dict(x=at(1), xd=BF16, xs=256, res=at(2), rd=F32, rs=256, T=4, sum=at(3), ss=256, y=at(4), yd=E4M3, ys=256, sc=at(5), scs=2)
    a.update(kw)
    nd = m.NormDesc(**d)
    return m.lib().moe_add_rms_norm(C.byref(nd), a["x"], a["xd"], a["xs"], a["res"], a["rd"], a["rs"], a["T"], a["sum"], a["ss"], a["y"], a["yd"],
                                    a["ys"], a["sc"], a["scs"], None)


@pytest.mark.parametrize("desc", [dict(d=0), dict(d=-5), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(w_dtype=2),
                                  dict(weight=AT + 4), dict(pow2=2)])
def test_norm_rejects_a_bad_descriptor(m, desc):
    assert _norm(m, desc) == m.MOE_EINVAL and m.last_error() != ""


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x=at(1) + 8), dict(xd=2), dict(xd=7), dict(xs=248), dict(xs=260), dict(res=at(2) + 4), dict(rd=2), dict(rs=255), dict(rs=258),
    dict(res=None), dict(T=-1), dict(sum=at(3) + 8), dict(ss=252), dict(y=None), dict(y=at(4) + 8), dict(yd=3), dict(ys=255), dict(ys=264), dict(sc=None),
    dict(sc=at(5) + 2), dict(scs=1), dict(xs=1 << 62)])
def test_norm_rejects_bad_arguments(m, kw):
    assert _norm(m, **kw) == m.MOE_EINVAL and m.last_error() != ""


@pytest.mark.parametrize("kw", [
    dict(sum=at(2) + 16), dict(sum=at(2), ss=260), dict(sum=at(1)), dict(y=at(1)), dict(y=at(2)), dict(y=at(3) + 4080), dict(sc=at(4) + 64),
    dict(sc=at(2) + 4), dict(y=at(9)), dict(sum=at(9) + 256), dict(y=at(1), yd=F32, ys=256)])
def test_norm_rejects_overlaps(m, kw):
    assert _norm(m, **kw) == m.MOE_EINVAL and "overlaps" in m.last_error()


def test_norm_sizes(m):
    assert m.lib().moe_add_rms_norm(None, at(1), 0, 8, None, 0, 0, 1, None, 0, at(2), 0, 8, None, 0, None) == m.MOE_EINVAL
    assert _norm(m, dict(d=32769), xs=40000, rs=40000, ss=40000, ys=40000, scs=300) == m.MOE_EUNSUPPORTED
    assert _norm(m, T=0, x=None, res=None, sum=None, y=None, sc=None) == m.MOE_OK


# ------------------------------------------------------------ quantise
def _quant(m, **kw):
    a = dict(x=at(1), xd=BF16, xs=512, rows=200, cols=500, block=1, pow2=0, codes=at(2), cs=512, sc=at(3), scs=4)
    a.update(kw)
    return m.lib().moe_quantise_e4m3(a["x"], a["xd"], a["xs"], a["rows"], a["cols"], a["block"], a["pow2"], a["codes"], a["cs"], a["sc"], a["scs"], None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(cols=-1), dict(block=0), dict(block=64), dict(pow2=2), dict(xd=2), dict(x=None), dict(x=at(1) + 8), dict(xs=499), dict(xs=508),
    dict(codes=None), dict(codes=at(2) + 8), dict(cs=496), dict(cs=504), dict(sc=None), dict(sc=at(3) + 1), dict(scs=3), dict(codes=at(1)),
    dict(sc=at(1) + 64), dict(sc=at(2) + 64)])
def test_quantise_rejects_bad_arguments(m, kw):
    assert _quant(m, **kw) == m.MOE_EINVAL and m.last_error() != ""


def test_quantise_sizes(m):
    for kw in (dict(rows=0), dict(cols=0)):
        assert _quant(m, x=None, codes=None, sc=None, **kw) == m.MOE_OK
    assert _quant(m, rows=1 << 30, cols=1000, xs=1024, cs=1024, scs=8) == m.MOE_EUNSUPPORTED
    assert _quant(m, rows=65535 * 128 + 1, cols=8, xs=16, cs=16, block=128) == m.MOE_EUNSUPPORTED


# ------------------------------------------------------------ product
def _product(m, desc=None, **kw):
    d = dict(N=300, K=500, w=at(1), w_stride=512, scales=at(2), scale_stride=4)
    d.update(desc or {})
    a = dict(x=at(3), xs=512, sx=at(4), sxs=4, T=7, out=at(5), od=BF16, os=304, ws=at(6), wb=1 << 20)
    a.update(kw)
    wd = m.ScaledMatrixDesc(**d)
    return m.lib().moe_scaled_product(C.byref(wd), a["x"], a["xs"], a["sx"], a["sxs"], a["T"], a["out"], a["od"], a["os"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("desc", [dict(N=0), dict(K=0), dict(N=-1), dict(w=None), dict(w=at(1) + 8), dict(w_stride=496), dict(w_stride=504),
                                  dict(scales=None), dict(scales=at(2) + 2), dict(scale_stride=3)])
def test_product_rejects_a_bad_matrix(m, desc):
    assert _product(m, desc) == m.MOE_EINVAL and m.last_error() != ""


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x=at(3) + 4), dict(xs=496), dict(xs=510), dict(sx=None), dict(sx=at(4) + 1), dict(sxs=3), dict(T=-1), dict(out=None),
    dict(out=at(5) + 8), dict(od=2), dict(os=299), dict(os=300), dict(out=at(3)), dict(out=at(1) + 4096), dict(out=at(2)), dict(out=at(4)), dict(out=at(6)),
    dict(ws=at(3)), dict(ws=at(1))])
def test_product_rejects_bad_arguments(m, kw):
    assert _product(m, **kw) == m.MOE_EINVAL and m.last_error() != ""


def test_product_workspace_and_sizes(m):
    wd = m.ScaledMatrixDesc(N=300, K=500, w=at(1), w_stride=512, scales=at(2), scale_stride=4)
    need = m.moe_scaled_product_workspace_bytes(wd, 7)
    assert need > 0
    assert m.lib().moe_scaled_product_workspace_bytes(None, 7) == 0 and m.moe_scaled_product_workspace_bytes(wd, -1) == 0
    assert _product(m, ws=None) == m.MOE_ENOSPACE and _product(m, ws=at(6) + 64) == m.MOE_ENOSPACE and _product(m, wb=need - 1) == m.MOE_ENOSPACE
    assert _product(m, T=0, x=None, sx=None, out=None, ws=None) == m.MOE_OK
    assert m.lib().moe_scaled_product(None, at(3), 512, at(4), 4, 7, at(5), BF16, 304, at(6), 256, None) == m.MOE_EINVAL


# ------------------------------------------------------------ rotary
def _rd(m, **kw):
    a = dict(D=64, rot=32, first=16, layout=0, scaling=0, trained=4096, base=10000.0, factor=4.0, low=1.0, high=32.0, amplitude=1.0)
    a.update(kw)
    return m.RotaryDesc(**a)


def _rotary(m, desc=None, **kw):
    a = dict(turns=at(1), places=at(2), T=5, dt=BF16, q=at(3), qs=256, Hq=4, qo=at(4), qos=256, k=at(5), ks=128, Hk=2, ko=at(6), kos=128)
    a.update(kw)
    rd = _rd(m, **(desc or {}))
    return m.lib().moe_rotary(C.byref(rd), a["turns"], a["places"], a["T"], a["dt"], a["q"], a["qs"], a["Hq"], a["qo"], a["qos"], a["k"], a["ks"], a["Hk"],
                              a["ko"], a["kos"], None)


BAD_ROTARY = [dict(D=1), dict(D=1026), dict(rot=0), dict(rot=31), dict(rot=66), dict(first=-1), dict(first=33), dict(layout=2), dict(amplitude=float("nan")),
              dict(amplitude=float("inf"))]


@pytest.mark.parametrize("desc", BAD_ROTARY)
def test_rotary_rejects_a_bad_descriptor(m, desc):
    assert _rotary(m, desc) == m.MOE_EINVAL and m.last_error() != ""
    assert m.lib().moe_rotary_table(C.byref(_rd(m, **desc)), at(1), None) == m.MOE_EINVAL


@pytest.mark.parametrize("desc", [dict(scaling=-1), dict(scaling=5), dict(base=1.0), dict(base=float("inf")), dict(scaling=1, factor=0.5),
                                  dict(scaling=2, factor=float("nan")), dict(scaling=3, trained=0), dict(scaling=3, low=0.0), dict(scaling=4, high=1.0),
                                  dict(scaling=4, high=float("inf"))])
def test_rotary_table_rejects_bad_scalings(m, desc):
    assert m.lib().moe_rotary_table(C.byref(_rd(m, **desc)), at(1), None) == m.MOE_EINVAL and m.last_error() != ""


def test_rotary_table_rejects_a_bad_result(m):
    for turns in (None, at(1) + 4):
        assert m.lib().moe_rotary_table(C.byref(_rd(m)), turns, None) == m.MOE_EINVAL
    assert m.lib().moe_rotary_table(None, at(1), None) == m.MOE_EINVAL


@pytest.mark.parametrize("kw", [
    dict(turns=None), dict(turns=at(1) + 4), dict(places=None), dict(places=at(2) + 2), dict(T=-1), dict(dt=2), dict(q=None), dict(q=at(3) + 1), dict(qs=255),
    dict(Hq=-1), dict(Hk=65537), dict(qo=None), dict(qos=200), dict(k=None), dict(ks=127), dict(ko=None), dict(kos=100), dict(qo=at(3) + 16),
    dict(qo=at(3), qos=260), dict(qo=at(5)), dict(ko=at(4) + 64), dict(ko=at(3)), dict(qo=at(2)), dict(ko=at(1)), dict(dt=F32, q=at(3) + 2)])
def test_rotary_rejects_bad_arguments(m, kw):
    assert _rotary(m, **kw) == m.MOE_EINVAL and m.last_error() != ""


def test_rotary_of_nothing(m):
    assert _rotary(m, T=0, q=None, k=None, qo=None, ko=None, turns=None, places=None) == m.MOE_OK
    assert _rotary(m, Hq=0, Hk=0, q=None, k=None, qo=None, ko=None) == m.MOE_OK


# ------------------------------------------------------------ binding
def test_binding_refuses_types(m):
    import torch
    x, c = torch.zeros((2, 128)), torch.zeros((2, 128), dtype=torch.uint8)
    s = torch.zeros((2, 1))
    with pytest.raises(TypeError):
        m.moe_quantise_e4m3(x, 2, 128, x, s, stream=0)
    with pytest.raises(TypeError):
        m.moe_quantise_e4m3(x.half(), 2, 128, c, s, stream=0)
    with pytest.raises(TypeError):
        m.moe_quantise_e4m3(x, 2, 128, c, s.double(), stream=0)
    with pytest.raises(TypeError):
        m.moe_add_rms_norm(m.NormDesc(d=128), x, 2, x.clone(), res=x, sum=x.bfloat16(), stream=0)
    with pytest.raises(TypeError):
        m.moe_scaled_product(m.ScaledMatrixDesc(N=128, K=128), x, s, 2, x, c, stream=0)
    with pytest.raises(TypeError):
        m.moe_rotary(m.RotaryDesc(D=128, rot=128), c, c, 2, x, 1, x.bfloat16(), stream=0)
    with pytest.raises(ValueError):
        m.moe_quantise_e4m3(torch.zeros((128, 2)).t(), 2, 128, c, s, stream=0)


def test_paged_decoder_refuses_another_dense_type(m):
    from int4_expert_gemv_gb300 import paged
    with pytest.raises(ValueError):
        paged.PagedDecoder(None, None, 4, dense="int8")
