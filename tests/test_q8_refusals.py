"""The 8-bit cache's and the block selection's calls refuse bad arguments on
the host: status codes of the C functions before any CUDA call, ValueErrors of
the Python binding (no GPU needed)."""
import ctypes
import os

import pytest
import torch

import paged_kv_cache_311_gb300 as pkv
from paged_kv_cache_311_gb300.build import build, library_path

vp = ctypes.c_void_p
A = 1 << 20
EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -4


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(library_path()):
        build()
    return pkv.load_library()


def append(lib, **kw):
    a = dict(key=A, value=A, dtype=2, kc=A, vc=A, ks=A, vs=A, bt=A, mb=8, cl=A, qs=A, B=2, T=5, Hk=2, D=128, bs=16, NB=64)
    a.update(kw)
    return lib.pkv_append_cache_q8(vp(a["key"]), vp(a["value"]), a["dtype"], vp(a["kc"]), vp(a["vc"]), vp(a["ks"]),
                                   vp(a["vs"]), vp(a["bt"]), a["mb"], vp(a["cl"]), vp(a["qs"]) if a["qs"] else None,
                                   a["B"], a["T"], a["Hk"], a["D"], a["bs"], a["NB"], None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), EINVAL), (dict(dtype=3), EINVAL), (dict(dtype=0), EUNSUPPORTED), (dict(D=96), EUNSUPPORTED),
    (dict(bs=24), EUNSUPPORTED), (dict(Hk=65536), EUNSUPPORTED), (dict(mb=1 << 28), EUNSUPPORTED), (dict(Hk=0), EINVAL),
    (dict(B=-1), EINVAL), (dict(T=-1), EINVAL), (dict(NB=0), EINVAL), (dict(NB=1 << 31), EINVAL), (dict(mb=0), EINVAL),
    (dict(qs=0), EINVAL),                       # without query_start one token per sequence
    (dict(key=0), EINVAL), (dict(ks=0), EINVAL), (dict(cl=0), EINVAL), (dict(key=A + 8), EINVAL), (dict(vc=A + 4), EINVAL),
    (dict(ks=A + 2), EINVAL), (dict(qs=A + 1), EINVAL), (dict(T=0), 0), (dict(B=0, T=0, qs=0, key=0), 0),
])
def test_append_host_checks(lib, kw, code):
    assert append(lib, **kw) == code


def summarize(lib, **kw):
    a = dict(kc=A, dt=2, ks=0, sm=A, sdt=2, bt=A, mb=8, cl=A, qs=A, B=2, T=5, Hk=2, D=128, bs=16, NB=64)
    a.update(kw)
    return lib.pkv_summarize_blocks(vp(a["kc"]), a["dt"], vp(a["ks"]) if a["ks"] else None, vp(a["sm"]), a["sdt"],
                                    vp(a["bt"]), a["mb"], vp(a["cl"]), vp(a["qs"]) if a["qs"] else None, a["B"], a["T"],
                                    a["Hk"], a["D"], a["bs"], a["NB"], None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=9), EINVAL), (dict(sdt=3), EINVAL), (dict(dt=0, sdt=0), EUNSUPPORTED), (dict(dt=1), EUNSUPPORTED),
    (dict(dt=3, ks=A, sdt=1), EUNSUPPORTED), (dict(dt=3), EINVAL), (dict(ks=A), EINVAL), (dict(sm=0), EINVAL),
    (dict(sm=A + 8), EINVAL), (dict(D=80), EUNSUPPORTED), (dict(bs=64), EUNSUPPORTED), (dict(qs=0), EINVAL), (dict(T=0), 0),
])
def test_summarize_host_checks(lib, kw, code):
    assert summarize(lib, **kw) == code


def select(lib, **kw):
    a = dict(sel=A, q=A, qdt=1, sm=A, sdt=2, bt=A, mb=64, cl=A, B=2, H=8, Hk=2, D=128, bs=16, NB=64, maxL=1000, K=8, first=1, last=2, ws=None, wsb=0)
    a.update(kw)
    return lib.pkv_select_blocks(vp(a["sel"]), vp(a["q"]), a["qdt"], vp(a["sm"]), a["sdt"], vp(a["bt"]), a["mb"], vp(a["cl"]),
                                 a["B"], a["H"], a["Hk"], a["D"], a["bs"], a["NB"], a["maxL"], a["K"], a["first"], a["last"],
                                 a["ws"], a["wsb"], None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(H=7), EINVAL), (dict(H=18), EUNSUPPORTED), (dict(maxL=1025), EINVAL), (dict(K=0), EINVAL), (dict(K=2), EINVAL),
    (dict(first=-1), EINVAL), (dict(last=2147483647), EINVAL), (dict(qdt=0), EUNSUPPORTED), (dict(sdt=0), EUNSUPPORTED),
    (dict(qdt=3), EINVAL), (dict(D=32), EUNSUPPORTED), (dict(mb=1 << 20, maxL=40961 * 16), EUNSUPPORTED),
    (dict(sel=0), EINVAL), (dict(q=A + 4), EINVAL), (dict(B=65536), EUNSUPPORTED), (dict(B=0, sel=0), 0),
    (dict(B=4096, mb=4096, maxL=65536), EWORKSPACE), (dict(B=4096, mb=4096, maxL=65536, ws=vp(A), wsb=4096 * 2 * 4096), EWORKSPACE),
    (dict(B=4096, mb=4096, maxL=65536, ws=vp(A + 8), wsb=1 << 40), EWORKSPACE),
])
def test_select_host_checks(lib, kw, code):
    assert select(lib, **kw) == code


def decode(lib, selected=False, **kw):
    a = dict(out=A, odt=0, q=A, qdt=1, kc=A, vc=A, kdt=3, ks=A, vs=A, bt=A, mb=8, cl=A, sel=A, K=4, B=2, H=4, Hk=2, D=128,
             bs=16, NB=64, maxL=100, scale=0.1, P=0, ws=None, wsb=0)
    a.update(kw)
    p = lambda x: vp(x) if x else None
    if selected:
        return lib.pkv_paged_attention_decode_selected(
            p(a["out"]), a["odt"], p(a["q"]), a["qdt"], p(a["kc"]), p(a["vc"]), a["kdt"], p(a["ks"]), p(a["vs"]), p(a["bt"]),
            a["mb"], p(a["cl"]), p(a["sel"]), a["K"], a["B"], a["H"], a["Hk"], a["D"], a["bs"], a["NB"], a["maxL"],
            ctypes.c_float(a["scale"]), a["P"], a["ws"], a["wsb"], None, None)
    return lib.pkv_paged_attention_decode_q8(
        p(a["out"]), a["odt"], p(a["q"]), a["qdt"], p(a["kc"]), p(a["vc"]), p(a["ks"]), p(a["vs"]), p(a["bt"]), a["mb"],
        p(a["cl"]), a["B"], a["H"], a["Hk"], a["D"], a["bs"], a["NB"], a["maxL"], ctypes.c_float(a["scale"]), a["P"],
        a["ws"], a["wsb"], None, None)


@pytest.mark.parametrize("selected", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(H=5), EINVAL), (dict(H=18), EUNSUPPORTED), (dict(odt=3), EINVAL), (dict(qdt=3), EINVAL), (dict(qdt=0), EUNSUPPORTED),
    (dict(D=96), EUNSUPPORTED), (dict(bs=24), EUNSUPPORTED), (dict(maxL=129), EINVAL), (dict(scale=float("inf")), EINVAL),
    (dict(scale=float("nan")), EINVAL), (dict(P=48), EINVAL), (dict(P=-32), EINVAL), (dict(out=0), EINVAL), (dict(ks=0), EINVAL),
    (dict(vs=0), EINVAL), (dict(kc=A + 8), EINVAL), (dict(q=A + 2), EINVAL), (dict(vs=A + 2), EINVAL), (dict(B=65536), EUNSUPPORTED),
    (dict(B=0, out=0, q=0, kc=0), 0), (dict(P=32), EWORKSPACE), (dict(P=32, ws=vp(A), wsb=16), EWORKSPACE),
    (dict(P=32, ws=vp(A + 8), wsb=1 << 30), EWORKSPACE),
])
def test_decode_host_checks(lib, selected, kw, code):
    assert decode(lib, selected, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(sel=0), EINVAL), (dict(K=0), EINVAL), (dict(sel=A + 2), EINVAL), (dict(kdt=1), EINVAL), (dict(kdt=2, ks=0, vs=0), EINVAL),
    (dict(kdt=7), EINVAL), (dict(kdt=0, qdt=0, ks=0, vs=0), EUNSUPPORTED),
])
def test_selected_host_checks(lib, kw, code):
    assert decode(lib, True, **kw) == code


def test_list_workspace(lib):
    w = lib.pkv_paged_attention_list_workspace_bytes
    # 100 tokens in 32-token partitions: 4 partials of (max, sum) and 128 sums for each of 2 x 4 rows
    assert w(2, 4, 2, 128, 16, 7, 32) == ((2 * 4 * 4 * 8 + 255) // 256) * 256 + 2 * 4 * 4 * 128 * 4
    assert w(2, 4, 2, 128, 16, 7, 1024) == 0
    assert w(0, 4, 2, 128, 16, 7, 0) == 0 and w(2, 4, 2, 128, 16, 7, 40) == 0 and w(2, 4, 2, 128, 16, 0, 0) == 0
    assert w(65535, 65535, 8191, 128, 8, 1 << 28, 32) == 0     # past 64 bits: the call then refuses


def test_select_workspace(lib):
    w = lib.pkv_select_blocks_workspace_bytes
    assert w(4, 8, 8192, 16) == 0                                       # one launch
    # 4096 keys of each of 16 x 8 rows, then a bound for each 128 of them (a warp's)
    assert w(16, 8, 65536, 16) == 128 * 4096 * 4 + 128 * 32 * 4
    assert w(0, 8, 65536, 16) == 0 and w(16, 8, 40961 * 16, 16) == 0


def test_binding_refuses_host_tensors():
    z = torch.zeros
    kc = z(4, 2, 16, 128, dtype=torch.float8_e4m3fn)
    bt, cl = z(2, 2, dtype=torch.int32), z(2, dtype=torch.int32)
    q = z(2, 4, 128, dtype=torch.float16)
    sc = pkv.q8_scales(4, 2)
    assert sc.shape == (4, 4) and sc.dtype == torch.float32 and not sc.any()
    with pytest.raises(ValueError, match="CUDA"):
        pkv.append_cache_q8(z(2, 2, 128, dtype=torch.float16), z(2, 2, 128, dtype=torch.float16), kc, kc, sc, sc, bt, cl)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_attention_decode_q8(q, q, kc, kc, sc, sc, bt, cl, 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_attention_decode_selected(q, q, kc, kc, bt, cl, z(2, 2, 4, dtype=torch.int32), 1.0, k_scales=sc, v_scales=sc)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.select_blocks(z(2, 2, 4, dtype=torch.int32), q, z(4, 2, 2, 128, dtype=torch.float16), bt, cl, 16)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.summarize_blocks(kc, z(4, 2, 2, 128, dtype=torch.bfloat16), bt, cl, k_scales=sc)
