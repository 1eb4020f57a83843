"""The 4-bit cache's calls refuse bad arguments on the host: status codes of the
C functions before any CUDA call, ValueErrors of the Python binding (no GPU
needed)."""
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


def p(x):
    return vp(x) if x else None


def rows(lib, gather=False, **kw):
    a = dict(key=A, kst=256, value=A, vst=256, dtype=2, odt=2, kc=A, vc=A, slots=A, T=5, Hk=2, D=128, bs=16, NB=64)
    a.update(kw)
    tail = (p(a["slots"]), a["T"], a["Hk"], a["D"], a["bs"], a["NB"], None, None)
    if gather:
        return lib.pkv_gather_cache_q4(p(a["key"]), a["kst"], p(a["value"]), a["vst"], a["odt"], p(a["kc"]), p(a["vc"]),
                                       a["dtype"], *tail)
    return lib.pkv_reshape_and_cache_q4(p(a["key"]), a["kst"], p(a["value"]), a["vst"], a["dtype"], p(a["kc"]), p(a["vc"]), *tail)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), EINVAL), (dict(dtype=3), EINVAL), (dict(dtype=-1), EINVAL), (dict(dtype=0, odt=0), EUNSUPPORTED),
    (dict(D=96), EUNSUPPORTED), (dict(D=256), EUNSUPPORTED), (dict(bs=24), EUNSUPPORTED), (dict(bs=64), EUNSUPPORTED),
    (dict(Hk=65536, kst=1 << 24, vst=1 << 24), EUNSUPPORTED), (dict(Hk=0), EINVAL), (dict(T=-1), EINVAL), (dict(NB=0), EINVAL),
    (dict(NB=1 << 31), EINVAL), (dict(D=0), EINVAL), (dict(bs=0), EINVAL),
    (dict(kst=255), EINVAL), (dict(vst=128), EINVAL), (dict(kst=260), EINVAL), (dict(kst=0), EINVAL), (dict(vst=-256), EINVAL),
    (dict(kst=1 << 62), EINVAL), (dict(key=0), EINVAL), (dict(value=0), EINVAL), (dict(kc=0), EINVAL), (dict(slots=0), EINVAL),
    (dict(key=A + 8), EINVAL), (dict(value=A + 2), EINVAL), (dict(vc=A + 4), EINVAL), (dict(slots=A + 4), EINVAL),
    (dict(T=0, key=0, kc=0, slots=0), 0),
])
def test_rows_host_checks(lib, gather, kw, code):
    assert rows(lib, gather, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(odt=1), EUNSUPPORTED), (dict(odt=3), EINVAL), (dict(odt=0, dtype=0), EUNSUPPORTED), (dict(odt=0, kst=258), EINVAL),
    (dict(odt=0, kst=252), EINVAL),
])
def test_gather_host_checks(lib, kw, code):
    assert rows(lib, True, **kw) == code


def decode(lib, **kw):
    a = dict(out=A, odt=0, q=A, qst=512, qdt=1, kc=A, vc=A, bt=A, mb=8, cl=A, B=2, H=4, Hk=2, D=128, bs=16, NB=64, maxL=100,
             scale=0.1, P=0, ws=None, wsb=0)
    a.update(kw)
    return lib.pkv_paged_attention_decode_q4(
        p(a["out"]), a["odt"], p(a["q"]), a["qst"], a["qdt"], p(a["kc"]), p(a["vc"]), p(a["bt"]), a["mb"], p(a["cl"]), a["B"],
        a["H"], a["Hk"], a["D"], a["bs"], a["NB"], a["maxL"], ctypes.c_float(a["scale"]), a["P"], a["ws"], a["wsb"], None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(H=5), EINVAL), (dict(H=18, qst=1 << 12), EUNSUPPORTED), (dict(odt=3), EINVAL), (dict(qdt=3), EINVAL),
    (dict(qdt=0), EUNSUPPORTED), (dict(D=96), EUNSUPPORTED), (dict(bs=24), EUNSUPPORTED), (dict(maxL=129), EINVAL),
    (dict(maxL=-1), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(P=48), EINVAL),
    (dict(P=-32), EINVAL), (dict(qst=511), EINVAL), (dict(qst=516), EINVAL), (dict(qst=0), EINVAL), (dict(qst=1 << 62), EINVAL),
    (dict(out=0), EINVAL), (dict(q=0), EINVAL), (dict(kc=0), EINVAL), (dict(cl=0), EINVAL), (dict(kc=A + 8), EINVAL),
    (dict(q=A + 2), EINVAL), (dict(bt=A + 2), EINVAL), (dict(B=65536), EUNSUPPORTED), (dict(NB=1 << 31), EINVAL), (dict(mb=0), EINVAL),
    (dict(B=0, out=0, q=0, kc=0), 0),
])
def test_decode_host_checks(lib, kw, code):
    assert decode(lib, **kw) == code


def test_binding_refuses_host_tensors():
    kc = pkv.q4_cache(4, 2, 16, 128)
    assert kc.shape == (4, 2, 16, 72) and kc.dtype == torch.uint8 and not kc.any()
    with pytest.raises(ValueError, match="64"):
        pkv.q4_cache(4, 2, 16, 96)
    x = torch.zeros(3, 2, 128, dtype=torch.float16)
    at = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.reshape_and_cache_q4(x, x, kc, kc, at)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.gather_cache_q4(x, x, kc, kc, at)
    with pytest.raises(ValueError, match="dtype"):
        pkv.gather_cache_q4(x, x, kc, kc, at, dtype=torch.int32)
    q = torch.zeros(3, 4, 128, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_attention_decode_q4(q, q, kc, kc, torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), 1.0)
