"""Attention over an 8-bit cache and over selected blocks on the GPU, where an
error of the softmax weights shows: values that cancel, so that the output is
small beside them; weights close to each other; many that are tiny beside one
whose value is 0."""
import numpy as np
import pytest
import torch

import paged_kv_cache_311_gb300 as pkv
from tests import q8_support as S
from tests.test_gpu_q8 import dev

pytestmark = pytest.mark.gpu
DEV = "cuda"
# a weight's two parts: half a step of the part's type, twice
SPLIT = {"q8": 2.0 ** -22, "f16": 2.0 ** -22, "bf16": 2.0 ** -16}
E4M3 = {float(x): b for b, x in enumerate(S.TABLE) if not np.isnan(x)}


def tolerance(ref, size, bound, L, D, kind, out_dtype):
    """How far a row may be from the 64-bit one, element by element; `size`:
    sum_i w_i |v_i|.  A score is a sum of D products in fp32 (D + 4 roundings
    with the scales): off by ds <= (D + 4) 2^-24 * bound, and every weight by
    a factor within e^(2 ds); by 2^-20 for the exponential and the division, by
    its split into two parts, and the sums over L tokens round L times.  A
    16-bit output adds half a step."""
    rel = np.expm1(2 * (D + 4) * 2.0 ** -24 * bound) + 2.0 ** -20 + SPLIT[kind] + (L + 8) * 2.0 ** -24
    tol = rel[..., None] * size
    if out_dtype != torch.float32:
        tiny = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}[out_dtype]
        tol = tol + (np.abs(ref) + tol) * torch.finfo(out_dtype).eps / 2 + tiny
    return tol


def cache(kind, k, v, bs):
    """Tokens' k, v [L, D] (values that e4m3 holds) of one sequence and kv head as a cache in random places."""
    L, D = k.shape
    n = -(-L // bs)
    tables, NB = S.make_tables(np.random.RandomState(L), [n])
    out = []
    for x in (k, v):
        full = np.zeros((NB, 1, bs, D))
        rows = np.zeros((n * bs, D))
        rows[:L] = x
        full[tables[0], 0] = rows.reshape(n, bs, D)
        if kind == "q8":
            bits = np.vectorize(E4M3.__getitem__, otypes=[np.uint8])(full + 0.0)
            out.append((full, dev(bits).view(torch.float8_e4m3fn), dev(np.ones((NB, 4), np.float32))))
        else:
            out.append((full, torch.from_numpy(full).to(S.DT[kind]).to(DEV), None))
    return tables, out


def attend(kind, q, tables, kv, L, bs, scale, out_dtype, P, listed):
    (_, k, ks), (_, v, vs) = kv
    out = torch.full(tuple(q.shape), float("nan"), dtype=out_dtype, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = (dev(tables), dev(np.array([L], np.int32)))
    if listed:
        sel = dev(np.arange(-(-L // bs), dtype=np.int32)[None, None])
        pkv.paged_attention_decode_selected(out, q.to(DEV), k, v, *args, sel, scale, k_scales=ks, v_scales=vs, partition_size=P,
                                            device_status=st)
    else:
        pkv.paged_attention_decode_q8(out, q.to(DEV), k, v, ks, vs, *args, scale, partition_size=P, device_status=st)
    assert st.item() == 0
    return out.double().cpu().numpy()


def compare(kind, q, k, v, L, bs, scale, out_dtypes, parts=(0,)):
    tables, kv = cache(kind, k, v, bs)
    lens, qd = np.array([L], np.int32), q.double().numpy()
    ref, bound = S.attention_reference(qd, kv[0][0], kv[1][0], tables, lens, bs, scale)
    size, _ = S.attention_reference(qd, kv[0][0], np.abs(kv[1][0]), tables, lens, bs, scale)
    for out_dtype in out_dtypes:
        tol = tolerance(ref, size, bound, L, q.shape[2], kind, out_dtype)
        for P in parts:
            for listed in (False, True) if kind == "q8" else (True,):
                got = attend(kind, q, tables, kv, L, bs, scale, out_dtype, P, listed)
                bad = ~(np.abs(got - ref) <= tol)
                assert not bad.any(), (out_dtype, P, listed, np.argwhere(bad)[:3], got[bad][:3], ref[bad][:3], tol[bad][:3])


@pytest.mark.parametrize("kind", ["q8", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("L", [2, 64, 1000])
def test_values_that_cancel(kind, D, bs, L):
    """Half the tokens have scores 2^-8 to 2^-5 and the value -448, the others
    score 0 and the value 448: the output is a hundredth of the values and all
    of it is the weights' difference.  (Weights in one f16 part would be off by
    up to 2^-12 in it, bfloat16's half step there is 2^-8 * 448 * 2^-7.)"""
    k, v = np.zeros((L, D)), np.full((L, D), 448.0)
    k[1::2, 0], v[1::2] = 1.0, -448.0
    t = "bf16" if kind == "q8" else kind
    for types in (("bf16", "f16") if kind == "q8" else (t,)):
        q = torch.zeros(1, 8, D)
        q[0, :, 0] = torch.tensor([1.0, -1.25, 1.5, 1.75, -2.25, 3.5, 5.0, -7.0])
        compare(kind, q.to(S.DT[types]), k, v, L, bs, 2.0 ** -8, (torch.float32, torch.float16, torch.bfloat16), (0, 32))


@pytest.mark.parametrize("kind", ["q8", "f16", "bf16"])
@pytest.mark.parametrize("L", [1, 33, 500])
def test_scores_near_zero(kind, L):
    """Queries of 2^-20: scores and their errors vanish, the weights are all
    but equal and only the arithmetic behind the scores can be off."""
    rng = np.random.RandomState(L)
    D = 128
    k = S.nearest(np.clip(rng.randn(L, D) * 60, -448, 448))
    v = S.nearest(np.clip(rng.randn(L, D) * 60, -448, 448))
    q = torch.from_numpy(rng.randn(1, 8, D) * 2.0 ** -20).to(S.DT["bf16" if kind == "q8" else kind])
    compare(kind, q, k, v, L, 16, D ** -0.5, (torch.float32, torch.bfloat16), (0, 64))


@pytest.mark.parametrize("kind", ["q8", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 32])
def test_tiny_weights_that_count_together(kind, D, bs):
    """4096 tokens: four with a large score and the value 0 (the first of four
    tiles of 16), the others with weights of 2^-23 to 2^-30 of theirs and the
    value 448: the output is those weights' sum.  A weight in f16 parts may
    also be off by 2^-32 of the largest."""
    L = 4096
    k, v = np.zeros((L, D)), np.full((L, D), 448.0)
    k[[0, 16, 32, 48], 0], v[[0, 16, 32, 48]] = 16.0, 0.0
    x = torch.tensor([23.0, 23.5, 24.0, 25.0, 26.0, 27.0, 28.5, 30.0])   # all f16 and bfloat16 numbers
    for t in ("bf16", "f16") if kind == "q8" else (kind,):
        q = torch.zeros(1, 8, D)
        q[0, :, 0] = x
        scale = float(np.float32(np.log(2.0) / 16))
        tables, kv = cache(kind, k, v, bs)
        args = (q.double().numpy(), kv[0][0])
        lens = np.array([L], np.int32)
        ref, bound = S.attention_reference(*args, kv[1][0], tables, lens, bs, scale)
        w = np.exp(-scale * 16.0 * x.double().numpy())
        largest = 1 / (4 + (L - 4) * w)
        np.testing.assert_allclose(ref[0, :, 0], 448.0 * (L - 4) * w * largest, rtol=1e-12)
        for out_dtype in (torch.float32, torch.float16, torch.bfloat16):
            tol = tolerance(ref, ref, bound, L, D, kind, out_dtype)   # every value is positive
            if kind != "bf16":   # (rounded with the output)
                tol = tol + (2.0 ** -32 * largest * (L - 4) * 448.0)[None, :, None] * (1 + 2.0 ** -8)
            assert (tol < ref * 0.6).all()
            for P in (0, 4096):
                for listed in (False, True) if kind == "q8" else (True,):
                    got = attend(kind, q.to(S.DT[t]), tables, kv, L, bs, scale, out_dtype, P, listed)
                    bad = ~(np.abs(got - ref) <= tol)
                    assert not bad.any(), (out_dtype, P, listed, np.argwhere(bad)[:3], got[bad][:3], ref[bad][:3], tol[bad][:3])


@pytest.mark.parametrize("kind", ["q8", "f16", "bf16"])
@pytest.mark.parametrize("L", [1, 40, 700])
def test_scores_far_below_zero(kind, L):
    """Finite scores of -3e32, and some of -6e32: the first share all weight."""
    k, v = np.zeros((L, 64)), np.zeros((L, 64))
    k[:, 0], v[:] = -1.0, np.arange(1, 65) % 8
    k[1::3, 0], v[1::3] = -2.0, 448.0
    tables, kv = cache(kind, k, v, 8)
    q = torch.zeros(1, 8, 64, dtype=S.DT["bf16" if kind == "q8" else kind])
    q[0, :, 0] = 1.0
    for P in (0, 32, 2048):
        for listed in (False, True) if kind == "q8" else (True,):
            got = attend(kind, q, tables, kv, L, 8, 3e32, torch.float32, P, listed)
            # equal weights: only the sum and the division round
            np.testing.assert_allclose(got, np.broadcast_to(np.arange(1, 65) % 8, (1, 8, 64)), rtol=(L + 8) * 2.0 ** -24, atol=0)
