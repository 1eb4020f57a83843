"""The selection's bound of a score's error, and where it is tight: weights too
small for the parts that the tensor cores multiply, what their sums drop, and
how close scores may be that the exact comparison tells apart."""
import numpy as np
import pytest
import torch

import paged_kv_cache_311_gb300 as pkv
from tests import q8_support as S
from tests.test_gpu_q8 import dev

pytestmark = pytest.mark.gpu
DEV = "cuda"
BLOCKS = {"one launch": 100, "two launches": 2200}


def select(q, sums, tables, lens, bs, K, first, last):
    sel = torch.full((len(lens), sums.shape[1], K), 99, dtype=torch.int32, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.select_blocks(sel, q.to(DEV), sums.to(DEV), dev(tables), dev(lens), bs, keep_first=first, keep_last=last, device_status=st)
    assert st.item() == 0
    s = sums.double().numpy()
    want = S.select_reference(q.double().numpy(), s[:, :, 0], s[:, :, 1], tables, lens, bs, K, first, last)
    return sel.cpu().numpy(), want


@pytest.mark.parametrize("path", list(BLOCKS))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sign", [1, -1])
def test_weights_below_f16s_last_bit(path, D, sign):
    """One dimension of q is 60000, where every summary is 0; the weights that
    tell the blocks apart are 2^-25 and 1.5 * 2^-25 of the scaled row, so the
    parts hold 0 and 2^-24.  Block 5 adds up 20 of the small ones, block 9 eight
    of the larger: 5 is ahead, and its parts' score is 0."""
    n, bs = BLOCKS[path], 8
    assert (pkv.select_blocks_workspace_bytes(1, 1, n * bs, bs) > 0) == (path == "two launches")
    tables, NB = S.make_tables(np.random.RandomState(n), [n])
    q = torch.zeros(1, 8, D, dtype=torch.float16)
    q[0, :, 0] = 60000.0
    q[0, 0, 1:21], q[0, 0, 21:29] = 2.0 ** -21 * sign, 1.5 * 2.0 ** -21 * sign
    sums = torch.zeros(NB, 1, 2, D, dtype=torch.float16)
    side = 1 if sign > 0 else 0
    sums[tables[0, 5], 0, side, 1:21] = sign
    sums[tables[0, 9], 0, side, 21:29] = sign
    lens = np.array([n * bs], np.int32)
    for K in (1, 2, 5):
        got, want = select(q, sums, tables, lens, bs, K, 0, 0)
        if K == 1:
            assert want[0, 0, 0] == 5
        np.testing.assert_array_equal(got, want)


def score_case(kind, D, t, seed):
    """q [B, Hk, D] (one head per kv head) and summaries of n blocks per sequence, by kind."""
    B, Hk, n = 17, 8, 1030
    rng = np.random.RandomState(seed)
    tables, NB = S.make_tables(rng, [n] * B)
    dt = S.DT[t]
    q, sums = np.ones((B, Hk, D)), np.zeros((NB, Hk, 2, D))
    if kind == "normal":
        q, sums = rng.randn(B, Hk, D), np.sort(rng.randn(NB, Hk, 2, D), axis=2)
    elif kind == "cut off":
        # one number, and behind it numbers just below 2^-23 of it: the bits that an aligned sum drops
        last = 2.0 - 2.0 ** (-9 if t == "f16" else -6)
        sums[:, :, 1] = last * 2.0 ** -14
        sums[:, :, 0] = -last * 2.0 ** -14
        at = rng.randint(0, D, (NB, Hk, 1))
        np.put_along_axis(sums[:, :, 1], at, 2.0 ** 10, -1)
        q = np.where(rng.rand(B, Hk, 1) < 0.5, 1.0, -1.0) * np.ones(D)
        sums[:, :, 0] = -sums[:, :, 1]
    elif kind == "cancel":
        # large numbers of both signs whose sum is small beside them
        x = rng.randn(NB, Hk, D) * 1000
        x[:, :, 1::2] = -x[:, :, ::2] * (1 + rng.randn(NB, Hk, D // 2) * 2.0 ** -8)
        sums[:, :, 0] = sums[:, :, 1] = x
        q = rng.rand(B, Hk, D) + 0.5
    elif kind == "wide":
        sign = lambda *s: np.where(rng.rand(*s) < 0.5, 1.0, -1.0)
        q = sign(B, Hk, D) * 2.0 ** rng.uniform(-14, 4, (B, Hk, D))
        sums = np.sort(sign(NB, Hk, 2, D) * 2.0 ** rng.uniform(-14, 4, (NB, Hk, 2, D)), axis=2)
    return torch.from_numpy(q).to(dt), torch.from_numpy(sums).to(dt), tables, n


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["normal", "cut off", "cancel", "wide"])
def test_scores_stay_within_their_bound(kind, D, t):
    """The scores that the tensor cores add up, read from the workspace (a
    row's keys first), against 64-bit ones: every one of them within the
    40 * 2^-23 of the sum of its terms' magnitudes that the bound is made of,
    2^-25 a weight more in f16.  (How many bits the tensor cores keep of a sum is
    not documented; this is what the bound rests on.)"""
    q, sums, tables, n = score_case(kind, D, t, D)
    B, Hk, bs = q.shape[0], q.shape[1], 8
    lens = np.full(B, n * bs, np.int32)
    ws = torch.zeros(pkv.select_blocks_workspace_bytes(B, Hk, n * bs, bs), dtype=torch.uint8, device=DEV)
    stride = -(-n // 4) * 4
    assert ws.numel() >= B * Hk * stride * 4
    sel = torch.zeros(B, Hk, 8, dtype=torch.int32, device=DEV)
    pkv.select_blocks(sel, q.to(DEV), sums.to(DEV), dev(tables), dev(lens), bs, workspace=ws)
    bits = ws[: B * Hk * stride * 4].cpu().numpy().view(np.uint32).reshape(B, Hk, stride)[:, :, :n]
    got = np.where(bits & 0x80000000, bits & 0x7FFFFFFF, ~bits).astype(np.uint32).view(np.float32).astype(np.float64)
    qd, sd = q.double().numpy(), sums.double().numpy()[tables]          # [B, n, Hk, 2, D]
    w = np.stack([-np.maximum(-qd, 0), np.maximum(qd, 0)], 2)           # [B, Hk, 2, D]
    terms = sd * w[:, None]
    exact = terms.sum((-1, -2)).transpose(0, 2, 1)
    size = np.abs(terms).sum((-1, -2)).transpose(0, 2, 1)
    scale = 2.0 ** (14 - np.floor(np.log2(np.abs(qd).max(-1))))[:, :, None]
    pad = 2.0 ** -25 * np.abs(sd).sum((-1, -2)).transpose(0, 2, 1) if t == "f16" else 0.0
    off = np.abs(got - exact * scale)
    print(f"{kind} {t} {D}: off by up to {((off - pad).clip(0) / (size * scale)).max() * 2 ** 23:.2f} x 2^-23 of the terms")
    assert (off <= 40 * 2.0 ** -23 * size * scale + pad).all()


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("path", list(BLOCKS))
def test_scores_close_to_each_other(path, t):
    """Scores that differ by multiples of 2^-39 of the sum of their terms'
    magnitudes (f16), of 2^-40.6 of it (bfloat16, where two terms cancel): told
    apart; equal summaries go to the lower block."""
    n, bs, D = BLOCKS[path], 8, 128
    rng = np.random.RandomState(n)
    tables, NB = S.make_tables(rng, [n])
    x = np.zeros((NB, 1, D))
    if t == "bf16":   # two large numbers cancel; three of them in all
        perm = np.argsort(rng.rand(NB, D), -1)
        for k, v in ((0, 2.0 ** 13), (1, 2.0 ** 13), (2, -2.0 ** 13)):
            np.put_along_axis(x[:, 0], perm[:, k:k + 1], v, -1)
        at = perm[:, 3:4]
    else:
        perm = np.argsort(rng.rand(NB, D), -1)
        np.put_along_axis(x[:, 0], perm[:, :1], 2.0 ** 15, -1)
        at = perm[:, 1:2]
    np.put_along_axis(x[:, 0], at, rng.randint(1, 250, (NB, 1)) * 2.0 ** (-26 if t == "bf16" else -24), -1)
    x[tables[0, 60:80]] = x[tables[0, 40]]          # twenty-one alike
    sums = torch.from_numpy(np.stack([x, x], 2)).to(S.DT[t])
    assert torch.equal(sums[:, :, 0].double(), torch.from_numpy(x))
    q = torch.ones(1, 1, D, dtype=S.DT[t])
    for K in (1, 7, 45, 50, 55, 90):
        got, want = select(q, sums, tables, np.array([n * bs], np.int32), bs, K, 0, 0)
        np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("path", list(BLOCKS))
@pytest.mark.parametrize("qt,st", [("f16", "bf16"), ("bf16", "f16")])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -14, 2.0 ** 13])
def test_queries_and_summaries_of_different_types(path, qt, st, size):
    """What an 8-bit cache (bfloat16 summaries) of an f16 model gives, and the other way round."""
    n, bs, D = BLOCKS[path], 8, 64
    rng = np.random.RandomState(n)
    tables, NB = S.make_tables(rng, [n, n // 2])
    sums = torch.from_numpy(np.sort(rng.randn(NB, 2, 2, D), axis=2)).to(S.DT[st])
    q = torch.from_numpy(rng.randn(2, 10, D) * size).to(S.DT[qt])
    for K in (3, 20):
        got, want = select(q, sums, tables, np.array([n * bs, n // 2 * bs - 3], np.int32), bs, K, 1, 1)
        np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("alike", [False, True])
def test_the_longest_contexts(alike):
    """40,960 blocks, the most that a row may have; all alike: every one of them in doubt."""
    n, bs, D = 40960, 8, 64
    rng = np.random.RandomState(3)
    tables, NB = S.make_tables(rng, [n, 100])
    sums = torch.from_numpy(np.sort(rng.randn(NB, 1, 2, D), axis=2)).bfloat16()
    if alike:
        sums[:] = sums[0].clone()
    q = torch.from_numpy(rng.randn(2, 4, D)).bfloat16()
    for K in (1, 300, 40959):
        got, want = select(q, sums, tables, np.array([n * bs, 100 * bs], np.int32), bs, K, 0, 1)
        np.testing.assert_array_equal(got, want)
