"""Decode attention over a 4-bit cache where tokens whose V rows are zeros stand
beside large values: the softmax's reference counts a weight times its scale, so
such tokens' weights are far from one, and their sum has to come through every
change of the reference: a warp's, the warps' join, a cluster's, the
partitions', the shares'."""
import numpy as np
import pytest
import torch

import paged_kv_cache_311_gb300 as pkv
from tests import q4_support as S
from tests.q8_support import DT, make_tables

pytestmark = pytest.mark.gpu
DEV = "cuda"


def scored(seed, *, t, D, bs, G, Hk, score, top):
    """One sequence whose token i has about the score score[i] (head g of a group: (1 + g / 8) times it) and, where
    top[i] is not 0, values between 0 and about top[i]: codes in half of the groups, a minimum alone in the others.
    Keys are constant in their first group, queries have a few dimensions there: scores are exact but for one rounding."""
    rng = np.random.RandomState(seed)
    dt, L = DT[t], len(score)
    q = np.zeros((1, Hk, G, D))
    q[..., :8] = (1 + np.arange(G)[:, None] / 8) / 8
    tables, NB = make_tables(rng, [-(-L // bs)])
    parts = {}
    for n in "kv":
        u = rng.randint(0, 16, (NB * bs, Hk, D // 64, 64)).astype(np.uint8)
        s, m = (np.full((NB * bs, Hk, D // 64), np.nan) for _ in "sm")
        at = (tables[0].astype(np.int64)[:, None] * bs + np.arange(bs)).reshape(-1)[:L]
        if n == "k":
            s[at], m[at] = 0.0, S.rounded(np.asarray(score), dt)[:, None, None]
        else:
            coded = rng.rand(L, Hk, D // 64) < 0.5
            each = np.asarray(top, np.float64)[:, None, None]
            s[at] = S.rounded(np.where(coded, each / 15, 0.0), dt)
            m[at] = S.rounded(np.where(coded, 0.0, each), dt)
        u, s, m = (a.reshape(NB, bs, *a.shape[1:]).swapaxes(1, 2) for a in (u, s, m))
        parts[n + "_parts"], parts[n] = (u, s, m), S.pack(u, s, m, dt)
    return dict(q=torch.from_numpy(q.reshape(1, Hk * G, D)).to(dt), tables=tables, lens=np.array([L], np.int32), NB=NB, Hk=Hk,
                G=G, D=D, bs=bs, t=t, scale=1.0, B=1, **parts)


def exact(c):
    """The row in 64 bits, and its sum of weights times the values' parts (15 s + |m|), all parts being positive."""
    (uk, sk, mk), (uv, sv, mv) = (c[n + "_parts"] for n in "kv")
    L, G = int(c["lens"][0]), c["G"]
    out, size = (np.zeros((c["Hk"] * G, c["D"])) for _ in range(2))
    q = c["q"].double().numpy()[0]
    for h in range(c["Hk"]):
        rows = lambda a: a[c["tables"][0], h].reshape(-1, *a.shape[3:])[:L]  # noqa: E731
        k = S.numbers(rows(uk), rows(sk), rows(mk))
        v = S.numbers(rows(uv), rows(sv), rows(mv))
        z = c["scale"] * (q[h * G:(h + 1) * G] @ k.T)
        p = np.exp(z - z.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        out[h * G:(h + 1) * G] = p @ v
        size[h * G:(h + 1) * G] = np.repeat(p @ (15 * rows(sv) + np.abs(rows(mv))), 64, -1)
    return out, size


def tolerance(L, size):
    """A score of up to 64 is one product and a few additions: off by 2^-22 of it, 2^-16 of the weight.  A weight's and a
    factor's exponent (differences of numbers below 2^8, log2) are rounded to 2^-17 and less, which is 2^-17.5 of the
    weight; a sum passes at most eight such factors: together below 2^-14.  Sums of positive numbers: a lane adds L / 8
    at most, off by 2^-24 each, the tensor cores' sums (both kinds of steps) stand at L / 8 cuts of 2^-23.  The quotient
    has all of it twice."""
    return 2 * (2.0 ** -14 + L / 8 * (2.0 ** -24 + 2.0 ** -23)) * size


def run(c, P, most=None):
    out = torch.full(tuple(c["q"].shape), float("nan"), device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    tables = c["tables"]
    if most:                                                # a table with room for it
        tables = np.pad(tables, ((0, 0), (0, max(0, -(-most // c["bs"]) - tables.shape[1]))), constant_values=-1)
    pkv.paged_attention_decode_q4(out, c["q"].to(DEV), dev(c["k"]), dev(c["v"]), dev(tables), dev(c["lens"]), c["scale"],
                                  max_context_len=most or int(c["lens"][0]), partition_size=P, device_status=st)
    assert st.item() == 0
    return out[0].double().cpu().numpy()


def cuts(L):
    """(partition_size, max_context_len): one CTA, partitions through the workspace, a cluster (or shares, where the row is
    long), shares."""
    return [(L // 32 * 32 + 32, None), (64, None), (32, None), (0, None), (0, 1 << 17)]


def check(c, which=None):
    want, size = exact(c)
    tol = tolerance(int(c["lens"][0]), size)
    for P, most in which or cuts(int(c["lens"][0])):
        got = run(c, P, most)
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), (P, most, np.argwhere(bad)[:3], got[bad][:3], want[bad][:3], tol[bad][:3])


@pytest.mark.parametrize("t,top", [("f16", 1000.0), ("f16", 65000.0), ("bf16", 2.0 ** 70)])
@pytest.mark.parametrize("D,bs,G", [(128, 16, 3), (64, 8, 8)])
@pytest.mark.parametrize("zeros", [32, 64, 1024])
@pytest.mark.parametrize("first", [True, False])
def test_rows_of_zeros_beside_large_values(t, top, D, bs, G, zeros, first):
    """Tokens whose values are zeros before or behind 32 others, of scores 10 to 28 below or above theirs (14 to 40 in
    powers of two)."""
    for apart in (10.0, 14.25, 20.0, 23.5, 28.0, -10.0, -14.25, -20.0, -23.5, -28.0):
        score = np.concatenate([np.zeros(zeros), np.full(32, apart / 1.25)])
        tops = np.concatenate([np.zeros(zeros), np.full(32, top)])
        if not first:
            score, tops = score[::-1], tops[::-1]
        check(scored(zeros + G, t=t, D=D, bs=bs, G=G, Hk=2, score=score, top=tops))


@pytest.mark.parametrize("t,top,apart", [("f16", 1000.0, 14.25), ("f16", 65504.0, 10.0), ("bf16", 2.0 ** 80, 30.0)])
@pytest.mark.parametrize("place", [0, 700, 1023])
def test_one_token_among_rows_of_zeros(t, top, apart, place):
    """One token that is not zero, anywhere in 1024."""
    score, tops = np.zeros(1024), np.zeros(1024)
    score[place], tops[place] = apart, top
    for D, bs, G in ((128, 32, 1), (64, 16, 5)):
        check(scored(place, t=t, D=D, bs=bs, G=G, Hk=1, score=score, top=tops))


def test_65536_rows_of_zeros_before_one_token():
    for t, top, apart in (("f16", 1000.0, 14.25), ("bf16", 2.0 ** 60, 12.0)):
        score, tops = np.zeros(65537), np.zeros(65537)
        score[-1], tops[-1] = apart, top
        check(scored(1, t=t, D=64, bs=32, G=2, Hk=1, score=score, top=tops), [(65568, None), (2048, None), (0, None)])


@pytest.mark.parametrize("seed", range(6))
def test_sizes_and_scores_of_all_kinds(seed):
    """Stretches of tokens of very different sizes (none at all, 2^-60 to 2^80) and scores, in any order."""
    rng = np.random.RandomState(seed)
    score, tops = [], []
    for _ in range(rng.randint(3, 12)):
        n = int(2 ** rng.uniform(0, 8))
        score += [rng.uniform(-16, 16)] * n
        tops += [0.0 if rng.rand() < 0.5 else 2.0 ** rng.uniform(-60, 80)] * n
    check(scored(seed, t="bf16", D=(64, 128)[seed % 2], bs=(8, 16, 32)[seed % 3], G=1 + seed, Hk=2, score=score, top=tops))


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("D,G,first", [(64, 1, 5.4375), (128, 2, 4.8125), (64, 8, 2.90625)])
@pytest.mark.parametrize("zeros", [65536, 400000])
def test_sums_of_many_large_weights(t, D, G, first, zeros):
    """Tokens of zeros whose scores lie just below the step that would move the reference (7.86, log2, above the first
    ones'; the head with the largest): the most that a weight can be, 65,536 and 400,000 times, before a token whose
    value counts."""
    score, tops = np.full(zeros + 1, first), np.zeros(zeros + 1)
    score[:128] = 0.0                                       # the first unit of each warp
    score[-1], tops[-1] = first + np.log(zeros), 1000.0
    whole = (zeros // 32 * 32 + 32, None)
    check(scored(zeros, t=t, D=D, bs=32, G=G, Hk=1, score=score, top=tops), [whole, (2048, None), (0, None)])


def test_values_near_the_largest():
    """Scales of V from 2^80 to 2^122, where a weight is next to nothing and has to stay a number: sums of weights are
    kept scaled down."""
    for e in (80, 100, 115, 122):
        for n in (1, 40, 500):
            check(scored(e, t="bf16", D=128, bs=16, G=3, Hk=2, score=np.linspace(0, 3, n), top=np.full(n, 15 * 2.0 ** e)))
