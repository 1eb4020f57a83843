"""Decode attention over a 4-bit cache where its work is cut: shares of several
chunks, rows that begin and end anywhere in them, partitions of every size.  The
rows' values have a level of their own for each stretch of tokens, the tolerance
is checked against what a lost piece would change."""
import numpy as np
import pytest
import torch

import paged_kv_cache_311_gb300 as pkv
from tests.q4_cut import UNIT, Rows, all_chunks
from tests.test_q4_cut import RAGGED

pytestmark = pytest.mark.gpu
DEV = "cuda"


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def check_row(rows, s, got, additions, pieces=None):
    """Sequence s's outputs [Hk, G, D], and that they would be refused without any of its pieces: {head: [(first unit,
    units)]}, each whole unit if none are given.  A piece that changes the exact output by more than twice the tolerance
    is missed by an output that lacks it and is itself off by no more than the tolerance."""
    den, num = rows.sums(s)
    want = num.sum(2) / den.sum(2)[..., None]
    tol = rows.tolerance(s, additions)
    off = (got.double() - want).abs()
    assert bool((off <= tol).all()), (s, float((off / tol).max()))
    if den.shape[2] == 1:
        return
    if pieces is None:
        without = (num.sum(2, keepdim=True) - num) / (den.sum(2, keepdim=True) - den)[..., None]
        tells = ((without - want[:, :, None]).abs() > 2 * tol[:, :, None]).any(-1)
        assert bool(tells[..., : rows.lens[s] // UNIT].all()), s
        return
    den0, num0 = (torch.nn.functional.pad(x.cumsum(2), p) for x, p in ((den, (1, 0)), (num, (0, 0, 1, 0))))
    for h, cuts in pieces.items():
        for u, n in cuts:
            if n == den.shape[2]:
                continue
            d = den0[h, :, -1] - (den0[h, :, u + n] - den0[h, :, u])
            x = num0[h, :, -1] - (num0[h, :, u + n] - num0[h, :, u])
            assert bool(((x / d[:, None] - want[h]).abs() > 2 * tol[h]).any(-1).all()), (s, h, u, n)


def ragged(dtype, D, seed):
    return Rows(pkv, seed, RAGGED, dtype=dtype, Hk=32, G=1 if D == 128 else 3, D=D, bs=16 if D == 128 else 8)


@pytest.mark.parametrize("dtype,D", [(torch.float16, 128), (torch.bfloat16, 128), (torch.bfloat16, 64)])
def test_shares_of_many_short_rows(dtype, D):
    """Shares longer than a chunk over rows shorter than one: chunks end in front of a row, rows begin in one chunk and go on
    in the next.  Every unit of every row counts."""
    found = [how for share in all_chunks(RAGGED, 32, sms()) for _, how in share]
    assert found.count("row") >= 20
    rows = ragged(dtype, D, 1)
    got, st = rows.decode(most=2080)                        # past 2048 tokens rows are not left whole
    assert st == 0
    for s in range(len(RAGGED)):
        check_row(rows, s, got[s], 64 + 16)


@pytest.mark.parametrize("D", [128, 64])
def test_bad_blocks_at_the_borders_of_chunks(D):
    """Sequences with a row that goes on in the next chunk, or in front of which one ends, get a bad block in the piece
    before the border, behind it, or at the row's end: all their rows are zero, all others as without."""
    rows = ragged(torch.bfloat16, D, 2)
    good, st = rows.decode(most=2080)
    assert st == 0
    where = {}
    for share in all_chunks(RAGGED, 32, sms()):
        for (pieces, how), (after, _) in zip(share, share[1:]):
            s, h, u, n = pieces[-1]
            s1, _, u1, n1 = after[0]
            if (s, h) == after[0][:2]:
                where.setdefault(s, []).extend([u + n - 1, u1, u1 + n1 - 1])
            elif how == "row":
                where.setdefault(s1, []).extend([0, n1 - 1])
    assert len(where) >= 20
    rng = np.random.RandomState(3)
    for hurt in (sorted(where)[::3], sorted(where)[1::5]):
        tables = rows.tables.clone()
        for s in hurt:
            unit = where[s][rng.randint(len(where[s]))]
            last = -(-int(RAGGED[s]) // rows.bs) - 1
            tables[s, min(last, unit * UNIT // rows.bs + rng.randint(UNIT // rows.bs))] = [-1, rows.NB][rng.randint(2)]
        got, st = rows.decode(most=2080, tables=tables)
        assert st == pkv.DEV_BAD_BLOCK
        rest = [s for s in range(len(RAGGED)) if s not in hurt]
        assert not got[hurt].any() and torch.equal(got[rest], good[rest])


@pytest.mark.parametrize("dtype,bs,G", [(torch.bfloat16, 32, 1), (torch.float16, 8, 4)])
def test_long_rows_in_shares_of_many_chunks(dtype, bs, G):
    """One context of 131,067 tokens, 64 kv heads: a share is some 575 units, its chunks end inside rows. A chunk's part of a
    row would be missed, and so would a share's."""
    L, Hk = 131067, 64
    rows = Rows(pkv, 4, [L], dtype=dtype, Hk=Hk, G=G, D=64, bs=bs, stretch=1024)
    got, st = rows.decode()
    assert st == 0
    pieces, most = {}, 0
    for share in all_chunks([L], Hk, sms()):
        most = max(most, sum(p[3] for c, _ in share for p in c))
        whole = {}
        for chunk, _ in share:
            for _, h, u, n in chunk:
                pieces.setdefault(h, []).append((u, n))
                first, so_far = whole.get(h, (u, 0))
                whole[h] = (first, so_far + n)
        for h, (u, n) in whole.items():
            pieces[h].append((u, n))
    assert most > 4 * 128 and len(pieces) == Hk
    # pieces of a few units next to a row's end tell less than a tolerance does
    pieces = {h: [p for p in cuts if p[1] >= 64] for h, cuts in pieces.items()}
    assert all(pieces.values())
    # a lane adds four tokens of each fourth unit; the merge adds the parts of a row, at most eight here
    check_row(rows, 0, got[0], most + 16, pieces)


@pytest.mark.parametrize("dtype,D,bs,G", [(torch.bfloat16, 128, 8, 4), (torch.float16, 64, 32, 8), (torch.bfloat16, 128, 16, 1)])
@pytest.mark.parametrize("lens,P", [((5000,), 0), ((5000,), 32), ((5000,), 1024), ((9000, 3), 0), ((9000, 3), 64), ((9000, 3), 4096),
                                    ((2, 4097, 1, 2049), 0), ((2, 4097, 1, 2049), 32), ((60000,), 60000), ((60000,), 2048), ((60000,), 0)])
def test_rows_of_thousands_of_tokens(dtype, D, bs, G, lens, P):
    """Few long rows: clusters, partitions through the workspace, one CTA, shares. Without any partition's (or each
    eighth of the row, where the cut is the library's) part of a row its output would be refused."""
    rows = Rows(pkv, 5, lens, dtype=dtype, Hk=1, G=G, D=D, bs=bs, stretch=max(UNIT, (P or 256) // 4 // UNIT * UNIT))
    got, st = rows.decode(P=P)
    assert st == 0
    for s, L in enumerate(lens):
        units = -(-L // UNIT)
        part = P // UNIT if P else -(-units // 8)
        cuts = [(u, min(part, units - u)) for u in range(0, units, part)]
        # a lane's additions of a part (four tokens of each fourth unit), and those of the parts
        check_row(rows, s, got[s], part + len(cuts) + 16, {0: [c for c in cuts if c[1] * UNIT * 64 >= L]})
