"""What decode attention over a 4-bit cache makes of a wait that gave up, run on
the GPU by the test hook pkv_test_q4_timeout (copies that are never issued, bounded
waits that return): the rows that the CTA still has a part in are zero, all others
as ever, and the next call is, too."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_311_gb300 as pkv
from tests.q4_cut import WARPS, Rows, all_chunks
from tests.test_q4_cut import RAGGED

EINVAL = -1
BOTH = pkv.DEV_TIMEOUT | pkv.DEV_DRAIN_TIMEOUT


def lose(rows, cta, warp, unit, most, P=0):
    out = torch.full(rows.q.shape, float("nan"), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = torch.nn.functional.pad(rows.tables, (0, max(0, -(-most // rows.bs) - rows.tables.shape[1])), value=-1)
    need = pkv.paged_attention_q4_workspace_bytes(len(rows.lens), rows.Hk * rows.G, rows.Hk, rows.D, rows.bs, most, P)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    pkv.q4_timeout_hook(cta, warp, unit, out, rows.q, rows.k, rows.v, t, rows.context, 1.0, st, 1_000_000, max_context_len=most,
                        partition_size=P, workspace=ws)
    return out.view(len(rows.lens), rows.Hk, rows.G, rows.D), int(st.item())


@pytest.mark.gpu
@pytest.mark.parametrize("cta,warp,unit", [(0, 0, 0), (17, 3, 1), (100, 2, 20), (201, 1, 31), (300, 0, 32), (455, 1, 33)])
def test_a_share_whose_copies_do_not_come(cta, warp, unit):
    """Shares of several chunks and rows: rows that the CTA finished before are right; the one in which the wait gave up
    and the share's others are zero, those too of which other CTAs have parts."""
    lens = RAGGED
    rows = Rows(pkv, 6, lens, dtype=torch.bfloat16, Hk=32, G=2, D=64, bs=16)
    good, st = rows.decode(most=2080)
    assert st == 0
    share = all_chunks(lens, 32, torch.cuda.get_device_properties(0).multi_processor_count)[cta]
    # the warp's units, in order: every fourth of a chunk
    taken = [piece for chunk, _ in share for i, piece in enumerate([p[:2] for p in chunk for _ in range(p[3])]) if i % WARPS == warp]
    order = list(dict.fromkeys(p[:2] for chunk, _ in share for p in chunk))
    want = good.clone()
    for s, h in order[order.index(taken[unit]):]:
        want[s, h] = 0
    got, st = lose(rows, cta, warp, unit, 2080)
    assert st == BOTH and torch.equal(got, want)
    again, st = rows.decode(most=2080)
    assert st == 0 and torch.equal(again, good)
    got, st = lose(rows, 1 << 20, 0, 0, 2080)               # a CTA that is not there
    assert st == 0 and torch.equal(got, good)


@pytest.mark.gpu
@pytest.mark.parametrize("P", [0, 64, 1024])
@pytest.mark.parametrize("warp,unit", [(0, 0), (2, 0), (1, 1)])
def test_a_part_whose_copies_do_not_come(P, warp, unit):
    """Clusters, partitions through the workspace: the row is zero if the unit is there."""
    lens, Hk = (3000, 40, 2000), 4
    rows = Rows(pkv, 7, lens, dtype=torch.bfloat16, Hk=Hk, G=4, D=64, bs=16)
    good, st = rows.decode(P=P)
    assert st == 0
    grid = 8 if P == 0 else -(-3000 // P)
    units = [-(-n // 32) for n in lens]
    for x, h, s in ((0, 0, 0), (1, 3, 2), (grid - 1, 2, 0), (0, 1, 1)):
        part = P // 32 if P else -(-units[s] // grid)
        there = min(part, units[s] - x * part)              # units of the CTA
        want = good.clone()
        if warp + unit * WARPS < there:
            want[s, h] = 0
        got, st = lose(rows, (s * Hk + h) * grid + x, warp, unit, 3000, P)
        assert torch.equal(got, want) and st == (BOTH if warp + unit * WARPS < there else 0)


@pytest.mark.gpu
def test_whole_rows_whose_copies_do_not_come():
    lens = np.full(100, 500)
    rows = Rows(pkv, 8, lens, dtype=torch.bfloat16, Hk=8, G=1, D=64, bs=16)
    good, st = rows.decode()
    assert st == 0
    for cta, warp, unit in ((0, 0, 0), (399, 3, 3), (799, 1, 2)):
        want = good.clone()
        want[cta // 8, cta % 8] = 0
        got, st = lose(rows, cta, warp, unit, 500)
        assert st == BOTH and torch.equal(got, want)


def test_hook_checks_its_arguments_on_the_host():
    fn = pkv.load_library().pkv_test_q4_timeout
    A = ctypes.c_void_p(1 << 20)
    good = [1000, 0, 0, 0, A, A, A, A, A, 8, A, 2, 4, 2, 64, 100, 1.0, 0, None, 0, A, None]
    for i, bad in ((0, 0), (0, 2_000_000_001), (1, -1), (2, 4), (2, -1), (3, -1), (4, None), (12, 10), (13, 0), (15, 129), (20, None)):
        assert fn(*good[:i], bad, *good[i + 1:]) == EINVAL
