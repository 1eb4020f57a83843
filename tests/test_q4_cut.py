"""The host model of the 4-bit decode's cut: every unit of every row is some
share's, once; a row that is cut leaves a unit to every warp; and the sizes that
the GPU tests take reach every way in which a chunk ends."""
import numpy as np
import pytest

from tests.q4_cut import CHUNK, CTAS, UNIT, WARPS, all_chunks

#: A batch whose shares are longer than a chunk although its rows are shorter, as tests/test_gpu_q4_cut.py takes it.
RAGGED = np.random.RandomState(64).randint(128, 2049, 64)


@pytest.mark.parametrize("lens,heads", [(RAGGED, 32), ([131067], 64), ([1] * 2000, 3), ([5000, 0, 31, 32, 33, 0, 70000], 5),
                                        ([4097] * 150, 8), ([130 * 32] * 300, 4)])
def test_every_unit_once(lens, heads):
    for sms in (152, 148, 7):
        seen = {}
        for share in all_chunks(lens, heads, sms):
            last = {}
            for pieces, how in share:
                assert 0 < sum(p[3] for p in pieces) <= CHUNK
                for s, h, u, n in pieces:
                    assert n > 0
                    seen.setdefault((s, h), []).append((u, n))
                    # a row that is not fresh: each warp has a unit in the piece that may be its last
                    if (s, h) in last:
                        assert n >= WARPS
                    last = {(s, h): True}
        for s, length in enumerate(lens):
            for h in range(heads):
                at = 0
                for u, n in sorted(seen.get((s, h), [])):
                    assert u == at
                    at += n
                assert at == -(-int(length) // UNIT)


def test_the_ragged_batch_reaches_every_end_of_a_chunk():
    ends, carried = {}, 0
    for share in all_chunks(RAGGED, 32, 152):
        for i, (pieces, how) in enumerate(share):
            ends[how] = ends.get(how, 0) + 1
            if i + 1 < len(share) and len(pieces) > 1 and share[i + 1][0][0][:2] == pieces[-1][:2]:
                carried += 1                                # begun inside a chunk, goes on in the next
    assert ends["row"] >= 20 and carried >= 100
    # no row here is longer than a chunk; one context is, and may end a few units behind it
    long_ends = {how for share in all_chunks([131067], 64, 152) for _, how in share}
    assert CTAS * 152 == 456 and "" in long_ends


def test_rows_a_little_longer_than_a_chunk_leave_a_unit_to_every_warp():
    ends = [how for share in all_chunks([(CHUNK + 2) * UNIT] * 300, 4, 152) for _, how in share]
    assert ends.count("four") >= 40
