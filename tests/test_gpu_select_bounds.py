"""Where the selection's bound of a score's error is tight: weights too small
for the parts that the tensor cores multiply."""
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
