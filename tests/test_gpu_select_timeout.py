"""What a block selection makes of a wait that gave up, run on the GPU by the
test hook pkv_test_select_timeout (a barrier that nothing completes, bounded
waits that return): the row selects nothing, the timeout is reported whoever
noticed it, and no block id is blamed for it."""
import ctypes

import pytest
import torch

import paged_kv_cache_311_gb300 as pkv

EINVAL = -1


@pytest.mark.gpu
@pytest.mark.parametrize("what,bits", [
    (0, pkv.DEV_TIMEOUT | pkv.DEV_DRAIN_TIMEOUT),   # noticed by all threads but the one that reports
    (1, 0),                                         # reported where it happened, and not as a bad block
    (2, pkv.DEV_BAD_BLOCK),
])
@pytest.mark.parametrize("K", [1, 99])
def test_a_row_whose_wait_gave_up_selects_nothing(what, bits, K):
    sel = torch.full((K,), 7, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.select_timeout_hook(what, sel, st, 1_000_000)
    torch.cuda.synchronize()
    assert st.item() == bits and (sel == -1).all()


def test_hook_checks_its_arguments_on_the_host():
    fn = pkv.load_library().pkv_test_select_timeout
    p = ctypes.c_void_p(1 << 20)
    for a in ((-1, 1, p, 5, p), (3, 1, p, 5, p), (0, 0, p, 5, p), (0, 2_000_000_001, p, 5, p), (0, 1, None, 5, p), (0, 1, p, 0, p),
              (0, 1, p, 100, p), (0, 1, p, 5, None)):
        assert fn(*a, None) == EINVAL
