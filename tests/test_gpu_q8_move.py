"""Blocks of an 8-bit cache with scales and summaries, copied and swapped out
and back to other places: selection and attention over them stay the same."""
import numpy as np
import pytest
import torch

import paged_kv_cache_311_gb300 as pkv
from tests import q8_support as S
from tests.test_gpu_q8 import dev

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("Hk,D,bs", [(2, 128, 16), (5, 64, 8)])
@pytest.mark.parametrize("layers", [1, 2])
def test_selection_and_attention_follow_moved_blocks(Hk, D, bs, layers):
    rng = np.random.RandomState(Hk)
    lens, G, K = np.array([300, 77, 1]), 4, 5
    need = [-(-int(n) // bs) for n in lens]
    used, NB = S.make_tables(rng, need, NB=2 * sum(need) + 4)
    MB = used.shape[1]
    starts = dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
    r = lambda *s: torch.from_numpy(rng.randn(*s)).bfloat16().to(DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    bt, cl, n = dev(used), dev(lens.astype(np.int32)), int(lens.sum())
    caches = []
    for _ in range(layers):
        k, v = (torch.zeros(NB, Hk, bs, D, dtype=torch.float8_e4m3fn, device=DEV) for _ in "kv")
        ks, vs = pkv.q8_scales(NB, Hk, DEV), pkv.q8_scales(NB, Hk, DEV)
        sums = r(NB, Hk, 2, D)
        pkv.append_cache_q8(r(n, Hk, D) * 3, r(n, Hk, D), k, v, ks, vs, bt, cl, starts, device_status=st)
        pkv.summarize_blocks(k, sums, bt, cl, starts, num_tokens=n, k_scales=ks, device_status=st)
        caches.append([k, v, ks, vs, sums])
    q = [r(3, Hk * G, D) for _ in range(layers)]

    def step(tables):
        out = []
        for (k, v, ks, vs, sums), x in zip(caches, q):
            sel, o = torch.zeros(3, Hk, K, dtype=torch.int32, device=DEV), torch.zeros(3, Hk * G, D, device=DEV)
            pkv.select_blocks(sel, x, sums, dev(tables), cl, bs, keep_last=2, device_status=st)
            pkv.paged_attention_decode_selected(o, x, k, v, dev(tables), cl, sel, D ** -0.5, k_scales=ks, v_scales=vs, device_status=st)
            out += [sel.cpu(), o.cpu()]
        return out

    def kinds():
        """What moves, as the K and the V lists of one call each."""
        yield [c[0] for c in caches], [c[1] for c in caches]
        yield [c[2] for c in caches], [c[3] for c in caches]
        yield ([caches[0][4]], [caches[-1][4]])   # two layers', or one layer's in both places

    want = step(used)
    old = np.concatenate([used[s, :m] for s, m in enumerate(need)]).astype(np.int64)
    free = np.setdiff1d(np.arange(NB), old)
    new = rng.permutation(free)[: len(old)]
    place = dict(zip(old, new))
    moved = np.vectorize(lambda b: place.get(b, b), otypes=[np.int32])(used)

    for k, v in kinds():
        pkv.copy_blocks(k, v, dev(np.stack([old, new], 1)), device_status=st)
    assert all(torch.equal(a, b) for a, b in zip(want, step(moved)))

    # out to the host, the pool overwritten, back to a third arrangement
    host = [[[torch.zeros(len(old), *t.shape[1:], dtype=t.dtype).pin_memory() for t in ts] for ts in kv] for kv in kinds()]
    back = rng.permutation(NB)[: len(old)]
    slot = np.arange(len(old))
    for (k, v), (hk, hv) in zip(kinds(), host):
        pkv.swap_blocks(k, v, hk, hv, dev(np.stack([new, slot], 1)), pkv.SWAP_OUT, device_status=st)
    torch.cuda.synchronize()
    for c in caches:
        for t in c:
            t.view(torch.uint8).fill_(0x7F)
    for (k, v), (hk, hv) in zip(kinds(), host):
        pkv.swap_blocks(k, v, hk, hv, dev(np.stack([back, slot], 1)), pkv.SWAP_IN, device_status=st)
    place = dict(zip(old, back))
    again = np.vectorize(lambda b: place.get(b, b), otypes=[np.int32])(used)
    assert all(torch.equal(a, b) for a, b in zip(want, step(again)))
    assert st.item() == 0 and used.shape[1] == MB
