"""Selections of many rows of many blocks (two launches through the
workspace) queued between kernels that write their inputs just before each
call and overwrite them just after it."""
import numpy as np
import pytest
import torch

import paged_kv_cache_311_gb300 as pkv
from tests import q8_support as S
from tests.test_gpu_q8 import dev

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, Hk, G, D, bs, n, K, STEPS = 24, 8, 4, 64, 8, 1100, 40, 12


class Steps:
    def __init__(self, seed):
        assert pkv.select_blocks_workspace_bytes(B, Hk, n * bs, bs) > 0
        g = torch.Generator(device=DEV).manual_seed(seed)
        rng = np.random.RandomState(seed)
        tables, self.NB = S.make_tables(rng, [n] * B)
        self.all_tables = dev(np.stack([tables[rng.permutation(B)] for _ in range(STEPS)]))
        self.all_lens = dev(rng.randint(0, n * bs + 1, (STEPS, B)).astype(np.int32))
        self.all_q = torch.randn(STEPS, B, Hk * G, D, generator=g, device=DEV).bfloat16()
        self.all_sums = torch.sort(torch.randn(3, self.NB, Hk, 2, D, generator=g, device=DEV).bfloat16(), dim=3)[0].contiguous()
        self.tables, self.lens = torch.zeros_like(self.all_tables[0]), torch.zeros_like(self.all_lens[0])
        self.q, self.sums = torch.zeros_like(self.all_q[0]), torch.zeros_like(self.all_sums[0])
        self.sel = torch.zeros(B, Hk, K, dtype=torch.int32, device=DEV)
        self.st = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.ws = torch.empty(pkv.select_blocks_workspace_bytes(B, Hk, n * bs, bs), dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()

    def step(self, i, pause=lambda: None):
        self.sums.copy_(self.all_sums[i % 3])
        self.tables.copy_(self.all_tables[i])
        self.lens.copy_(self.all_lens[i])
        self.q.copy_(self.all_q[i])
        pause()
        pkv.select_blocks(self.sel, self.q, self.sums, self.tables, self.lens, bs, keep_last=2, workspace=self.ws,
                          device_status=self.st)
        pause()
        # what follows must not reach the call: a length of 0, a q of NaN
        self.q.fill_(float("nan"))
        self.lens.zero_()
        self.tables.zero_()
        pause()
        return self.sel.clone()


def test_queued_selections_equal_synchronised_ones():
    a, b = Steps(1), Steps(1)
    want = [a.step(i, torch.cuda.synchronize) for i in range(STEPS)]
    got = [b.step(i) for i in range(STEPS)]
    torch.cuda.synchronize()
    assert all(torch.equal(w, g) for w, g in zip(want, got))
    assert a.st.item() == 0 and b.st.item() == 0
    # and the synchronised ones are those of the definition
    s = a.all_sums[(STEPS - 1) % 3].double().cpu().numpy()
    ref = S.select_reference(a.all_q[-1].double().cpu().numpy(), s[:, :, 0], s[:, :, 1], a.all_tables[-1].cpu().numpy(),
                             a.all_lens[-1].cpu().numpy(), bs, K, 1, 2)
    np.testing.assert_array_equal(want[-1].cpu().numpy(), ref)


def test_two_streams_and_a_graph():
    a, b = Steps(2), Steps(3)
    want = [[x.step(i, torch.cuda.synchronize) for i in range(STEPS)] for x in (a, b)]
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for i in range(STEPS):
        for k, x in enumerate((a, b)):
            with torch.cuda.stream(streams[k]):
                got[k].append(x.step(i))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(w, g) for w, g in zip(want[k], got[k]))
    graphs = []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = [x.step(i) for i in range(3)]
        graphs.append((g, outs))
    for _ in range(4):
        for k in range(2):
            graphs[k][0].replay()
        torch.cuda.synchronize()
        for k in range(2):
            assert all(torch.equal(w, o) for w, o in zip(want[k][:3], graphs[k][1]))
