"""The 8-bit cache's and the selection's calls in streams and graphs: queued
behind and before other kernels without a synchronise, on two streams at
once, and in graphs that share a workspace."""
import numpy as np
import pytest
import torch

import paged_kv_cache_311_gb300 as pkv
from tests import q8_support as S
from tests.test_gpu_q8 import dev

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, Hk, G, D, bs, K, STEPS = 6, 4, 4, 128, 16, 12, 24


class Loop:
    """Decode steps over an 8-bit cache whose inputs torch kernels make just
    before each call and overwrite just after it."""

    def __init__(self, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device=DEV)
        first = np.array([700, 5, 64, 161, 32, 1999])
        tables, NB = S.make_tables(np.random.RandomState(seed), [-(-(int(n) + STEPS) // bs) for n in first])
        self.bt, self.lens = dev(tables), dev(first.astype(np.int32))
        self.k, self.v = (torch.zeros(NB, Hk, bs, D, dtype=torch.float8_e4m3fn, device=DEV) for _ in "kv")
        self.ks, self.vs = pkv.q8_scales(NB, Hk, DEV), pkv.q8_scales(NB, Hk, DEV)
        self.sums = torch.zeros(NB, Hk, 2, D, dtype=torch.bfloat16, device=DEV)
        starts = dev(np.concatenate([[0], np.cumsum(first)]).astype(np.int32))
        n = int(first.sum())
        key, value = r(n, Hk, D).bfloat16(), r(n, Hk, D).bfloat16()
        pkv.append_cache_q8(key, value, self.k, self.v, self.ks, self.vs, self.bt, self.lens, starts)
        pkv.summarize_blocks(self.k, self.sums, self.bt, self.lens, starts, num_tokens=n, k_scales=self.ks)
        self.new = r(STEPS, 3, B, Hk * G, D)
        self.q, self.nk, self.nv = (torch.zeros(B, h, D, dtype=torch.bfloat16, device=DEV) for h in (Hk * G, Hk, Hk))
        self.sel = torch.zeros(B, Hk, K, dtype=torch.int32, device=DEV)
        self.out, self.all = (torch.zeros(B, Hk * G, D, dtype=torch.float32, device=DEV) for _ in range(2))
        self.st = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()

    def step(self, i, pause, stream=None):
        self.lens.add_(1)
        size = 3.0 if i % 7 == 3 else 1.0
        self.q.copy_(self.new[i, 0])
        self.nk.copy_(self.new[i, 1, :, :Hk] * size)
        self.nv.copy_(self.new[i, 2, :, :Hk] * size)
        a = dict(device_status=self.st, stream=stream)
        pkv.append_cache_q8(self.nk, self.nv, self.k, self.v, self.ks, self.vs, self.bt, self.lens, **a)
        pause()
        self.nk.fill_(float("nan"))
        self.nv.fill_(float("nan"))
        pkv.summarize_blocks(self.k, self.sums, self.bt, self.lens, k_scales=self.ks, **a)
        pause()
        pkv.select_blocks(self.sel, self.q, self.sums, self.bt, self.lens, bs, keep_last=2, **a)
        pause()
        pkv.paged_attention_decode_selected(self.out, self.q, self.k, self.v, self.bt, self.lens, self.sel, D ** -0.5,
                                            k_scales=self.ks, v_scales=self.vs, **a)
        pause()
        # the whole context too, through the workspace
        pkv.paged_attention_decode_q8(self.all, self.q, self.k, self.v, self.ks, self.vs, self.bt, self.lens, D ** -0.5,
                                      partition_size=64, workspace=self.ws, **a)
        pause()
        self.q.fill_(float("nan"))
        return self.sel.clone(), self.out.clone(), self.all.clone()

    def state(self):
        return [t.view(torch.uint8).cpu() for t in (self.k, self.v, self.ks, self.vs, self.sums)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_queued_steps_equal_synchronised_ones():
    slow, fast = Loop(1), Loop(1)
    want = [slow.step(i, torch.cuda.synchronize) for i in range(STEPS)]
    got = [fast.step(i, lambda: None) for i in range(STEPS)]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert same(w, g) and not torch.isnan(g[1]).any() and not torch.isnan(g[2]).any()
    assert same(slow.state(), fast.state()) and fast.st.item() == 0


def test_two_streams_at_once():
    want = [Loop(s) for s in (2, 3)]
    ref = [[x.step(i, torch.cuda.synchronize) for i in range(STEPS)] for x in want]
    loops, streams = [Loop(s) for s in (2, 3)], [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for i in range(STEPS):
        for n in range(2):
            with torch.cuda.stream(streams[n]):
                got[n].append(loops[n].step(i, lambda: None))
    torch.cuda.synchronize()
    for n in range(2):
        assert all(same(w, g) for w, g in zip(ref[n], got[n])) and same(want[n].state(), loops[n].state())


def test_graphs_that_share_a_workspace():
    """Two captured decode calls with the same workspace, replayed in turn."""
    a, b = Loop(4), Loop(5)
    b.ws = a.ws
    qs = [torch.randn(B, Hk * G, D, device=DEV).bfloat16() for _ in range(2)]
    want, graphs = [], []
    for x, q in zip((a, b), qs):
        call = lambda x=x, q=q: pkv.paged_attention_decode_q8(x.all, q, x.k, x.v, x.ks, x.vs, x.bt, x.lens, D ** -0.5,
                                                               partition_size=64, workspace=x.ws)
        call()
        torch.cuda.synchronize()
        want.append(x.all.clone())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append(graph)
    for _ in range(5):
        a.all.zero_()
        b.all.zero_()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(a.all, want[0]) and torch.equal(b.all, want[1])
