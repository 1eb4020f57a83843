"""Calls on a stream that is not the current one, without a workspace, while
the current stream still works on memory that it has given back."""
import numpy as np
import pytest
import torch

import paged_kv_cache_311_gb300 as pkv
from tests import q8_support as S
from tests.test_gpu_q8 import dev

pytestmark = pytest.mark.gpu
DEV = "cuda"


def calls():
    """(name, call(out, stream), out, bytes of its workspace)."""
    g = torch.Generator(device=DEV).manual_seed(5)
    r = lambda *s, t=torch.bfloat16: torch.randn(*s, generator=g, device=DEV).to(t)
    B, Hk, G, D, bs = 4, 8, 4, 128, 16
    tables, NB = S.make_tables(np.random.RandomState(1), [128] * B)
    bt, lens = dev(tables), dev(np.array([2048, 2040, 1, 777], np.int32))
    q, k, v = r(B, Hk * G, D), r(NB, Hk, bs, D), r(NB, Hk, bs, D)
    ks = pkv.q8_scales(NB, Hk, DEV).fill_(1.0)
    k8, v8 = k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn)
    yield ("decode", lambda o, s: pkv.paged_attention_decode(o, q, k, v, bt, lens, 0.1, max_context_len=2048, partition_size=128, stream=s), q,
           pkv.paged_attention_workspace_bytes(B, Hk * G, 2048, D, 128))
    yield ("q8", lambda o, s: pkv.paged_attention_decode_q8(o, q, k8, v8, ks, ks, bt, lens, 0.1, partition_size=128, stream=s), q,
           pkv.paged_attention_list_workspace_bytes(B, Hk * G, Hk, D, bs, 128, 128))
    sel = torch.arange(0, 128, 2, dtype=torch.int32, device=DEV).expand(2, Hk, 64).contiguous()
    yield ("selected", lambda o, s: pkv.paged_attention_decode_selected(o, q[:2], k, v, bt[:2], lens[:2], sel, 0.1,
                                                                     partition_size=32, stream=s), q[:2],
           pkv.paged_attention_list_workspace_bytes(2, Hk * G, Hk, D, bs, 64, 32))
    many, NB2 = S.make_tables(np.random.RandomState(2), [1100] * 32)
    q2, sums = r(32, 16, 64), torch.sort(r(NB2, 4, 2, 64), dim=2)[0].contiguous()
    lens2, bt2 = torch.full((32,), 8800, dtype=torch.int32, device=DEV), dev(many)
    yield ("select", lambda o, s: pkv.select_blocks(o, q2, sums, bt2, lens2, 8, stream=s),
           torch.zeros(32, 4, 20, dtype=torch.int32, device=DEV), pkv.select_blocks_workspace_bytes(32, 4, 8800, 8))
    htab, hlens = np.zeros((B, 128), np.int32), lens.cpu().numpy()
    htab[:] = tables
    htab[1, :64] = htab[0, :64]
    plan = pkv.plan_shared_prefix(htab, hlens, Hk * G, Hk, D, bs)
    on, dt = plan.to(DEV), dev(htab)
    yield ("shared", lambda o, s: pkv.paged_attention_decode_shared(o, q, k, v, dt, lens, 0.1, plan, on, max_context_len=2048, stream=s), q,
           max(plan.workspace_bytes, 16))


@pytest.mark.parametrize("raw", [False, True])
def test_memory_that_another_stream_gave_back_is_not_used(raw):
    side = torch.cuda.Stream()
    for name, call, like, nbytes in calls():
        assert nbytes > 0, name
        want, got = torch.zeros_like(like), torch.zeros_like(like)
        call(want, None)
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        # the current stream sleeps, then reads a block of the workspace's size that it has already freed
        block = torch.full((nbytes,), 7, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        torch.cuda._sleep(200_000_000)
        total = (block == 7).sum()
        del block
        call(got, side.cuda_stream if raw else side)
        torch.cuda.synchronize()
        assert int(total) == nbytes, name
        assert torch.equal(got, want), name


def test_the_default_stream_by_number_and_from_another_one():
    """stream=0 while another stream is current."""
    for name, call, like, nbytes in calls():
        want, got = torch.zeros_like(like), torch.zeros_like(like)
        call(want, None)
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.Stream()):
            call(got, 0)
        torch.cuda.synchronize()
        assert torch.equal(got, want), name


@pytest.mark.parametrize("raw", [False, True])
def test_a_captured_call_allocates_for_itself(raw):
    """No workspace, the capturing stream named: the graph keeps its own."""
    for name, call, like, nbytes in calls():
        want, got = torch.zeros_like(like), torch.zeros_like(like)
        call(want, None)
        torch.cuda.synchronize()
        graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=s):
            call(got, s.cuda_stream if raw else s)
        got.zero_()
        block = torch.full((nbytes,), 255, dtype=torch.uint8, device=DEV)   # not what the graph writes into
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and bool((block == 255).all()), name
