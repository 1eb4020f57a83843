"""The 4-bit cache's calls in streams and graphs: queued behind and before
other kernels without a synchronise, on two streams at once, in graphs that
share a workspace; what the binding refuses of GPU tensors."""
import numpy as np
import pytest
import torch

import paged_kv_cache_311_gb300 as pkv
from tests import q4_support as S
from tests.q8_support import make_tables
from tests.test_gpu_q4 import check, dev, run_decode

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, Hk, G, D, bs, STEPS = 6, 4, 4, 128, 16, 24


class Loop:
    """Decode steps over a 4-bit cache whose inputs torch kernels make just
    before each call and overwrite just after it."""

    def __init__(self, seed, seqs=B):
        g = torch.Generator(device=DEV).manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
        first = np.resize(np.array([700, 5, 64, 161, 32, 2999]), seqs)
        tables, NB = make_tables(np.random.RandomState(seed), [-(-(int(n) + STEPS) // bs) for n in first])
        self.bt, self.lens = dev(tables), dev(first.astype(np.int32))
        self.k, self.v = (pkv.q4_cache(NB, Hk, bs, D, DEV) for _ in "kv")
        seq = np.repeat(np.arange(seqs), first)
        pos = np.concatenate([np.arange(n) for n in first])
        slots = dev(tables[seq, pos // bs].astype(np.int64) * bs + pos % bs)
        key, value = r(len(pos), Hk, D).bfloat16(), r(len(pos), Hk, D).bfloat16()
        pkv.reshape_and_cache_q4(key, value, self.k, self.v, slots)
        self.new = r(STEPS, 3, seqs, Hk * G, D)
        self.q, self.nk, self.nv = (torch.zeros(seqs, h, D, dtype=torch.bfloat16, device=DEV) for h in (Hk * G, Hk, Hk))
        self.slots = torch.zeros(seqs, dtype=torch.int64, device=DEV)
        self.rk, self.rv = (torch.zeros(seqs, Hk, D, dtype=torch.bfloat16, device=DEV) for _ in "kv")
        self.out, self.cut = (torch.zeros(seqs, Hk * G, D, dtype=torch.float32, device=DEV) for _ in range(2))
        self.st = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()

    def step(self, i, pause, stream=None):
        pos = self.lens.long()
        self.slots.copy_(self.bt.long().gather(1, (pos // bs)[:, None])[:, 0] * bs + pos % bs)
        self.lens.add_(1)
        self.q.copy_(self.new[i, 0])
        self.nk.copy_(self.new[i, 1, :, :Hk])
        self.nv.copy_(self.new[i, 2, :, :Hk])
        a = dict(device_status=self.st, stream=stream)
        pkv.reshape_and_cache_q4(self.nk, self.nv, self.k, self.v, self.slots, **a)
        pause()
        self.nk.fill_(float("nan"))
        self.nv.fill_(float("nan"))
        pkv.gather_cache_q4(self.rk, self.rv, self.k, self.v, self.slots, **a)
        pause()
        # streamed (or a cluster), and in partitions through the workspace
        pkv.paged_attention_decode_q4(self.out, self.q, self.k, self.v, self.bt, self.lens, D ** -0.5, workspace=self.ws,
                                      max_context_len=8192 if self.bt.shape[1] * bs >= 8192 else None, **a)
        pause()
        pkv.paged_attention_decode_q4(self.cut, self.q, self.k, self.v, self.bt, self.lens, D ** -0.5,
                                      partition_size=64, workspace=self.ws, **a)
        pause()
        self.q.fill_(float("nan"))
        got = self.rk.clone(), self.rv.clone(), self.out.clone(), self.cut.clone()
        self.out.fill_(float("nan"))
        self.cut.fill_(float("nan"))
        return got

    def state(self):
        return [t.cpu() for t in (self.k, self.v)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("seqs", [B, 64])
def test_queued_steps_equal_synchronised_ones(seqs):
    slow, fast = Loop(1, seqs), Loop(1, seqs)
    want = [slow.step(i, torch.cuda.synchronize) for i in range(STEPS)]
    got = [fast.step(i, lambda: None) for i in range(STEPS)]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert same(w, g) and not any(torch.isnan(x).any() for x in g)
    assert same(slow.state(), fast.state()) and fast.st.item() == 0


def test_two_streams_at_once():
    want = [Loop(s, 48) for s in (2, 3)]
    ref = [[x.step(i, torch.cuda.synchronize) for i in range(STEPS)] for x in want]
    loops, streams = [Loop(s, 48) for s in (2, 3)], [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for i in range(STEPS):
        for n in range(2):
            with torch.cuda.stream(streams[n]):
                got[n].append(loops[n].step(i, lambda: None))
    torch.cuda.synchronize()
    for n in range(2):
        assert all(same(w, g) for w, g in zip(ref[n], got[n])) and same(want[n].state(), loops[n].state())


def test_a_stream_given_by_object_and_by_number():
    x = Loop(6, 48)
    want = x.step(0, torch.cuda.synchronize)[2]
    side = torch.cuda.Stream()
    q = x.new[0, 0].bfloat16()
    for stream in (side, side.cuda_stream):
        for ws in (x.ws, None):
            out = torch.full_like(x.out, float("nan"))
            side.wait_stream(torch.cuda.current_stream())
            pkv.paged_attention_decode_q4(out, q, x.k, x.v, x.bt, x.lens, D ** -0.5, workspace=ws, stream=stream)
            side.synchronize()
            assert torch.equal(out, want)


def test_graphs_that_share_a_workspace():
    """Captured decode calls with the same workspace, replayed in turn; a captured write and read of other rows between."""
    a, b = Loop(4, 48), Loop(5, 48)
    b.ws = a.ws
    qs = [torch.randn(48, Hk * G, D, device=DEV).bfloat16() for _ in range(2)]
    want, graphs = [], []
    for x, q in zip((a, b), qs):
        call = lambda x=x, q=q: pkv.paged_attention_decode_q4(x.out, q, x.k, x.v, x.bt, x.lens, D ** -0.5, workspace=x.ws)  # noqa: E731
        call()
        torch.cuda.synchronize()
        want.append(x.out.clone())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append(graph)
    key = torch.randn(48, Hk, D, device=DEV).bfloat16()
    back = [torch.zeros_like(key) for _ in "kv"]
    # slots behind every sequence's last token: rows that no decode call reads
    pos = a.lens.long() + 1
    slots = a.bt.long().gather(1, (pos // bs)[:, None])[:, 0] * bs + pos % bs
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.reshape_and_cache_q4(key, key, a.k, a.v, slots)
        pkv.gather_cache_q4(*back, a.k, a.v, slots)
    for i in range(5):
        key.normal_()
        a.out.zero_()
        b.out.zero_()
        graphs[0].replay()
        graph.replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])
        u = S.quantize(key.double().cpu().numpy(), torch.bfloat16)
        assert torch.equal(back[0].cpu(), torch.from_numpy(S.numbers(*u)).bfloat16()) and torch.equal(back[0], back[1])


def test_workspace_is_what_the_call_needs():
    """The size that is asked for is enough, one byte less is refused, and nothing behind it is written."""
    c = S.q4_case(3, t="bf16", G=4, Hk=2, lens=(3000, 100) * 40)
    for P in (0, 256):
        need = pkv.paged_attention_q4_workspace_bytes(c["B"], 8, 2, 128, 16, 3000, P)
        assert need > 0
        ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
        got, st = run_decode(c, P, max_len=3000, workspace=ws[:need])
        assert st == 0 and bool((ws[need:] == 0x5A).all())
        check(c, got)
        with pytest.raises(pkv.PkvError) as e:
            run_decode(c, P, max_len=3000, workspace=ws[: need - 1])
        assert e.value.status == -4
    assert pkv.paged_attention_q4_workspace_bytes(1, 32, 8, 128, 16, 700) == 0


def test_empty_calls():
    k = pkv.q4_cache(2, 2, 16, 128, DEV)
    none = torch.empty(0, 2, 128, dtype=torch.float16, device=DEV)
    at = torch.empty(0, dtype=torch.int64, device=DEV)
    pkv.reshape_and_cache_q4(none, none, k, k, at)
    pkv.gather_cache_q4(none, none, k, k, at)
    q = torch.empty(0, 4, 128, dtype=torch.float16, device=DEV)
    pkv.paged_attention_decode_q4(q, q, k, k, torch.empty(0, 4, dtype=torch.int32, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV), 1.0)
    assert not k.any()


@pytest.mark.parametrize("lens", [(0,), (0, 0, 0), (0,) * 300])
def test_no_tokens_at_all(lens):
    c = S.q4_case(4, t="f16", G=3, Hk=2, lens=lens)
    for P, most in ((0, None), (0, 0), (0, 16), (32, 16)):
        got, st = run_decode(c, P, max_len=most)
        assert st == 0 and (got == 0).all()


def test_binding_refuses():
    x = torch.zeros(3, 2, 128, dtype=torch.float16, device=DEV)
    k, at = pkv.q4_cache(4, 2, 16, 128, DEV), torch.zeros(3, dtype=torch.int64, device=DEV)
    write = lambda *a: pkv.reshape_and_cache_q4(*a)  # noqa: E731
    read = lambda *a, **kw: pkv.gather_cache_q4(*a, **kw)  # noqa: E731
    for f in (write, read):
        for bad, text in (((x.float()[..., :64].half(), x, k, k, at), "mismatch|three dimensions"), ((x, x.bfloat16(), k, k, at), "dtype"),
                          ((x, x, k.to(torch.int8), k, at), "uint8"), ((x, x, k[..., :64].contiguous(), k, at), "D / 2"),
                          ((x, x, k, k[:3], at), "D / 2"), ((x, x, k, k, at.int()), "int64"), ((x, x, k, k, at[:2]), "int64"),
                          ((x.transpose(1, 2), x, k, k, at), "three dimensions"), ((x, x, k.cpu(), k, at), "CUDA"),
                          ((x, x[:, :1], k, k, at), "mismatch")):
            with pytest.raises(ValueError, match=text):
                f(*bad)
    with pytest.raises(TypeError):
        write(x, x, k, None, at)
    with pytest.raises(pkv.PkvError):                       # rows of tokens that overlap
        write(x[:1].expand(3, 2, 128), x, k, k, at)
    with pytest.raises(pkv.PkvError):                       # rows that are not 16-byte pieces apart
        write(torch.zeros(3 * 257, dtype=torch.float16, device=DEV).as_strided((3, 2, 128), (257, 128, 1)), x, k, k, at)
    with pytest.raises(pkv.PkvError):                       # float32 numbers of a cache whose type is not said
        read(x.float(), x.float(), k, k, at)
    with pytest.raises(pkv.PkvError):
        read(x, x, k, k, at, dtype=torch.bfloat16)
    q, out = torch.zeros(3, 4, 128, dtype=torch.float16, device=DEV), torch.zeros(3, 4, 128, device=DEV)
    bt, cl = torch.zeros(3, 2, dtype=torch.int32, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    good = [out, q, k, k, bt, cl, 1.0]
    pkv.paged_attention_decode_q4(*good)
    for i, bad in ((0, out[:2]), (0, out.int()), (1, q.int()), (2, k.int()), (3, k[..., :40].contiguous()), (4, bt.long()), (4, bt[:2]), (5, cl.long()),
                   (5, cl[:1]), (0, out.transpose(0, 1))):
        with pytest.raises(ValueError):
            pkv.paged_attention_decode_q4(*good[:i], bad, *good[i + 1:])
    with pytest.raises(pkv.PkvError):
        pkv.paged_attention_decode_q4(out, q.float(), k, k, bt, cl, 1.0)
    with pytest.raises(pkv.PkvError):
        pkv.paged_attention_decode_q4(*good, max_context_len=33)
    with pytest.raises(pkv.PkvError):
        pkv.paged_attention_decode_q4(*good, partition_size=48)
