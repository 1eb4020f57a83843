"""The 8-bit cache on the GPU: the append call bit for bit against its
definition, decode attention over the cache within its derived tolerance."""
import numpy as np
import pytest
import torch

import paged_kv_cache_311_gb300 as pkv
from tests import q8_support as S

pytestmark = pytest.mark.gpu
DEV = "cuda"


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to(DEV)


class Pool:
    """An 8-bit cache on the GPU and its 64-bit twin."""

    def __init__(self, NB, Hk, bs, D, fill=0xFF):
        self.k = torch.full((NB, Hk, bs, D), fill, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
        self.v = torch.full((NB, Hk, bs, D), fill, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
        self.ks, self.vs = (pkv.q8_scales(NB, Hk, DEV).fill_(float("nan")) for _ in "kv")
        self.rk, self.rv = S.Q8Cache(NB, Hk, bs, D), S.Q8Cache(NB, Hk, bs, D)
        self.written = np.zeros((NB, bs), bool)
        self.Hk, self.bs, self.D, self.NB = Hk, bs, D, NB
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def append(self, key, value, tables, total, starts, decode_step=False, reference=True):
        """key, value [T, Hk, D] torch tensors (CPU)."""
        pkv.append_cache_q8(key.to(DEV), value.to(DEV), self.k, self.v, self.ks, self.vs, dev(tables),
                            dev(np.asarray(total, np.int32)), None if decode_step else dev(np.asarray(starts, np.int32)),
                            device_status=self.status)
        if reference:
            S.append_reference(self.rk, key.double().numpy(), tables, total, starts)
            S.append_reference(self.rv, value.double().numpy(), tables, total, starts)
            for s in range(len(total)):
                for j, a, b, _ in S.touched(int(total[s]), int(starts[s + 1] - starts[s]), self.bs):
                    self.written[tables[s, j], a:b] = True

    def check(self):
        for t, sc, r in ((self.k, self.ks, self.rk), (self.v, self.vs, self.rv)):
            bits = t.view(torch.uint8).cpu().numpy()
            hit = self.written.any(1)
            scale = sc.cpu().numpy()
            np.testing.assert_array_equal(scale[hit][:, : self.Hk].astype(np.float64), r.s[hit])
            assert np.isnan(scale[~hit]).all() and np.isnan(scale[:, self.Hk:]).all()
            rows = np.broadcast_to(self.written[:, None, :, None], bits.shape)
            np.testing.assert_array_equal(S.decode(bits)[rows], r.v[rows])
            assert (bits[~rows] == 0xFF).all()          # rows that nothing wrote keep their bytes


def rows(rng, T, Hk, D, t, size=1.0):
    return torch.from_numpy(rng.randn(T, Hk, D) * size).to(S.DT[t])


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("Hk", [1, 3, 8])
def test_append_prompts_and_steps(t, D, bs, Hk):
    """Prompts of ragged lengths (one of them empty), then several calls of one
    or a few tokens whose sizes grow and shrink, so that scales grow over held
    rows, blocks fill up in the middle of a call and new ones open."""
    rng = np.random.RandomState(D + bs + Hk)
    first = [1, bs - 1, 0, bs, bs + 1, 3 * bs + 2]
    most = [n + 3 * bs for n in first]
    tables, NB = S.make_tables(rng, [-(-n // bs) for n in most])
    pool = Pool(NB, Hk, bs, D)
    total = np.array(first)
    starts = np.concatenate([[0], np.cumsum(first)])
    pool.append(rows(rng, starts[-1], Hk, D, t), rows(rng, starts[-1], Hk, D, t), tables, total, starts)
    assert pool.status.item() == 0
    pool.check()
    for step, size in enumerate((1.0, 40.0, 0.01, 300.0, 3.0, 6.0)):
        new = rng.randint(0, bs // 2, len(first)) if step % 2 else np.ones(len(first), int)
        total = total + new
        starts = np.concatenate([[0], np.cumsum(new)])
        pool.append(rows(rng, starts[-1], Hk, D, t, size), rows(rng, starts[-1], Hk, D, t, 1 / size), tables, total,
                    starts, decode_step=step % 2 == 0)
        assert pool.status.item() == 0
        pool.check()


@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_append_borders_of_the_scale(t):
    """Magnitudes at, just under and just over 448 2^e, the smallest and the
    largest of the type, zeros only; and values on e4m3's rounding borders."""
    dt = S.DT[t]
    info = torch.finfo(dt)
    step = float(info.eps)
    amax = [448.0, 448.0 * (1 + step), 448.0 * (1 - step / 2), 256.0, 0.0, float(info.max), float(info.tiny), float(info.tiny) * step,
            1.75, 1.75 * (1 + step), 1.0, 0.875]
    Hk, D, bs = len(amax), 64, 8
    x = torch.zeros(1, Hk, D, dtype=torch.float64)
    grid = torch.tensor([0.0, 1 / 1024, 1 / 512, 3 / 1024, 17 / 448, 1.0625 / 448, 1.1875 / 448, -0.5, -13.5 / 448, 1.0])
    for h, a in enumerate(amax):
        x[0, h, : len(grid)] = grid * a
        x[0, h, -1] = -a
    pool = Pool(2, Hk, bs, D)
    pool.append(x.to(dt), x.to(dt).flip(1), np.array([[1]], np.int32), np.array([1]), np.array([0, 1]))
    assert pool.status.item() == 0
    pool.check()
    # the largest after the smallest: held rows underflow
    pool.append(x.to(dt).flip(1), x.to(dt), np.array([[1]], np.int32), np.array([2]), np.array([0, 1]))
    pool.check()


def test_append_nan_and_infinity():
    rng = np.random.RandomState(0)
    Hk, D, bs = 4, 128, 16
    key, value = rows(rng, 5, Hk, D, "bf16"), rows(rng, 5, Hk, D, "bf16")
    key[1, 0, 3], key[2, 1, 7], key[4, 1, 9], key[:, 2] = float("nan"), float("inf"), float("-inf"), float("inf")
    value[0, 3, 0], value[3, 3, 100] = float("-inf"), float("nan")
    pool = Pool(3, Hk, bs, D)
    pool.append(key, value, np.array([[2]], np.int32), np.array([5]), np.array([0, 5]))
    pool.check()
    pool.append(rows(rng, 1, Hk, D, "bf16", 50.0), rows(rng, 1, Hk, D, "bf16", 50.0), np.array([[2]], np.int32),
                np.array([6]), np.array([0, 1]), decode_step=True)
    pool.check()   # NaN rows stay NaN when their block is rescaled


def test_append_many_sequences_and_padding():
    """1500 sequences, many of them without new tokens, found by their starts;
    padding tokens before the first and behind the last sequence."""
    rng = np.random.RandomState(5)
    B, Hk, D, bs = 1500, 2, 64, 8
    new = np.where(rng.rand(B) < 0.6, 0, rng.randint(1, 20, B))
    total = new + rng.randint(0, 1, B)
    tables, NB = S.make_tables(rng, [-(-int(n) // bs) for n in total])
    lead, tail = 3, 7
    starts = lead + np.concatenate([[0], np.cumsum(new)])
    T = int(starts[-1]) + tail
    pool = Pool(NB, Hk, bs, D)
    pool.append(rows(rng, T, Hk, D, "f16"), rows(rng, T, Hk, D, "f16"), tables, total, starts)
    assert pool.status.item() == 0
    pool.check()
    # a decode step over a padded batch: lengths 0 are padding
    total2 = np.where(total > 0, total, 0)
    pool2 = Pool(NB, Hk, bs, D)
    new2 = (total2 > 0).astype(int)
    key, value = rows(rng, B, Hk, D, "f16"), rows(rng, B, Hk, D, "f16")
    pool2.append(key, value, tables, total2, np.arange(B + 1), decode_step=True, reference=False)
    for s in np.nonzero(new2)[0]:
        j, a, b, _ = S.touched(int(total2[s]), 1, bs)[0]
        if a == 0:
            pool2.rk.append(key[s:s + 1].double().numpy(), tables[s, j], 0)
            np.testing.assert_array_equal(pool2.ks[tables[s, j], :Hk].cpu().double().numpy(), pool2.rk.s[tables[s, j]])
            assert S.same_values(pool2.k.view(torch.uint8)[tables[s, j], :, 0].cpu().numpy(), pool2.rk.v[tables[s, j], :, 0])
    assert pool2.status.item() == 0


@pytest.mark.parametrize("what", ["short", "long", "negative", "starts", "starts_end", "block", "block_negative"])
def test_append_refuses_bad_data(what):
    """The sequence with bad data is skipped and reported, the others written."""
    rng = np.random.RandomState(1)
    Hk, D, bs = 2, 64, 8
    tables = np.array([[0, 1], [2, 3], [4, 5]], np.int32)
    total, starts = np.array([10, 9, 16], np.int32), np.array([0, 10, 12, 14], np.int32)
    bad_seq, bit = 1, pkv.DEV_BAD_CONTEXT_LEN
    pool = Pool(6, Hk, bs, D)
    key, value = rows(rng, 14, Hk, D, "f16"), rows(rng, 14, Hk, D, "f16")
    if what == "short":
        total[1] = 1
    elif what == "long":
        total[1] = 17
    elif what == "negative":
        total[1] = -3
    elif what == "starts":
        starts[2] = 9           # sequence 1 ends before it starts: its tokens are nobody's
        bit = None
    elif what == "starts_end":
        bad_seq, starts[3] = 2, 15
    else:
        tables[1, 1] = 6 if what == "block" else -1
        bit = pkv.DEV_BAD_BLOCK
    pool.append(key, value, tables, total, starts, reference=False)
    torch.cuda.synchronize()
    if bit is not None:
        assert pool.status.item() == bit
    good, gs = [s for s in range(3) if s != bad_seq], starts.copy()
    if what == "starts":
        good = [0]
    for s in good:
        for cache, x in ((pool.rk, key), (pool.rv, value)):
            for j, a, b, t in S.touched(int(total[s]), int(gs[s + 1] - gs[s]), bs):
                if a == 0:
                    cache.append(x[gs[s] + t: gs[s] + t + b - a].double().numpy(), tables[s, j], a)
                    got = pool.k if cache is pool.rk else pool.v
                    assert S.same_values(got.view(torch.uint8)[tables[s, j], :, :b].cpu().numpy(), cache.v[tables[s, j], :, :b])


def test_copy_and_swap_move_an_8_bit_cache():
    """Blocks and scales go through copy_blocks and swap_blocks as they are."""
    rng = np.random.RandomState(2)
    Hk, D, bs = 5, 64, 8
    pool = Pool(6, Hk, bs, D)
    pool.append(rows(rng, 12, Hk, D, "f16"), rows(rng, 12, Hk, D, "f16"), np.array([[3, 1]], np.int32), np.array([12]), np.array([0, 12]))
    pairs = dev(np.array([[3, 0], [1, 5]], np.int64))
    pkv.copy_blocks([pool.k], [pool.v], pairs, device_status=pool.status)
    pkv.copy_blocks([pool.ks], [pool.vs], pairs, device_status=pool.status)
    out = [torch.zeros(2, *t.shape[1:], dtype=t.dtype).pin_memory() for t in (pool.k, pool.v, pool.ks, pool.vs)]
    swap = dev(np.array([[0, 1], [5, 0]], np.int64))
    pkv.swap_blocks([pool.k], [pool.v], out[:1], out[1:2], swap, pkv.SWAP_OUT, device_status=pool.status)
    pkv.swap_blocks([pool.ks], [pool.vs], out[2:3], out[3:], swap, pkv.SWAP_OUT, device_status=pool.status)
    torch.cuda.synchronize()
    assert pool.status.item() == 0
    raw = lambda t: t.view(torch.uint8).cpu()
    for a, b, h in ((3, 0, 1), (1, 5, 0)):
        for t, o in zip((pool.k, pool.v, pool.ks, pool.vs), out):
            assert torch.equal(raw(t[a]), raw(t[b])) and torch.equal(raw(t[a]), raw(o[h]))


# ------------------------------------------------------------------ decode


def run_decode(c, P=0, out_dtype=torch.float32, max_len=None, stream=None):
    f8 = lambda b: dev(b).view(torch.float8_e4m3fn)
    out = torch.full(tuple(c["q"].shape), float("nan"), dtype=out_dtype, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.paged_attention_decode_q8(out, c["q"].to(DEV), f8(c["k_bits"]), f8(c["v_bits"]), dev(c["k_scale"]), dev(c["v_scale"]),
                                  dev(c["tables"]), dev(c["lens"]), c["scale"], max_context_len=max_len, partition_size=P,
                                  device_status=st, stream=stream)
    torch.cuda.synchronize()
    return out.double().cpu().numpy(), int(st.item())


def reference(c, listed=None):
    k = S.decode(c["k_bits"]) * c["k_scale"][:, : c["Hk"], None, None].astype(np.float64)
    v = S.decode(c["v_bits"]) * c["v_scale"][:, : c["Hk"], None, None].astype(np.float64)
    ref, bound = S.attention_reference(c["q"].double().numpy(), k, v, c["tables"], c["lens"], c["bs"], c["scale"], listed)
    return ref, bound, v


def check(c, got, out_dtype, listed=None):
    ref, bound, v = reference(c, listed)
    tol = S.attention_tolerance(ref, bound, v, c["lens"], c["D"], out_dtype)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (np.abs(got - ref)[bad][:5], tol[bad][:5], np.argwhere(bad)[:5])


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("G", [1, 2, 3, 5, 8])
def test_decode_matrix(t, D, bs, G):
    lens = (1, bs - 1, bs, bs + 1, 3 * bs + 5, 0, 64, 100, 511, 513, 1100)
    c = S.q8_case(D + bs + G, qdtype=t, G=G, Hk=2 if G < 8 else 3, D=D, bs=bs, lens=lens)
    for P in (0, 32, 2048):
        for od in (torch.float32, S.DT[t]):
            got, st = run_decode(c, P, od)
            assert st == 0
            assert not got[5].any()
            check(c, got, od)


@pytest.mark.parametrize("bs", [8, 16, 32])
def test_decode_scales_far_apart(bs):
    """Neighbouring blocks whose scales differ by up to 2^40, for K (some
    blocks' scores then vanish or rule) and for V."""
    c = S.q8_case(7, G=4, Hk=2, bs=bs, lens=(700, 33, 260), spread=20.0)
    for P in (0, 64):
        got, st = run_decode(c, P)
        assert st == 0
        check(c, got, torch.float32)


def test_decode_long_and_strong():
    """A long context whose scores climb along it (each partition and tile
    raises the maximum) beside short ones."""
    c = S.q8_case(3, G=8, Hk=1, lens=(20000, 5, 9000), bs=16)
    c["q"] = c["q"].abs() * 2
    c["scale"] = 0.5
    nblk = -(-20000 // 16)
    c["k_scale"][c["tables"][0, :nblk], 0] = (2.0 ** np.floor(np.linspace(-12, -6, nblk))).astype(np.float32)
    c["k_bits"] = np.where(c["k_bits"] == 0x7F, c["k_bits"], np.where(c["k_bits"] == 0xFF, 0xFF, c["k_bits"] & 0x7F)).astype(np.uint8)
    for P in (0, 64, 1024):
        got, st = run_decode(c, P)
        assert st == 0
        check(c, got, torch.float32)


def test_decode_placement_and_repeats_are_bit_equal():
    c = S.q8_case(11, G=4, Hk=2, lens=(70, 513, 1200), garbage=False)
    base, _ = run_decode(c)
    again, _ = run_decode(c)
    np.testing.assert_array_equal(base, again)
    perm = np.random.RandomState(0).permutation(c["NB"])
    d = dict(c)
    inv = np.argsort(perm)
    for n in ("k_bits", "v_bits", "k_scale", "v_scale"):
        d[n] = c[n][perm]
    d["tables"] = np.where(c["tables"] >= 0, inv[np.maximum(c["tables"], 0)], -1).astype(np.int32)
    moved, _ = run_decode(d)
    np.testing.assert_array_equal(base, moved)


@pytest.mark.parametrize("P", [0, 32])
def test_decode_refuses_bad_rows(P):
    c = S.q8_case(13, G=2, Hk=2, lens=(100, 100, 100, 100))
    good, _ = run_decode(c, P)
    d = dict(c, tables=c["tables"].copy(), lens=c["lens"].copy())
    d["tables"][1, 3] = c["NB"]
    d["lens"][2] = -1
    got, st = run_decode(d, P, max_len=100)
    assert st == pkv.DEV_BAD_BLOCK | pkv.DEV_BAD_CONTEXT_LEN
    assert not got[1].any() and not got[2].any()
    np.testing.assert_array_equal(got[[0, 3]], good[[0, 3]])
    d["lens"][2] = 101
    got, st = run_decode(d, P, max_len=100)
    assert st == pkv.DEV_BAD_BLOCK | pkv.DEV_BAD_CONTEXT_LEN and not got[2].any()


def test_decode_nan_reaches_the_output_of_its_head_only():
    c = S.q8_case(17, G=2, Hk=2, lens=(50, 50))
    for n, s, h, tok in (("k_bits", 0, 0, 49), ("v_bits", 1, 1, 0)):
        c[n] = c[n].copy()
        c[n][c["tables"][s, tok // 16], h, tok % 16, 5] = 0x7F
    for P in (0, 32):
        got, st = run_decode(c, P)
        assert st == 0
        nan = np.isnan(got)
        assert nan[0, :2].all() and not nan[0, 2:].any()
        assert nan[1, 2:, 5].all() and nan.sum() == 2 * 128 + 2


def test_decode_beyond_32_bit_offsets():
    """Blocks whose byte offsets in the cache pass 2^32."""
    Hk, bs, D = 8, 16, 128
    NB = (1 << 32) // (Hk * bs * D) + 300
    c = S.q8_case(19, G=4, Hk=Hk, D=D, bs=bs, lens=(200, 77))
    f8 = torch.zeros(NB, Hk, bs, D, dtype=torch.uint8, device=DEV)
    v8 = torch.zeros_like(f8)
    ks, vs = pkv.q8_scales(NB, Hk, DEV), pkv.q8_scales(NB, Hk, DEV)
    off = NB - c["NB"]
    for t, n in ((f8, "k_bits"), (v8, "v_bits"), (ks, "k_scale"), (vs, "v_scale")):
        t[off:] = dev(c[n])
    tables = np.where(c["tables"] >= 0, c["tables"] + off, -1).astype(np.int32)
    out = torch.empty(2, 4 * Hk, D, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.paged_attention_decode_q8(out, c["q"].to(DEV), f8.view(torch.float8_e4m3fn), v8.view(torch.float8_e4m3fn), ks, vs,
                                  dev(tables), dev(c["lens"]), c["scale"], device_status=st)
    assert st.item() == 0
    check(c, out.double().cpu().numpy(), torch.float32)


def test_decode_on_another_stream():
    """The workspace that the call allocates belongs to the stream it runs on."""
    c = S.q8_case(23, G=4, Hk=2, lens=(3000, 1))
    base, _ = run_decode(c, 64)
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        s.wait_stream(torch.cuda.current_stream())
        got, st = run_decode(c, 64, stream=stream)
        assert st == 0
        np.testing.assert_array_equal(base, got)
