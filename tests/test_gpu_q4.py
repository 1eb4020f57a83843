"""The 4-bit cache on the GPU: writing and reading back bit for bit against
their definitions, decode attention over the cache within its derived
tolerance."""
import numpy as np
import pytest
import torch

import paged_kv_cache_311_gb300 as pkv
from tests import q4_support as S
from tests.q8_support import DT, make_tables

pytestmark = pytest.mark.gpu
DEV = "cuda"
FILL = 0xA5


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to(DEV)


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def cache(NB, Hk, bs, D):
    return pkv.q4_cache(NB, Hk, bs, D, DEV).fill_(FILL)


def check_written(rec, x, slots, t, NB, bs):
    """Records on the GPU after rows x [T, Hk, D] (CPU tensor) went to `slots`: codes and pairs of those
    rows are the definition's, every other byte is as it was."""
    T, Hk, D = x.shape
    got = rec.cpu().numpy()
    u, s, m = S.unpack(got, t, D)
    hit = np.zeros((NB, bs), bool)
    wu, ws, wm = S.quantize(x.double().numpy(), t)
    for i, slot in enumerate(slots):
        if 0 <= slot < NB * bs:
            b, r = slot // bs, slot % bs
            hit[b, r] = True
            np.testing.assert_array_equal(s[b, :, r], ws[i])
            np.testing.assert_array_equal(m[b, :, r], wm[i])
            ok = ~np.isnan(ws[i])
            np.testing.assert_array_equal(u[b, :, r][ok], wu[i][ok])
    byte, _ = S.places(bs, D)
    flat = got.reshape(NB, Hk, -1)
    for r in range(bs):
        rest = flat[~hit[:, r]]
        assert (rest[..., byte[r]] == FILL).all()
        for j in range(D // 64):
            at = S.pair_place(r, j, D, bs)
            assert (rest[..., at: at + 4] == FILL).all()


def rows(rng, T, Hk, D, t, size=1.0):
    return torch.from_numpy(rng.randn(T, Hk, D) * size + 0.3 * size * rng.randn(T, Hk, 1)).to(DT[t])


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("Hk", [1, 3, 8])
@pytest.mark.parametrize("T", [1, 37])
def test_write_and_read(t, D, bs, Hk, T):
    """Rows of many sizes to slots in any order, some of them padding; the numbers read back are s u + m rounded once."""
    rng = np.random.RandomState(D + bs + Hk + T)
    NB = 11
    slots = rng.permutation(NB * bs)[:T]
    if T > 1:
        slots[rng.rand(T) < 0.2] = -1
    key, value = rows(rng, T, Hk, D, t), rows(rng, T, Hk, D, t, 40.0)
    key[T // 2] *= 2.0 ** -12
    k, v, st = cache(NB, Hk, bs, D), cache(NB, Hk, bs, D), status()
    pkv.reshape_and_cache_q4(key.to(DEV), value.to(DEV), k, v, dev(slots), device_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    for rec, x in ((k, key), (v, value)):
        check_written(rec, x, slots, DT[t], NB, bs)
    for out_t in (DT[t], torch.float32):
        out = [torch.full((T, Hk, D), 7.0, dtype=out_t, device=DEV) for _ in "kv"]
        pkv.gather_cache_q4(out[0], out[1], k, v, dev(slots), dtype=DT[t] if out_t == torch.float32 else None, device_status=st)
        for o, x in zip(out, (key, value)):
            want = torch.from_numpy(S.numbers(*S.quantize(x.double().numpy(), DT[t]))).to(out_t)
            want[torch.from_numpy(slots < 0)] = 7.0
            assert torch.equal(o.cpu(), want)
    assert st.item() == 0


@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_write_borders(t):
    """Groups of one value, of two, quotients halfway between codes, the type's largest and smallest, ranges of which
    1/15 is not a normal number, zeros of both signs, NaN and infinities."""
    dt = DT[t]
    info = torch.finfo(dt)
    big, tiny, sub = float(info.max), float(info.tiny), float(info.tiny) * float(info.eps)
    rng = np.random.RandomState(1)
    g = [np.full(64, 3.25), np.full(64, -0.0), np.zeros(64), np.where(np.arange(64) % 2, 0.0, -0.0),
         np.arange(64) % 16, np.arange(64) % 31 / 2.0, -(np.arange(64) % 31) / 2.0, 1000.0 + np.arange(64) % 31 / 2.0,
         np.where(np.arange(64) == 5, big, -big), np.where(np.arange(64) == 5, big, 0.0), big * (np.arange(64) - 31.5) / 32,
         np.where(np.arange(64) == 7, tiny, 0.0), sub * (np.arange(64) % 3), sub * (np.arange(64) % 22), sub * (np.arange(64) % 7) - 3 * sub,
         1.0 + sub * np.arange(64), np.where(np.arange(64) == 0, 1.0, 1e-6 * rng.randn(64)),
         np.where(np.arange(64) == 9, np.nan, rng.randn(64)), np.where(np.arange(64) == 9, np.inf, rng.randn(64)),
         np.where(np.arange(64) == 9, -np.inf, rng.randn(64)), np.full(64, np.inf), np.full(64, np.nan)]
    if len(g) % 2:
        g.append(rng.randn(64))
    x = torch.from_numpy(np.stack(g)).to(dt)                # [groups, 64]
    for D in (64, 128):
        key = x.reshape(1, -1, D)
        Hk, bs = key.shape[1], 8
        value = key.flip(1).contiguous()
        k, v, st = cache(2, Hk, bs, D), cache(2, Hk, bs, D), status()
        pkv.reshape_and_cache_q4(key.to(DEV), value.to(DEV), k, v, dev(np.array([11])), device_status=st)
        check_written(k, key, [11], dt, 2, bs)
        check_written(v, value, [11], dt, 2, bs)
        out = [torch.zeros(1, Hk, D, dtype=dt, device=DEV) for _ in "kv"]
        pkv.gather_cache_q4(*out, k, v, dev(np.array([11])))
        for o, y in zip(out, (key, value)):
            want = torch.from_numpy(S.numbers(*S.quantize(y.double().numpy(), dt))).to(dt)
            assert torch.equal(torch.isnan(o.cpu()), torch.isnan(want))
            assert torch.equal(o.cpu().nan_to_num(nan=0.5), want.nan_to_num(nan=0.5))


def test_numbers_are_near_what_was_written():
    """Off by half a scale (1/30 of the range), the rounding of the scale (15 times half a step of it) and one of the result."""
    rng = np.random.RandomState(3)
    for t in ("f16", "bf16"):
        eps = torch.finfo(DT[t]).eps
        key = rows(rng, 200, 4, 128, t, 3.0)
        k, v = cache(13, 4, 16, 128), cache(13, 4, 16, 128)
        slots = dev(rng.permutation(13 * 16)[:200])
        pkv.reshape_and_cache_q4(key.to(DEV), key.to(DEV), k, v, slots)
        out = [torch.empty(200, 4, 128, device=DEV) for _ in "kv"]
        pkv.gather_cache_q4(*out, k, v, slots, dtype=DT[t])
        x = key.double().reshape(200, 4, 2, 64)
        span = x.amax(-1, keepdim=True) - x.amin(-1, keepdim=True)
        off = (out[0].cpu().double().reshape(200, 4, 2, 64) - x).abs()
        assert bool((off <= span / 30 * (1 + eps) + span * eps / 2 + 2.0 ** -16 * span + 1e-6).all())
        assert torch.equal(out[0], out[1])


def test_strided_rows():
    """Keys, values and queries as slices of a fused projection's output; results into slices of a wider buffer."""
    rng = np.random.RandomState(4)
    T, H, Hk, D, bs, NB = 9, 8, 2, 128, 16, 3
    qkv = torch.from_numpy(rng.randn(T, (H + 2 * Hk) * D)).bfloat16().to(DEV)
    q, key, value = (a.unflatten(1, (-1, D)) for a in qkv.split([H * D, Hk * D, Hk * D], 1))
    assert not key.is_contiguous()
    slots = dev(rng.permutation(NB * bs)[:T])
    a, b, st = [cache(NB, Hk, bs, D) for _ in "kv"], [cache(NB, Hk, bs, D) for _ in "kv"], status()
    pkv.reshape_and_cache_q4(key, value, *a, slots, device_status=st)
    pkv.reshape_and_cache_q4(key.contiguous(), value.contiguous(), *b, slots)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    wide = torch.full((T, 3 * Hk, D), 5.0, dtype=torch.bfloat16, device=DEV)
    plain = [torch.empty(T, Hk, D, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    pkv.gather_cache_q4(wide[:, Hk:2 * Hk], wide[:, 2 * Hk:], *a, slots, device_status=st)
    pkv.gather_cache_q4(*plain, *a, slots)
    assert torch.equal(wide[:, Hk:2 * Hk], plain[0]) and torch.equal(wide[:, 2 * Hk:], plain[1])
    assert bool((wide[:, :Hk] == 5.0).all())
    tables, lens = dev(np.arange(NB, dtype=np.int32)[None].repeat(T, 0)), dev(np.arange(T, dtype=np.int32) * 5)
    full = torch.zeros(NB * bs, Hk, D, dtype=torch.bfloat16, device=DEV).normal_()
    pkv.reshape_and_cache_q4(full, full, *a, torch.arange(NB * bs, device=DEV))
    out = [torch.empty(T, H, D, device=DEV) for _ in "ab"]
    pkv.paged_attention_decode_q4(out[0], q, *a, tables, lens, 0.1, device_status=st)
    pkv.paged_attention_decode_q4(out[1], q.contiguous(), *a, tables, lens, 0.1)
    assert torch.equal(out[0], out[1]) and st.item() == 0
    # the only row of a wider batch: whatever its stride is
    one = torch.empty(1, H, D, device=DEV)
    pkv.paged_attention_decode_q4(one, q[3:4], *a, tables[3:4], lens[3:4], 0.1)
    assert torch.allclose(one[0], out[0][3], rtol=0, atol=1e-4)


def test_slots_out_of_range_and_repeated():
    rng = np.random.RandomState(5)
    T, Hk, D, bs, NB = 6, 3, 64, 8, 4
    x = rows(rng, T, Hk, D, "f16")
    slots = np.array([3, -1, NB * bs, 31, -(1 << 40), 1 << 40])
    k, v, st = cache(NB, Hk, bs, D), cache(NB, Hk, bs, D), status()
    pkv.reshape_and_cache_q4(x.to(DEV), x.to(DEV), k, v, dev(slots), device_status=st)
    assert st.item() == pkv.DEV_BAD_SLOT
    check_written(k, x, slots, torch.float16, NB, bs)
    out = [torch.full((T, Hk, D), 7.0, dtype=torch.float16, device=DEV) for _ in "kv"]
    st.zero_()
    pkv.gather_cache_q4(*out, k, v, dev(np.array([3, -1, 1 << 50, 31, 3, 3])), device_status=st)
    assert st.item() == pkv.DEV_BAD_SLOT
    assert bool((out[0][1:3] == 7.0).all()) and torch.equal(out[0][0], out[0][4]) and torch.equal(out[0][0], out[0][5])
    assert not bool((out[0][0] == 7.0).all())


def test_copy_and_swap_move_a_4_bit_cache():
    rng = np.random.RandomState(6)
    Hk, D, bs = 5, 64, 8
    k, v, st = cache(6, Hk, bs, D), cache(6, Hk, bs, D), status()
    x, y = rows(rng, 12, Hk, D, "f16"), rows(rng, 12, Hk, D, "f16")
    pkv.reshape_and_cache_q4(x.to(DEV), y.to(DEV), k, v, dev(np.concatenate([24 + np.arange(8), 8 + np.arange(4)])))
    pkv.copy_blocks([k], [v], dev(np.array([[3, 0], [1, 5]], np.int64)), device_status=st)
    host = [torch.zeros(2, *k.shape[1:], dtype=torch.uint8).pin_memory() for _ in "kv"]
    pkv.swap_blocks([k], [v], host[:1], host[1:], dev(np.array([[0, 1], [5, 0]], np.int64)), pkv.SWAP_OUT, device_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    for a, b, h in ((3, 0, 1), (1, 5, 0)):
        for c, o in zip((k, v), host):
            assert torch.equal(c[a], c[b]) and torch.equal(c[a].cpu(), o[h])


# ------------------------------------------------------------------ decode


def run_decode(c, P=0, out_dtype=torch.float32, max_len=None, stream=None, workspace=None):
    out = torch.full(tuple(c["q"].shape), float("nan"), dtype=out_dtype, device=DEV)
    st = status()
    pkv.paged_attention_decode_q4(out, c["q"].to(DEV), dev(c["k"]), dev(c["v"]), dev(c["tables"]), dev(c["lens"]), c["scale"],
                                  max_context_len=max_len, partition_size=P, workspace=workspace, device_status=st, stream=stream)
    torch.cuda.synchronize()
    return out.double().cpu().numpy(), int(st.item())


def check(c, got, out_dtype=torch.float32):
    ref, score, value = S.attention_reference(c)
    tol = S.attention_tolerance(c, ref, score, value, out_dtype)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (np.abs(got - ref)[bad][:5], tol[bad][:5], np.argwhere(bad)[:5])


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("G", [1, 2, 3, 5, 8])
def test_decode_matrix(t, D, bs, G):
    lens = (1, bs - 1, bs, bs + 1, 3 * bs + 5, 0, 64, 100, 511, 513, 1100)
    c = S.q4_case(D + bs + G, t=t, G=G, Hk=2 if G < 8 else 3, D=D, bs=bs, lens=lens)
    for P, out_dtype in ((0, torch.float32), (64, torch.float32), (256, DT[t]), (2048, torch.float32)):
        got, st = run_decode(c, P, out_dtype)
        assert st == 0
        check(c, got, out_dtype)
        assert (got[5] == 0).all()


@pytest.mark.parametrize("bs", [8, 32])
@pytest.mark.parametrize("lens", [(5000,), (9000, 3), (2, 4097, 1, 2049)])
def test_decode_long_and_few(bs, lens):
    """Few rows, so that a row's partitions are a cluster or go through the workspace."""
    for D, t in ((64, "f16"), (128, "bf16")):
        c = S.q4_case(7, t=t, G=4, Hk=1, D=D, bs=bs, lens=lens)
        for P in (0, 32, 1024):
            got, st = run_decode(c, P)
            assert st == 0
            check(c, got)


def test_decode_many_rows():
    """More rows than SMs; lengths from 0 on."""
    rng = np.random.RandomState(8)
    c = S.q4_case(8, t="f16", G=2, Hk=8, D=128, bs=16, lens=rng.randint(0, 70, 90))
    got, st = run_decode(c)
    assert st == 0
    check(c, got)


@pytest.mark.parametrize("size", [2.0 ** -12, 2.0 ** -3, 40.0])
@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_decode_sizes(t, size):
    """Small and large numbers in K and V; scores from next to none to hundreds."""
    c = S.q4_case(9, t=t, G=3, Hk=2, lens=(1, 130, 700), size=size)
    got, st = run_decode(c)
    assert st == 0
    check(c, got)


def test_decode_large_offsets_and_far_scores():
    """Minima far from zero, as keys with a common part have; a scale that puts the scores thousands apart; scale 0 and
    below 0."""
    for scale in (3.0, 0.0, -0.2):
        c = S.q4_case(10, t="bf16", G=4, lens=(77, 400), offset=20.0)
        c["scale"] = float(np.float32(scale))
        got, st = run_decode(c)
        assert st == 0
        check(c, got)


def test_decode_bfloat16_range():
    """V's numbers near the ends of bfloat16's range, and scales of 0 (groups of one value)."""
    for e in (2.0 ** 100, 2.0 ** -100):
        c = S.q4_case(11, t="bf16", G=2, lens=(50, 200))
        u, s, m = c["v_parts"]
        s, m = s * e, m * e
        s[:, :, 3] = 0.0
        c["v_parts"], c["v"] = (u, s, m), S.pack(u, s, m, torch.bfloat16)
        got, st = run_decode(c)
        assert st == 0
        check(c, got)


def test_decode_scales_far_apart_in_a_context():
    """One token whose value is 2^30 times the others' and whose weight is next to none, and the reverse."""
    for D in (64, 128):
        c = S.q4_case(12, t="bf16", G=4, Hk=1, D=D, lens=(300,))
        (uk, sk, mk), (uv, sv, mv) = c["k_parts"], c["v_parts"]
        b, r = c["tables"][0, 7], 5
        sv[b, :, r] *= 2.0 ** 30
        mv[b, :, r] *= 2.0 ** 30
        c["v"] = S.pack(uv, sv, mv, torch.bfloat16)
        got, st = run_decode(c)
        check(c, got)
        assert st == 0


def test_nan_groups_reach_their_heads_only():
    c = S.q4_case(13, t="f16", G=2, Hk=3, D=128, lens=(100, 33))
    for n, (h, j) in (("k", (0, 1)), ("v", (1, 1))):
        u, s, m = c[n + "_parts"]
        b = c["tables"][0, 2]
        s[b, h, 3, j] = m[b, h, 3, j] = np.nan
        c[n] = S.pack(u, s, m, torch.float16)
    got, st = run_decode(c)
    assert st == 0
    assert np.isnan(got[0, 0:2]).all()                      # a key: its kv head's rows
    assert np.isnan(got[0, 2:4, 64:]).all()                 # a value: its group of dimensions
    clean = S.q4_case(13, t="f16", G=2, Hk=3, D=128, lens=(100, 33))
    ref, score, value = S.attention_reference(clean)
    tol = S.attention_tolerance(clean, ref, score, value, torch.float32)
    rest = np.ones(got.shape, bool)
    rest[0, 0:2] = rest[0, 2:4, 64:] = False
    assert (np.abs(got - ref)[rest] <= tol[rest]).all()


@pytest.mark.parametrize("P", [0, 32])
def test_bad_data_gives_zero_rows(P):
    c = S.q4_case(14, t="bf16", G=4, Hk=2, lens=(100, 60, 90, 40, 200))
    good = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in c.items()}
    c["tables"][1, 2] = c["NB"]
    got, st = run_decode(c, P, max_len=200)
    assert st == pkv.DEV_BAD_BLOCK and (got[1] == 0).all()
    c["tables"][1, 2] = -7
    c["lens"][3] = -1
    got, st = run_decode(c, P, max_len=200)
    assert st == pkv.DEV_BAD_BLOCK | pkv.DEV_BAD_CONTEXT_LEN and (got[[1, 3]] == 0).all()
    c["lens"][3] = 201
    got, st = run_decode(c, P, max_len=200)
    assert st == pkv.DEV_BAD_BLOCK | pkv.DEV_BAD_CONTEXT_LEN and (got[[1, 3]] == 0).all()
    ref, score, value = S.attention_reference(good)
    tol = S.attention_tolerance(good, ref, score, value, torch.float32)
    for b in (0, 2, 4):
        assert (np.abs(got[b] - ref[b]) <= tol[b]).all()


def test_offsets_past_32_bits():
    """A pool of 2.6 GB per cache; the sequence's blocks and the written slots lie at its end."""
    NB, Hk, bs, D = 18000, 64, 32, 128
    k, v = (torch.empty(NB, Hk, bs, D // 2 + D // 16, dtype=torch.uint8, device=DEV) for _ in "kv")
    assert k.numel() > (1 << 31) + (1 << 28)
    L = 70
    g = torch.Generator(device=DEV).manual_seed(0)
    key, value = (torch.randn(L, Hk, D, generator=g, device=DEV).half() for _ in "kv")
    table = np.array([[NB - 1, NB - 2, NB - 3]], np.int32)
    pos = np.arange(L)
    slots = dev(table[0, pos // bs].astype(np.int64) * bs + pos % bs)
    st = status()
    pkv.reshape_and_cache_q4(key, value, k, v, slots, device_status=st)
    back = [torch.empty(L, Hk, D, device=DEV) for _ in "kv"]
    pkv.gather_cache_q4(*back, k, v, slots, dtype=torch.float16, device_status=st)
    wu, ws, wm = S.quantize(key.double().cpu().numpy(), torch.float16)
    assert torch.equal(back[0].cpu(), torch.from_numpy(S.numbers(wu, ws, wm)).float())
    q = torch.randn(1, Hk, D, generator=g, device=DEV).half()
    out = torch.empty(1, Hk, D, device=DEV)
    pkv.paged_attention_decode_q4(out, q, k, v, dev(table), dev(np.array([L], np.int32)), D ** -0.5, device_status=st)
    z = torch.einsum("hd,thd->ht", q[0].double(), back[0].double()) * D ** -0.5
    want = torch.einsum("ht,thd->hd", torch.softmax(z, -1), back[1].double())
    assert st.item() == 0 and float((out[0].double() - want).abs().max()) < 5e-5


def test_run_together():
    """Prompts, then decode steps that grow them, then a prefix read back: every step's attention over what the cache
    stands for at that time."""
    rng = np.random.RandomState(15)
    for t, D, bs, Hk, G in (("bf16", 128, 16, 2, 4), ("f16", 64, 8, 3, 2)):
        pool = pkv.BlockPool(200, bs)
        first, steps = [1, 30, 64, 7], 20
        tables = np.full((4, 16), -1, np.int32)
        k, v, st = cache(200, Hk, bs, D), cache(200, Hk, bs, D), status()
        all_k, all_v = [], []
        for s, n in enumerate(first):
            table, _ = pool.allocate_prompt(rng.randint(0, 1000, n))
            tables[s, : len(table)] = table
            x, y = rows(rng, n, Hk, D, t), rows(rng, n, Hk, D, t)
            pos = np.arange(n)
            pkv.reshape_and_cache_q4(x.to(DEV), y.to(DEV), k, v, dev(table[pos // bs].astype(np.int64) * bs + pos % bs), device_status=st)
            all_k.append(x)
            all_v.append(y)
        lens = np.array(first, np.int32)
        for step in range(steps):
            slots, pairs = pool.append_slots(tables, lens)
            assert len(pairs) == 0
            x, y = rows(rng, 4, Hk, D, t, 1 + step % 3), rows(rng, 4, Hk, D, t)
            pkv.reshape_and_cache_q4(x.to(DEV), y.to(DEV), k, v, dev(slots), device_status=st)
            for s in range(4):
                all_k[s], all_v[s] = torch.cat([all_k[s], x[s:s + 1]]), torch.cat([all_v[s], y[s:s + 1]])
            lens += 1
            if step % 6 == 0 or step == steps - 1:
                q = torch.from_numpy(rng.randn(4, Hk * G, D)).to(DT[t])
                out = torch.empty(4, Hk * G, D, device=DEV)
                pkv.paged_attention_decode_q4(out, q.to(DEV), k, v, dev(tables), dev(lens), D ** -0.5, device_status=st)
                for s in range(4):
                    kk, vv = (S.numbers(*S.quantize(a[s].double().numpy(), DT[t])) for a in (all_k, all_v))
                    for h in range(Hk):
                        z = q[s, h * G:(h + 1) * G].double().numpy() @ kk[:, h].T * D ** -0.5
                        p = np.exp(z - z.max(-1, keepdims=True))
                        want = (p / p.sum(-1, keepdims=True)) @ vv[:, h]
                        # scores of a few units and numbers below 16: the tolerance of q4_support is below this
                        assert np.abs(out[s, h * G:(h + 1) * G].double().cpu().numpy() - want).max() < 1e-3
        pos = np.arange(int(lens[2]))
        back = [torch.empty(len(pos), Hk, D, dtype=DT[t], device=DEV) for _ in "kv"]
        pkv.gather_cache_q4(*back, k, v, dev(tables[2, pos // bs].astype(np.int64) * bs + pos % bs), device_status=st)
        for b, a in zip(back, (all_k[2], all_v[2])):
            assert torch.equal(b.cpu(), torch.from_numpy(S.numbers(*S.quantize(a.double().numpy(), DT[t]))).to(DT[t]))
        assert st.item() == 0


def test_decode_shares_of_many_chunks():
    """8.4M tokens over all rows: a share of the stream is longer than what a CTA looks up at once, and its chunks end in
    the middle of rows.  Checked for some heads against 64-bit attention over the numbers read back."""
    Hk, D, bs, L = 64, 64, 32, 131072 - 5
    MB = -(-L // bs)
    g = torch.Generator(device=DEV).manual_seed(3)
    table = torch.randperm(MB + 3, generator=g, device=DEV)[:MB].to(torch.int32)
    k, v, st = cache(MB + 3, Hk, bs, D), cache(MB + 3, Hk, bs, D), status()
    pos = torch.arange(L, device=DEV)
    slots = table.long()[pos // bs] * bs + pos % bs
    back = []
    for c in (k, v):
        x = torch.randn(L, Hk, D, generator=g, device=DEV).bfloat16()
        pkv.reshape_and_cache_q4(x, x, c, c, slots, device_status=st)
        y = torch.empty(L, Hk, D, device=DEV)
        pkv.gather_cache_q4(y, y, c, c, slots, dtype=torch.bfloat16, device_status=st)
        back.append(y)
        del x
    q = torch.randn(1, Hk, D, generator=g, device=DEV).bfloat16()
    out = torch.empty(1, Hk, D, device=DEV)
    pkv.paged_attention_decode_q4(out, q, k, v, table[None], torch.tensor([L], dtype=torch.int32, device=DEV), D ** -0.5, device_status=st)
    assert st.item() == 0
    for h in range(0, Hk, 7):
        kk, vv = (b[:, h].double() for b in back)
        want = torch.softmax(q[0, h].double() @ kk.T * D ** -0.5, -1) @ vv
        # scores below 10 off by less than (D + 8) 2^-23 x 60; sums of 131,067 weights cut 2^-23 each: of numbers below 8
        assert float((out[0, h].double() - want).abs().max()) < 8 * (2 * 72 * 60 + L) * 2.0 ** -23 / 8


@pytest.mark.parametrize("lens", [(2600, 0, 33, 31, 700, 1, 32, 4000, 64, 0), tuple([5] * 300), tuple([200, 1] * 40), (1,) * 7 + (3000,)])
def test_decode_ragged_rows_in_a_stream(lens):
    """Rows that begin and end anywhere in the shares, sequences without tokens between them."""
    for D, t, bs in ((64, "f16", 8), (128, "bf16", 16), (128, "f16", 32)):
        c = S.q4_case(16, t=t, G=3, Hk=5, D=D, bs=bs, lens=lens)
        got, st = run_decode(c, max_len=8192 if max(lens) < 8192 and c["tables"].shape[1] * bs >= 8192 else None)
        assert st == 0
        check(c, got)


@pytest.mark.parametrize("what", ["block", "length"])
def test_bad_data_in_a_stream(what):
    """A refused sequence among many: its rows are zero, its neighbours in the same shares are not touched."""
    lens = [300, 900, 40, 2000, 64, 1500] * 4
    c = S.q4_case(17, t="bf16", G=4, Hk=7, lens=lens)
    good = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in c.items()}
    hurt = [3, 8, 23]
    for s in hurt:
        if what == "block":
            c["tables"][s, 1] = c["NB"] + s
        else:
            c["lens"][s] = -s if s % 2 else 2001
    got, st = run_decode(c, max_len=2000)
    assert st == (pkv.DEV_BAD_BLOCK if what == "block" else pkv.DEV_BAD_CONTEXT_LEN)
    assert (got[hurt] == 0).all()
    ref, score, value = S.attention_reference(good)
    tol = S.attention_tolerance(good, ref, score, value, torch.float32)
    rest = [s for s in range(len(lens)) if s not in hurt]
    assert (np.abs(got - ref)[rest] <= tol[rest]).all()


@pytest.mark.parametrize("t,D,bs,Hk,T", [("f16", 128, 16, 3, 20011), ("bf16", 64, 8, 5, 30011), ("bf16", 128, 32, 70, 1501), ("f16", 64, 16, 1, 50003),
                                         ("f16", 128, 8, 2500, 3), ("bf16", 64, 8, 40000, 1)])
def test_write_and_read_many(t, D, bs, Hk, T):
    """CTAs of many tokens, tokens of many CTAs; some of the tokens are padding."""
    rng = np.random.RandomState(T)
    g = torch.Generator(device=DEV).manual_seed(T)
    NB = -(-T // bs) + 2
    slots = rng.permutation(NB * bs)[:T]
    slots[rng.rand(T) < 0.1] = -5
    key, value = (torch.randn(T, Hk, D, generator=g, device=DEV).mul_(3).to(DT[t]) for _ in "kv")
    k, v, st = cache(NB, Hk, bs, D), cache(NB, Hk, bs, D), status()
    pkv.reshape_and_cache_q4(key, value, k, v, dev(slots), device_status=st)
    out = [torch.full((T, Hk, D), 7.0, device=DEV) for _ in "kv"]
    pkv.gather_cache_q4(*out, k, v, dev(slots), dtype=DT[t], device_status=st)
    assert st.item() == 0
    for o, x in zip(out, (key, value)):
        want = torch.from_numpy(S.numbers(*S.quantize(x.double().cpu().numpy(), DT[t]))).float()
        want[torch.from_numpy(slots < 0)] = 7.0
        assert torch.equal(o.cpu(), want)


@pytest.mark.parametrize("G", [2, 8])
def test_long_sums_have_no_bias(G):
    """Equal weights (q = 0) over one long context, by one CTA: an output is the mean of 60,000 numbers of both signs, far
    below the codes' part of it.  What tensor cores cut off always goes towards zero: within a step's four products it is
    at most 4 x 2^-23 of the codes' sum, and it must not build up over the 469 steps that a warp takes (codes of any value
    being as likely, half of the steps cut it from the other side)."""
    for t, D in (("f16", 128), ("bf16", 64)):
        c = S.q4_case(18, t=t, G=G, Hk=1, D=D, bs=32, lens=(60000,), offset=0.0)
        c["q"].zero_()
        got, st = run_decode(c, P=60032 - 60032 % 32)
        assert st == 0
        ref, _, value = S.attention_reference(c)
        assert np.abs(ref).max() < 0.1 * value.max()
        assert abs((got - ref).mean()) < 4 * 2.0 ** -23 * value.max()
        check(c, got)


@pytest.mark.parametrize("where", [3, 300, 700, 749])
def test_bad_block_in_a_row_of_several_chunks(where):
    """A CTA's part of a row is longer than what it looks up at once; the bad block lies in any piece of it.  All heads and
    dimensions are zero, every time."""
    c = S.q4_case(19, t="bf16", G=8, Hk=2, D=128, bs=16, lens=(12000, 5000))
    c["tables"][0, where] = -1
    for P in (0, 12000 // 32 * 32 + 32, 8192):
        for _ in range(5):
            got, st = run_decode(c, P)
            assert st == pkv.DEV_BAD_BLOCK and (got[0] == 0).all() and (got[1] != 0).all()


def test_rows_of_zeros():
    """A fresh cache (zeros: scales, minima and codes), one whose tokens are zeros in part, and values of zeros under keys
    that are not."""
    for G in (3, 8):
        c = S.q4_case(20, t="f16", G=G, Hk=2, lens=(900, 70))
        for n in ("kv", "v", "half"):
            for x in ("k", "v") if n == "kv" else ("v",):
                u, s, m = (a.copy() for a in c[x + "_parts"])
                hit = np.ones(s.shape, bool) if n != "half" else np.arange(s.shape[2])[None, None, :, None] % 3 > 0
                s[np.broadcast_to(hit, s.shape) & ~np.isnan(s)] = 0.0
                m[np.broadcast_to(hit, m.shape) & ~np.isnan(m)] = 0.0
                c2 = dict(c)
                c2[x + "_parts"], c2[x] = (u, s, m), S.pack(u, s, m, torch.float16)
                for P in (0, 64):
                    got, st = run_decode(c2, P)
                    assert st == 0
                    check(c2, got)
                    if n == "v" or x == "v" and n == "kv":
                        assert (got == 0).all()


@pytest.mark.parametrize("T", [1823, 1824, 3647, 3649, 7301])
@pytest.mark.parametrize("D,Hk", [(64, 5), (128, 8)])
def test_write_and_read_between(D, Hk, T):
    """Calls at which CTAs begin to take two, four and eight times their rows: the records that parts of the same
    rows leave, and the numbers that parts of the same slots give."""
    rng = np.random.RandomState(T + D)
    g = torch.Generator(device=DEV).manual_seed(T)
    NB = -(-T // 16) + 1
    slots = rng.permutation(NB * 16)[:T]
    slots[rng.rand(T) < 0.05] = -1
    at = dev(slots)
    key, value = (torch.randn(T, Hk, D, generator=g, device=DEV).to(torch.bfloat16) for _ in "kv")
    whole, parts = [[cache(NB, Hk, 16, D) for _ in "kv"] for _ in range(2)]
    pkv.reshape_and_cache_q4(key, value, *whole, at)
    for i in range(0, T, 200):
        pkv.reshape_and_cache_q4(key[i: i + 200], value[i: i + 200], *parts, at[i: i + 200])
    assert all(torch.equal(a, b) for a, b in zip(whole, parts))
    out, rest = [[torch.full((T, Hk, D), 7.0, dtype=torch.bfloat16, device=DEV) for _ in "kv"] for _ in range(2)]
    pkv.gather_cache_q4(*out, *whole, at)
    for i in range(0, T, 200):
        pkv.gather_cache_q4(rest[0][i: i + 200], rest[1][i: i + 200], *whole, at[i: i + 200])
    assert all(torch.equal(a, b) for a, b in zip(out, rest))
