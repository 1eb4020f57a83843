"""Block summaries, block selection and attention over selected blocks on the
GPU, against their definitions in 64 bits; and a run of the whole decode step
over an 8-bit cache, also captured in a graph."""
import numpy as np
import pytest
import torch

import paged_kv_cache_311_gb300 as pkv
from tests import q8_support as S
from tests.test_gpu_q8 import check, dev, reference, rows

pytestmark = pytest.mark.gpu
DEV = "cuda"
f8 = lambda b: dev(b).view(torch.float8_e4m3fn)  # noqa: E731


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# --------------------------------------------------------------- summaries


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("Hk", [1, 8, 9])
def test_summaries(kind, D, bs, Hk):
    """After prompts and after a step: touched blocks hold the range of the
    rows that are there, whatever lies behind them; others keep their bytes."""
    lens = np.array([1, bs - 1, bs, bs + 1, 3 * bs + 5, 0, 200])
    c = S.q8_case(D + bs + Hk, G=1, Hk=Hk, D=D, bs=bs, lens=lens)
    NB = c["NB"]
    if kind == "q8":
        k, ks, sdt = f8(c["k_bits"]), dev(c["k_scale"]), torch.bfloat16
        real = S.decode(c["k_bits"]) * c["k_scale"][:, :Hk, None, None].astype(np.float64)
    else:
        sdt = S.DT[kind]
        k, ks = torch.from_numpy(np.random.RandomState(1).randn(NB, Hk, bs, D)).to(sdt).to(DEV), None
        real = k.double().cpu().numpy()
        for s, L in enumerate(lens):
            if L % bs:
                k[c["tables"][s, L // bs], :, L % bs:] = float("nan")
    for new in (lens, np.minimum(lens, 1), np.minimum(lens, bs + 2)):
        sums = torch.full((NB, Hk, 2, D), 7.0, dtype=sdt, device=DEV)
        starts = np.concatenate([[0], np.cumsum(new)])
        st = status()
        pkv.summarize_blocks(k, sums, dev(c["tables"]), dev(c["lens"]), dev(starts.astype(np.int32)),
                             num_tokens=int(starts[-1]), k_scales=ks, device_status=st)
        assert st.item() == 0
        want = np.full((NB, Hk, 2, D), 7.0)
        for s in range(len(lens)):
            for j, a, b, _ in S.touched(int(lens[s]), int(new[s]), bs):
                blk = c["tables"][s, j]
                want[blk, :, 0], want[blk, :, 1] = real[blk, :, :b].min(1), real[blk, :, :b].max(1)
        np.testing.assert_array_equal(sums.double().cpu().numpy(), want)
    sums2 = torch.full((NB, Hk, 2, D), 7.0, dtype=sdt, device=DEV)
    pkv.summarize_blocks(k, sums2, dev(c["tables"]), dev(c["lens"]), k_scales=ks, device_status=st)   # a step, one length 0
    sums3 = torch.full((NB, Hk, 2, D), 7.0, dtype=sdt, device=DEV)
    new = np.minimum(lens, 1)
    pkv.summarize_blocks(k, sums3, dev(c["tables"]), dev(c["lens"]), dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)),
                         num_tokens=int(new.sum()), k_scales=ks, device_status=st)
    assert st.item() == 0 and torch.equal(sums2, sums3)


def test_summaries_show_nan():
    k = torch.randn(2, 2, 16, 64, device=DEV).half()
    k[1, 1, 3, 5] = float("nan")
    sums = torch.zeros(2, 2, 2, 64, dtype=torch.float16, device=DEV)
    pkv.summarize_blocks(k, sums, dev(np.array([[1]], np.int32)), dev(np.array([16], np.int32)))
    nan = torch.isnan(sums)
    assert nan[1, 1, :, 5].all() and nan.sum() == 2


# --------------------------------------------------------------- selection


def select_case(seed, lens, *, G=4, Hk=2, D=128, bs=16, t="f16", same=False):
    rng = np.random.RandomState(seed)
    lens = np.asarray(lens, np.int32)
    tables, NB = S.make_tables(rng, [-(-int(n) // bs) for n in lens])
    k = torch.from_numpy(rng.randn(NB, Hk, 4, D) + rng.randn(NB, Hk, 1, D)).to(S.DT[t])
    sums = torch.stack([k.amin(2), k.amax(2)], 2).contiguous()
    if same:
        sums[:] = sums[0]
    q = torch.from_numpy(rng.randn(len(lens), G * Hk, D)).to(S.DT[t])
    return dict(lens=lens, tables=tables, NB=NB, sums=sums, q=q, bs=bs, Hk=Hk)


def run_select(c, K, first=1, last=1, max_len=None):
    sel = torch.full((len(c["lens"]), c["Hk"], K), 99, dtype=torch.int32, device=DEV)
    st = status()
    pkv.select_blocks(sel, c["q"].to(DEV), c["sums"].to(DEV), dev(c["tables"]), dev(c["lens"]), c["bs"], keep_first=first,
                      keep_last=last, max_context_len=max_len, device_status=st)
    return sel.cpu().numpy(), int(st.item())


def want_select(c, K, first=1, last=1):
    s = c["sums"].double().numpy()
    return S.select_reference(c["q"].double().numpy(), s[:, :, 0], s[:, :, 1], c["tables"], c["lens"], c["bs"], K, first, last)


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [8, 32])
@pytest.mark.parametrize("G", [1, 3, 8])
def test_select_matrix(t, D, bs, G):
    c = select_case(D + bs + G, [0, 1, bs, 20 * bs - 1, 20 * bs, 77 * bs + 3, 300 * bs], G=G, D=D, bs=bs, t=t)
    for K, first, last in ((1, 0, 0), (1, 0, 1), (20, 1, 2), (64, 0, 3), (300, 1, 1), (5, 2, 3)):
        got, st = run_select(c, K, first, last)
        assert st == 0
        np.testing.assert_array_equal(got, want_select(c, K, first, last))


@pytest.mark.parametrize("blocks", [255, 256, 257, 600, 1025, 2049, 5000])
def test_select_over_several_ctas(blocks):
    """Long contexts, scored by one to eight CTAs, beside shorter ones."""
    c = select_case(blocks, [blocks * 8, blocks * 8 - 7, blocks * 4, 8 * 40], D=64, bs=8, t="bf16")
    for K in (17, 128, 250):
        got, st = run_select(c, K, 1, 2)
        assert st == 0
        np.testing.assert_array_equal(got, want_select(c, K, 1, 2))


@pytest.mark.parametrize("blocks", [100, 700, 3000])
def test_select_ties_go_to_the_lowest_block(blocks):
    """All summaries alike: the first blocks that are not kept anyway; then two
    kinds of blocks, the better one rarer than the places."""
    c = select_case(blocks, [blocks * 16, blocks * 8], same=True)
    got, st = run_select(c, 40, 1, 2)
    want = want_select(c, 40, 1, 2)
    np.testing.assert_array_equal(want[0, 0], np.concatenate([np.arange(38), [blocks - 2, blocks - 1]]))
    np.testing.assert_array_equal(got, want)
    rng = np.random.RandomState(0)
    for blk in rng.choice(c["NB"], c["NB"] // 10, replace=False):
        c["sums"][blk] = c["sums"][blk] + 1.0
    for K in (8, 30, 200):
        got, st = run_select(c, K, 0, 1)
        assert st == 0
        np.testing.assert_array_equal(got, want_select(c, K, 0, 1))


def test_select_scores_closer_than_fp32_tells():
    """Scores of the order of 2^14 that differ by 2^-12 and less: 26 bits and
    more apart, found by the 64-bit scores."""
    D, n, bs = 128, 900, 16
    c = select_case(5, [n * bs, 300 * bs], G=1, Hk=1, D=D, bs=bs, t="f16")
    c["q"][:] = 1.0
    s = torch.zeros(c["NB"], 1, 2, D, dtype=torch.float16)
    s[:, :, 1, :-2] = 128.0
    rng = np.random.RandomState(3)
    s[:, :, 1, -2] = torch.from_numpy(rng.randint(1, 40, (c["NB"], 1)) * 2.0 ** -12).half()
    s[:, :, 1, -1] = torch.from_numpy(rng.randint(0, 3, (c["NB"], 1)) * 2.0 ** -14).half()
    c["sums"] = s
    for K in (10, 100, 299):
        got, st = run_select(c, K, 0, 1)
        assert st == 0
        np.testing.assert_array_equal(got, want_select(c, K, 0, 1))


def test_select_nan_and_infinities():
    """A block with NaN or with an infinite bound is selected, and a bound that
    overflows fp32 but not fp64 counts as the number it is."""
    c = select_case(6, [500 * 16, 90 * 16], G=2, t="bf16")
    c["q"] = c["q"].abs() + 0.125
    t = c["tables"]
    for s, n in ((0, 500), (1, 90)):
        c["sums"][t[s, 41], 0, 1, 3] = float("nan")
        c["sums"][t[s, 57], :, 1, 9] = float("inf")
        c["sums"][t[s, 3], 1, :, 9] = 3.0e38
    got, st = run_select(c, 12, 1, 1)
    assert st == 0
    for s in range(2):
        assert 41 in got[s, 0] and 57 in got[s, 0] and 57 in got[s, 1] and 3 in got[s, 1]
    np.testing.assert_array_equal(got, want_select(c, 12, 1, 1))


@pytest.mark.parametrize("e", [-70, -100, -115, -126, -131])
@pytest.mark.parametrize("n", [500, 4000])
def test_select_of_tiny_summaries(e, n):
    """Keys near the end of bfloat16's range: the products leave fp32's normal
    numbers, the choice stays that of the definition (exact in fp64)."""
    c = select_case(14, [n * 16, n * 16 - 5], G=2, t="bf16")
    c["sums"] = (c["sums"].double() * 2.0 ** e).to(torch.bfloat16)
    for K in (12, 100):
        got, st = run_select(c, K, 1, 1)
        assert st == 0
        np.testing.assert_array_equal(got, want_select(c, K, 1, 1))


@pytest.mark.parametrize("x", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("n", [500, 4000])
def test_select_with_a_query_that_is_not_finite(x, n):
    """Every score of its row counts as +infinity: the lowest blocks are kept.
    An infinite key makes its block's score +infinity, of whatever sign."""
    c = select_case(15, [n * 16] * 3, G=2, t="bf16")
    c["q"][0, 1, 5] = x
    c["sums"][c["tables"][1, 41], 0, 0, 9] = -abs(x)
    c["sums"][c["tables"][1, 52], 0, :, 9] = -abs(x)
    got, st = run_select(c, 12, 1, 2)
    assert st == 0
    want = want_select(c, 12, 1, 2)
    want[0, 0] = list(range(10)) + [n - 2, n - 1]
    assert 41 in want[1, 0] and 52 in want[1, 0]
    np.testing.assert_array_equal(got, want)


def test_select_through_the_workspace():
    """Many rows of many blocks: scored by one launch, selected by another.
    Lengths from 0 on, a sequence of equal blocks, NaN, a bad table and a bad
    length among them; the workspace given and not."""
    rng = np.random.RandomState(2)
    lens = rng.randint(1, 1200 * 8, 28)
    lens[3], lens[5], lens[7] = 0, 1200 * 8, 1199 * 8 + 1
    c = select_case(12, lens, G=2, Hk=4, D=64, bs=8, t="bf16")
    assert pkv.select_blocks_workspace_bytes(28, 4, 1200 * 8, 8) > 0
    t = c["tables"]
    c["sums"][t[5, :1200]] = c["sums"][t[5, 0]].clone()
    c["sums"][t[7, 100], 2, 0, 5] = float("nan")
    for K in (3, 48, 200):
        got, st = run_select(c, K, 1, 2, max_len=1200 * 8)
        assert st == 0
        np.testing.assert_array_equal(got, want_select(c, K, 1, 2))
    ws = torch.full((pkv.select_blocks_workspace_bytes(28, 4, 1200 * 8, 8),), 255, dtype=torch.uint8, device=DEV)
    sel, st = torch.zeros(28, 4, 48, dtype=torch.int32, device=DEV), status()
    good, _ = run_select(c, 48, 0, 1, max_len=1200 * 8)
    c["tables"][11, (lens[11] - 1) // 8], c["lens"][12] = -1, 1201 * 8
    pkv.select_blocks(sel, c["q"].to(DEV), c["sums"].to(DEV), dev(c["tables"]), dev(c["lens"]), 8, keep_first=0, keep_last=1,
                      max_context_len=1200 * 8, workspace=ws, device_status=st)
    assert st.item() == pkv.DEV_BAD_BLOCK | pkv.DEV_BAD_CONTEXT_LEN
    good[[11, 12]] = -1
    np.testing.assert_array_equal(sel.cpu().numpy(), good)


@pytest.mark.parametrize("B, Hk, n", [(80, 8, 5), (80, 8, 200), (31, 5, 60), (40, 8, 130), (19, 8, 250)])
@pytest.mark.parametrize("D", [64, 128])
def test_select_of_many_rows(B, Hk, n, D):
    """More rows than SMs hold CTAs: smaller CTAs, in one launch and in two; bins of
    equal scores among them."""
    rng = np.random.RandomState(n)
    lens = rng.randint(0, n * 16 + 1, B)
    lens[0], lens[1] = n * 16, 0
    c = select_case(21, lens, G=2, Hk=Hk, D=D, t="bf16")
    c["sums"][c["tables"][0, :n]] = c["sums"][c["tables"][0, 0]].clone()
    for K in (4, n // 3 + 2):
        got, st = run_select(c, K, 1, 2)
        assert st == 0
        np.testing.assert_array_equal(got, want_select(c, K, 1, 2))


def test_select_refuses_bad_rows():
    c = select_case(8, [3000, 3000, 3000, 3000])
    good, _ = run_select(c, 16)
    c["tables"][1, 180] = c["NB"]
    c["lens"][2] = -5
    got, st = run_select(c, 16, max_len=3000)
    assert st == pkv.DEV_BAD_BLOCK | pkv.DEV_BAD_CONTEXT_LEN
    assert (got[1] == -1).all() and (got[2] == -1).all()
    np.testing.assert_array_equal(got[[0, 3]], good[[0, 3]])


# --------------------------------------------- attention over selected blocks


def dense16(c, t, seed=0):
    """A 16-bit cache in the case's place: garbage is NaN."""
    rng = np.random.RandomState(seed)
    live = ~np.isnan(S.decode(c["k_bits"]))
    out = {}
    for n in "kv":
        x = np.where(live, rng.randn(*live.shape), np.nan)
        out[n] = torch.from_numpy(x).to(S.DT[t])
    return out["k"], out["v"]


def run_selected(c, sel, kv=None, P=0, out_dtype=torch.float32):
    out = torch.full(tuple(c["q"].shape), float("nan"), dtype=out_dtype, device=DEV)
    st = status()
    args = dict(k_scales=dev(c["k_scale"]), v_scales=dev(c["v_scale"])) if kv is None else {}
    k, v = (f8(c["k_bits"]), f8(c["v_bits"])) if kv is None else (kv[0].to(DEV), kv[1].to(DEV))
    pkv.paged_attention_decode_selected(out, c["q"].to(DEV), k, v, dev(c["tables"]), dev(c["lens"]), dev(sel), c["scale"],
                                        partition_size=P, device_status=st, **args)
    torch.cuda.synchronize()
    return out.double().cpu().numpy(), int(st.item())


def random_lists(c, K, seed):
    rng = np.random.RandomState(seed)
    sel = np.full((c["B"], c["Hk"], K), -1, np.int32)
    for s in range(c["B"]):
        n = -(-int(c["lens"][s]) // c["bs"])
        for h in range(c["Hk"]):
            m = min(n, rng.randint(0, K + 1) if h else K)
            pick = rng.choice(n, m, replace=False) if n else np.zeros(0, int)
            if m and h != 1:
                pick[0] = n - 1 if n - 1 not in pick else pick[0]
            sel[s, h, :m] = np.sort(pick)
    return sel


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("G", [1, 3, 8])
def test_selected_attention(kind, D, bs, G):
    """Random lists of every kv head's own, empty ones among them, with and
    without the sequence's partial last block."""
    c = S.q8_case(D + bs + G, qdtype="bf16" if kind == "q8" else kind, G=G, Hk=3, D=D, bs=bs,
                  lens=(1, bs, 5 * bs + 3, 0, 30 * bs + 1, 64 * bs - 1))
    kv = None if kind == "q8" else dense16(c, kind)
    for K in (1, 7, 40):
        sel = random_lists(c, K, K)
        listed = lambda s, h: sel[s, h][sel[s, h] >= 0]  # noqa: E731
        if kv is None:
            ref, bound, v = reference(c, listed)
        else:
            v = kv[1].double().numpy()
            ref, bound = S.attention_reference(c["q"].double().numpy(), kv[0].double().numpy(), v, c["tables"], c["lens"], bs,
                                               c["scale"], listed)
        for P in (0, 32):
            for od in (torch.float32, c["q"].dtype):
                got, st = run_selected(c, sel, kv, P, od)
                assert st == 0
                tol = S.attention_tolerance(ref, bound, v, c["lens"], D, od)
                assert (np.abs(got - ref) <= tol).all(), np.abs(got - ref).max()


def test_lists_longer_than_the_contexts():
    """Many rows, and room for more blocks than any context has: the whole
    attention, and a list that goes on behind its end is still refused."""
    rng = np.random.RandomState(5)
    lens = rng.randint(0, 141, 100)
    c = S.q8_case(9, G=2, Hk=2, D=64, lens=lens)
    sel = np.full((100, 2, 300), -1, np.int32)
    for s, L in enumerate(lens):
        sel[s, :, : -(-int(L) // 16)] = np.arange(-(-int(L) // 16))
    got, st = run_selected(c, sel)
    assert st == 0
    check(c, got, torch.float32)
    sel[7, 1, 290] = 0
    bad, st = run_selected(c, sel)
    assert st == pkv.DEV_BAD_BLOCK
    got[7, 2:] = 0
    np.testing.assert_array_equal(bad, got)


@pytest.mark.parametrize("kind", ["bf16", "q8"])
def test_all_blocks_selected_is_the_whole_attention(kind):
    c = S.q8_case(3, G=4, Hk=2, lens=(700, 16, 1))
    n = [-(-int(x) // 16) for x in c["lens"]]
    sel = np.full((3, 2, 50), -1, np.int32)
    for s in range(3):
        sel[s, :, : n[s]] = np.arange(n[s])
    if kind == "q8":
        got, st = run_selected(c, sel)
        check(c, got, torch.float32)
    else:
        k, v = dense16(c, "bf16")
        got, st = run_selected(c, sel, (k, v))
        out = torch.empty(tuple(c["q"].shape), device=DEV)
        pkv.paged_attention_decode(out, c["q"].to(DEV), k.to(DEV), v.to(DEV), dev(c["tables"]), dev(c["lens"]), c["scale"])
        vn = v.double().numpy()
        _, bound = S.attention_reference(c["q"].double().numpy(), k.double().numpy(), vn, c["tables"], c["lens"], 16, c["scale"])
        tol = S.attention_tolerance(got, bound, vn, c["lens"], 128, torch.float32)
        assert (np.abs(got - out.double().cpu().numpy()) <= 2 * tol).all()
    assert st == 0


@pytest.mark.parametrize("kind", ["f16", "q8"])
@pytest.mark.parametrize("P", [0, 32])
@pytest.mark.parametrize("bad", [[4, 3, 6], [2, 2, 6], [1, 2, 44], [1, -1, 5], [-2, -1, -1], [-1, 0, 1]])
def test_selected_refuses_bad_lists(kind, bad, P):
    """Lists that are not ascending, that repeat a block, name one beyond the
    context, go on behind a -1 or hold another negative number."""
    c = S.q8_case(4, qdtype="f16", G=2, Hk=2, lens=(700, 700))
    kv = None if kind == "q8" else dense16(c, "f16")
    sel = np.tile(np.array([1, 5, 9], np.int32), (2, 2, 1))
    good, st = run_selected(c, sel, kv, P)
    assert st == 0
    sel[1, 0] = bad
    got, st = run_selected(c, sel, kv, P)
    assert st == pkv.DEV_BAD_BLOCK
    assert not got[1, :2].any()
    np.testing.assert_array_equal(got[0], good[0])
    np.testing.assert_array_equal(got[1, 2:], good[1, 2:])


def test_binding_refuses_mismatches():
    c = S.q8_case(1, qdtype="f16", G=2, Hk=2, lens=(20, 20))
    q, k, sc, bt, cl = c["q"].to(DEV), f8(c["k_bits"]), dev(c["k_scale"]), dev(c["tables"]), dev(c["lens"])
    sel = torch.zeros(2, 2, 4, dtype=torch.int32, device=DEV)
    out = torch.empty_like(q)
    bad = [
        lambda: pkv.paged_attention_decode_q8(out, q, k, k, sc[:, :2].contiguous(), sc, bt, cl, 1.0),
        lambda: pkv.paged_attention_decode_q8(out, q, k.view(torch.uint8), k, sc, sc, bt, cl, 1.0),
        lambda: pkv.paged_attention_decode_q8(out[:1], q, k, k, sc, sc, bt, cl, 1.0),
        lambda: pkv.paged_attention_decode_q8(out, q, k, k, sc, sc, bt[:1], cl, 1.0),
        lambda: pkv.paged_attention_decode_q8(out, q, k, k, sc, sc, bt.long(), cl, 1.0),
        lambda: pkv.paged_attention_decode_q8(out, q, k, k, sc.cpu(), sc, bt, cl, 1.0),
        lambda: pkv.paged_attention_decode_q8(out, q.transpose(0, 1), k, k, sc, sc, bt, cl, 1.0),
        lambda: pkv.paged_attention_decode_q8(out, q, k, k, sc, sc, bt, cl, 1.0, device_status=torch.zeros(1, device=DEV)),
        lambda: pkv.paged_attention_decode_selected(out, q, k, k, bt, cl, sel, 1.0),
        lambda: pkv.paged_attention_decode_selected(out, q, k, k, bt, cl, sel[:, :1].contiguous(), 1.0, k_scales=sc, v_scales=sc),
        lambda: pkv.paged_attention_decode_selected(out, q, k, k, bt, cl, sel.long(), 1.0, k_scales=sc, v_scales=sc),
        lambda: pkv.select_blocks(sel, q, torch.zeros(c["NB"], 2, 2, 64, dtype=torch.float16, device=DEV), bt, cl, 16),
        lambda: pkv.summarize_blocks(k, torch.zeros(c["NB"], 2, 2, 128, dtype=torch.float16, device=DEV), bt, cl, k_scales=sc),
        lambda: pkv.summarize_blocks(k, torch.zeros(c["NB"], 2, 2, 128, dtype=torch.bfloat16, device=DEV), bt, cl),
        lambda: pkv.append_cache_q8(q[:1], q[:1], k, k, sc, sc, bt, cl),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(pkv.PkvError):
        pkv.paged_attention_decode_q8(out, q, k, k, sc, sc, bt, cl, 1.0, max_context_len=33)
    with pytest.raises(pkv.PkvError):
        pkv.paged_attention_decode_q8(out.float(), q.float(), k, k, sc, sc, bt, cl, 1.0)
    with pytest.raises(pkv.PkvError):
        pkv.select_blocks(sel, q, torch.zeros(c["NB"], 2, 2, 128, dtype=torch.float16, device=DEV), bt, cl, 16, keep_first=3, keep_last=2)


# -------------------------------------------------- a run of them together


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("q8", [True, False])
def test_decode_steps_over_selected_blocks(q8, captured):
    """Prompts, then decode steps as a serving loop makes them: write the new
    token, renew its block's summary, select blocks, attend to them.  Captured:
    one graph of the step, replayed with new lengths, tokens and queries."""
    rng = np.random.RandomState(9)
    B, Hk, G, D, bs, K, steps = 5, 2, 4, 128, 16, 6, 20
    t = torch.bfloat16
    first = np.array([300, 5, 64, 161, 32])
    need = [-(-(int(n) + steps) // bs) for n in first]
    tables, NB = S.make_tables(rng, need)
    MB = tables.shape[1]
    bt = dev(tables)
    st = status()
    if q8:
        k, v = (torch.zeros(NB, Hk, bs, D, dtype=torch.float8_e4m3fn, device=DEV) for _ in "kv")
        ks, vs = pkv.q8_scales(NB, Hk, DEV), pkv.q8_scales(NB, Hk, DEV)
        rk, rv = S.Q8Cache(NB, Hk, bs, D), S.Q8Cache(NB, Hk, bs, D)
    else:
        k, v = (torch.zeros(NB, Hk, bs, D, dtype=t, device=DEV) for _ in "kv")
        ks = vs = None
        rk, rv = np.zeros((NB, Hk, bs, D)), np.zeros((NB, Hk, bs, D))
    sums = torch.zeros(NB, Hk, 2, D, dtype=t, device=DEV)

    def write(key, value, lens, starts):
        if q8:
            pkv.append_cache_q8(key, value, k, v, ks, vs, bt, lens, starts, device_status=st)
        else:
            s = torch.arange(B, device=DEV) if starts is None else None
            pkv.reshape_and_cache(key, value, k, v, slots if s is None else bt[s, (lens.long() - 1) // bs].long() * bs
                                  + (lens.long() - 1) % bs, device_status=st)
        pkv.summarize_blocks(k, sums, bt, lens, starts, num_tokens=key.shape[0], k_scales=ks, device_status=st)

    def write_reference(key, value, lens, starts):
        for r, x in ((rk, key), (rv, value)):
            x = x.double().cpu().numpy()
            if q8:
                S.append_reference(r, x, tables, lens, starts)
            else:
                for s in range(B):
                    for i in range(starts[s + 1] - starts[s]):
                        pos = lens[s] - (starts[s + 1] - starts[s]) + i
                        r[tables[s, pos // bs], :, pos % bs] = x[starts[s] + i]

    starts = np.concatenate([[0], np.cumsum(first)])
    slots = dev(np.concatenate([tables[s, np.arange(n) // bs].astype(np.int64) * bs + np.arange(n) % bs for s, n in enumerate(first)]))
    key, value = (rows(rng, starts[-1], Hk, D, "bf16").to(DEV) for _ in "kv")
    write(key, value, dev(first.astype(np.int32)), dev(starts.astype(np.int32)))
    write_reference(key, value, first, starts)

    lens = dev(first.astype(np.int32))
    q = torch.zeros(B, Hk * G, D, dtype=t, device=DEV)
    nk, nv = torch.zeros(B, Hk, D, dtype=t, device=DEV), torch.zeros(B, Hk, D, dtype=t, device=DEV)
    sel = torch.zeros(B, Hk, K, dtype=torch.int32, device=DEV)
    out = torch.zeros(B, Hk * G, D, dtype=torch.float32, device=DEV)
    ws = torch.empty(max(1, pkv.paged_attention_list_workspace_bytes(B, Hk * G, Hk, D, bs, K, 32)), dtype=torch.uint8, device=DEV)

    def step():
        write(nk, nv, lens, None)
        pkv.select_blocks(sel, q, sums, bt, lens, bs, keep_first=1, keep_last=2, device_status=st)
        pkv.paged_attention_decode_selected(out, q, k, v, bt, lens, sel, D ** -0.5, k_scales=ks, v_scales=vs,
                                            partition_size=32, workspace=ws, device_status=st)

    graph, total = None, first.copy()
    for i in range(steps):
        total = total + 1
        size = 4.0 if i == 7 else 1.0
        lens.copy_(dev(total.astype(np.int32)))
        q.copy_(rows(rng, B, Hk * G, D, "bf16").to(DEV))
        nk.copy_(rows(rng, B, Hk, D, "bf16", size).to(DEV))
        nv.copy_(rows(rng, B, Hk, D, "bf16", size).to(DEV))
        if captured and i == 2:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        if graph is None:
            step()
        else:
            graph.replay()
        write_reference(nk, nv, total, np.arange(B + 1))
        real_k, real_v = (rk.real(), rv.real()) if q8 else (rk, rv)
        low, high = np.zeros((NB, Hk, D)), np.zeros((NB, Hk, D))
        for s in range(B):
            for j in range(-(-int(total[s]) // bs)):
                m = min(bs, int(total[s]) - j * bs)
                low[tables[s, j]], high[tables[s, j]] = real_k[tables[s, j], :, :m].min(1), real_k[tables[s, j], :, :m].max(1)
        qd = q.double().cpu().numpy()
        want = S.select_reference(qd, low, high, tables, total, bs, K, 1, 2)
        np.testing.assert_array_equal(sel.cpu().numpy(), want)
        ref, bound = S.attention_reference(qd, real_k, real_v, tables, total, bs, D ** -0.5,
                                           lambda s, h: want[s, h][want[s, h] >= 0])
        tol = S.attention_tolerance(ref, bound, real_v, total, D, torch.float32)
        assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    assert st.item() == 0
