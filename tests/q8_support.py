"""Plain 64-bit forms of the 8-bit cache's and the block selection's operators,
written from their definitions (numpy, on the host), and cases for them."""
from __future__ import annotations

import numpy as np
import torch

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def e4m3_table() -> np.ndarray:
    """Value of each of the 256 bit patterns: 1 sign, 4 exponent (bias 7), 3
    mantissa bits; all exponent and mantissa bits set is NaN."""
    bits = np.arange(256)
    e, m = (bits >> 3) & 15, bits & 7
    x = np.where(e > 0, (8 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9.0)
    x[(bits & 127) == 127] = np.nan
    return np.where(bits >= 128, -x, x)


TABLE = e4m3_table()


def decode(bits: np.ndarray) -> np.ndarray:
    return TABLE[bits]


def nearest(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value, halves to even; |x| <= 448 or NaN."""
    a = np.abs(x)
    with np.errstate(invalid="ignore"):
        e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6.0)
    step = 2.0 ** (e - 3.0)
    return np.copysign(np.rint(a / step) * step, x)


def needed_scale(amax: np.ndarray) -> np.ndarray:
    """Smallest power of two 2^e, e >= -126, with amax <= 448 * 2^e (checked,
    not computed by a logarithm's rounding)."""
    e = np.full(amax.shape, -126.0)
    big = amax > 448.0 * 2.0 ** -126.0
    g = np.floor(np.log2(np.where(big, amax, 1.0) / 448.0)) - 1
    for _ in range(3):
        g = np.where(amax > 448.0 * 2.0 ** g, g + 1, g)
    assert np.all(~big | ((amax <= 448.0 * 2.0 ** g) & (amax > 448.0 * 2.0 ** (g - 1))))
    return 2.0 ** np.where(big, np.maximum(g, -126.0), e)


def same_values(bits: np.ndarray, want: np.ndarray) -> bool:
    """Stored bytes stand for `want` (NaN where it is NaN)."""
    return bool(np.array_equal(decode(bits), want, equal_nan=True))


class Q8Cache:
    """Values (float64) and scales of one K or V cache."""

    def __init__(self, NB, Hk, bs, D):
        self.v = np.zeros((NB, Hk, bs, D))
        self.s = np.zeros((NB, Hk))

    def append(self, rows, block, row0):
        """rows [n, Hk, D] float64 to rows row0.. of `block`."""
        x = np.where(np.isinf(rows), np.nan, rows)
        amax = np.nanmax(np.where(np.isnan(x), 0.0, np.abs(x)), axis=(0, 2))
        s = needed_scale(amax)
        if row0:
            s = np.maximum(s, self.s[block])
            self.v[block, :, :row0] = nearest(self.v[block, :, :row0] * (self.s[block] / s)[:, None, None])
        self.s[block] = s
        self.v[block, :, row0:row0 + len(rows)] = nearest(x / s[None, :, None]).transpose(1, 0, 2)

    def real(self):
        return self.v * self.s[:, :, None, None]


def touched(total, new, bs):
    """(logical block, first row, end row, first new token) of each block that a sequence's new tokens touch."""
    lo, hi = total - new, total
    return [(j, max(lo, j * bs) - j * bs, min(hi, (j + 1) * bs) - j * bs, max(lo, j * bs) - lo)
            for j in range(lo // bs, -(-hi // bs))] if new > 0 else []


def append_reference(cache, x, tables, total, starts):
    bs = cache.v.shape[2]
    for s in range(len(total)):
        n = starts[s + 1] - starts[s]
        for j, a, b, t in touched(int(total[s]), int(n), bs):
            cache.append(x[starts[s] + t: starts[s] + t + b - a], tables[s, j], a)


def make_tables(rng, need, NB=None):
    """Block tables for sequences of need[s] blocks, placed by a permutation -> (tables, NB)."""
    NB = NB or int(sum(need)) + 5
    order = rng.permutation(NB)
    tables = np.full((len(need), max(1, max(need))), -1, np.int32)
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = order[at:at + n]
        at += n
    return tables, NB


def q8_case(seed, *, qdtype="bf16", B=4, G=4, Hk=2, D=128, bs=16, lens=(1, 17, 40, 100), spread=2.0, garbage=True):
    """A quantised cache of random bytes of every block and random power-of-two
    scales; rows and blocks that no sequence reaches hold NaN patterns and NaN scales."""
    rng = np.random.RandomState(seed)
    lens = np.asarray(lens, np.int32)
    need = [-(-int(n) // bs) for n in lens]
    tables, NB = make_tables(rng, need)
    q = torch.from_numpy(rng.randn(len(lens), Hk * G, D)).to(DT[qdtype])
    out = dict(q=q, tables=tables, lens=lens, NB=NB, Hk=Hk, G=G, D=D, bs=bs, scale=float(np.float32(D ** -0.5)), B=len(lens))
    S = -(-Hk // 4) * 4
    for n in "kv":
        x = rng.randn(NB, Hk, bs, D)
        e = np.floor(rng.uniform(-spread, spread, (NB, Hk)))
        scale = 2.0 ** (e - 7)
        # the nearest table value, by comparison with every value
        vals = nearest(np.clip(x * 60.0, -448, 448))
        pos = {v: b for b, v in enumerate(TABLE) if not np.isnan(v)}
        keys = np.array(sorted(pos))
        bits = np.array([pos[k] for k in keys], np.uint8)[np.searchsorted(keys, vals)]
        live = np.zeros((NB, bs), bool)
        for s, L in enumerate(lens):
            for i in range(int(L)):
                live[tables[s, i // bs], i % bs] = True
        if garbage:
            bits[~live.any(1)] = 0xFF
            bits = np.where(live[:, None, :, None], bits, 0x7F).astype(np.uint8)
            scale[~live.any(1)] = np.nan
        sc = np.full((NB, S), np.nan, np.float32)
        sc[:, :Hk] = scale
        out[n + "_bits"], out[n + "_scale"] = bits, sc
    return out


def attention_reference(q, k, v, tables, lens, bs, scale, listed=None):
    """softmax attention in 64 bits.  q [B, H, D] float64; k, v [NB, Hk, bs, D]
    float64; listed(s, h) -> logical blocks (None: all).  -> out, and for each
    row the bound max_i |scale| sum_d |q_d k_id|."""
    B, H, D = q.shape
    Hk = k.shape[1]
    G = H // Hk
    out, bound = np.zeros((B, H, D)), np.zeros((B, H))
    for s in range(B):
        L = int(lens[s])
        for h in range(Hk):
            blocks = np.arange(-(-L // bs)) if listed is None else np.asarray(listed(s, h), int)
            if L == 0 or blocks.size == 0:
                continue
            pos = (blocks[:, None] * bs + np.arange(bs)).reshape(-1)
            kk = k[tables[s, blocks], h].reshape(-1, D)[pos < L]
            vv = v[tables[s, blocks], h].reshape(-1, D)[pos < L]
            qq = q[s, h * G:(h + 1) * G]
            z = scale * (qq @ kk.T)
            p = np.exp(z - z.max(-1, keepdims=True))
            out[s, h * G:(h + 1) * G] = (p / p.sum(-1, keepdims=True)) @ vv
            bound[s, h * G:(h + 1) * G] = (abs(scale) * (np.abs(qq) @ np.abs(kk).T)).max(-1)
    return out, bound


def attention_tolerance(ref, bound, v, lens, D, out_dtype):
    """How far a kernel's row may be from the 64-bit one, element by element.

    A score is a sum of D products in fp32 (any order, D + 4 roundings with the
    scales), so it is off by ds <= (D + 4) 2^-24 * bound; every weight is then
    off by a factor within e^(2 ds), by 2^-20 for the exponential, its split
    into two 16-bit parts and the division, and the sums over L tokens round L
    times: each relative to sum_i w_i |v_i| <= max |v|.  A 16-bit output adds
    half a step of its own, and where it is bfloat16 the weights may be held
    in 11 bits (half a step 2^-11)."""
    L = np.asarray(lens, float)[:, None]
    rel = np.expm1(2 * (D + 4) * 2.0 ** -24 * bound) + 2.0 ** -20 + (L + 8) * 2.0 ** -24
    if out_dtype == torch.bfloat16:
        rel = rel + 2.0 ** -11
    vmax = np.nanmax(np.abs(v)) if v.size else 0.0
    tol = rel[..., None] * vmax
    if out_dtype != torch.float32:
        tiny = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}[out_dtype]
        tol = tol + (np.abs(ref) + tol) * torch.finfo(out_dtype).eps / 2 + tiny
    return tol


def select_reference(q, low, high, tables, lens, bs, K, first, last):
    """Blocks by the definition, in 64 bits; low, high [NB, Hk, D] float64."""
    B, H, D = q.shape
    Hk = low.shape[1]
    G = H // Hk
    out = np.full((B, Hk, K), -1, np.int32)
    for s in range(B):
        n = -(-int(lens[s]) // bs)
        if n <= K:
            out[s, :, :n] = np.arange(n)
            continue
        for h in range(Hk):
            qq = q[s, h * G:(h + 1) * G]
            up, down = np.maximum(qq, 0).sum(0), np.maximum(-qq, 0).sum(0)
            with np.errstate(invalid="ignore"):
                z = high[tables[s, :n], h] @ up - low[tables[s, :n], h] @ down
            z = np.where(np.isnan(z), np.inf, z)
            j = np.arange(n)
            keep = (j < first) | (j >= n - last)
            rest = j[~keep]
            best = rest[np.lexsort((rest, -z[rest]))][: K - keep.sum()]
            out[s, h] = np.sort(np.concatenate([j[keep], best]))
    return out
