"""Plain 64-bit forms of the 4-bit cache's operators, written from their
definitions (numpy, on the host), and cases for them."""
from __future__ import annotations

import numpy as np
import torch

from tests.q8_support import DT, make_tables

GROUP = 64


def rounded(x, t):
    """float64 numbers -> fp32 -> the 16-bit type t, as float64 (halves to even each time)."""
    return torch.from_numpy(np.asarray(x, np.float64).astype(np.float32)).to(t).double().numpy()


def quantize(x, t):
    """Rows [..., D] of numbers of type t (float64) -> codes uint8 [..., G, 64], scales and minima float64 [..., G]."""
    x = np.asarray(x, np.float64)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    f32 = lambda a: a.astype(np.float32).astype(np.float64)  # noqa: E731
    odd = ~np.isfinite(g).all(-1)
    g = np.where(odd[..., None], 0.0, g)
    low, high = g.min(-1), g.max(-1)
    s = rounded(f32(f32(high / 2 - low / 2) / 7.5), t)
    s = np.where(s < 2.0 ** -126, 0.0, s)
    with np.errstate(divide="ignore"):
        c = np.where(s > 0, f32(np.where(s > 0, 2.0, 0.0) / np.where(s > 0, s, 1.0)), 0.0)
    q = f32(g / 2 - low[..., None] / 2) * c[..., None]      # exact in 64 bits
    u = np.minimum(np.rint(np.rint(q * 65536) / 65536), 15).astype(np.uint8)
    return np.where(odd[..., None], 0, u), np.where(odd, np.nan, s), np.where(odd, np.nan, low)


def code_place(r, d, D):
    """(byte, shift) of the code of row r, dimension d in a record."""
    groups = D // 64
    j, i, n = d // 64, d % 64 // 8, d % 8
    at = r * (D // 2) + 4 * (groups * i + j) + n // 2
    line = at // 128
    x = line % 8 if D == 128 else (0, 4, 2, 6)[line % 4]
    return at ^ (16 * x), 4 * (n % 2)


def pair_place(r, j, D, bs):
    return bs * D // 2 + r * (D // 16) + 4 * j


def places(bs, D):
    both = np.array([[code_place(r, d, D) for d in range(D)] for r in range(bs)])
    return both[..., 0], both[..., 1]


def bits16(x, t):
    """Numbers that type t holds -> their 16-bit patterns."""
    return torch.from_numpy(np.asarray(x, np.float64)).to(t).view(torch.int16).numpy().view(np.uint16)


def pack(u, s, m, t):
    """Codes [..., bs, G, 64], scales and minima [..., bs, G] -> records uint8 [..., bs, D / 2 + D / 16]."""
    bs, groups = u.shape[-3], u.shape[-2]
    D = groups * GROUP
    byte, shift = places(bs, D)
    lead = u.shape[:-3]
    rec = np.zeros((*lead, bs * (D // 2 + D // 16)), np.uint8)
    flat = u.reshape(*lead, bs, D)
    for half in range(2):                                   # the codes in the low and in the high half of a byte
        r, d = np.nonzero(shift == 4 * half)
        rec[..., byte[r, d]] |= (flat[..., r, d] << (4 * half)).astype(np.uint8)
    for r in range(bs):
        for j in range(groups):
            at = pair_place(r, j, D, bs)
            for k, x in enumerate((s, m)):
                b = bits16(x[..., r, j], t)
                rec[..., at + 2 * k], rec[..., at + 2 * k + 1] = b & 255, b >> 8
    return rec.reshape(*lead, bs, D // 2 + D // 16)


def unpack(rec, t, D):
    """Records [..., bs, D / 2 + D / 16] -> codes [..., bs, G, 64], scales and minima [..., bs, G] float64."""
    rec = np.asarray(rec)
    bs = rec.shape[-2]
    flat = np.ascontiguousarray(rec).reshape(*rec.shape[:-2], -1)
    byte, shift = places(bs, D)
    u = (flat[..., byte] >> shift) & 15
    pairs = flat[..., bs * D // 2:]
    p = torch.from_numpy(np.ascontiguousarray(pairs)).view(t).double().numpy().reshape(*rec.shape[:-2], bs, D // 64, 2)
    return u.reshape(*u.shape[:-1], D // 64, 64), p[..., 0], p[..., 1]


def numbers(u, s, m):
    """s u + m in 64 bits (exact), [..., D]."""
    x = s[..., None] * u + m[..., None]
    return x.reshape(*x.shape[:-2], -1)


def q4_case(seed, *, t="bf16", B=4, G=4, Hk=2, D=128, bs=16, lens=(1, 17, 40, 100), garbage=True, size=1.0, offset=0.5):
    """A 4-bit cache of random codes, scales and minima; rows and blocks that no
    sequence reaches have NaN scales and minima and random codes."""
    rng = np.random.RandomState(seed)
    lens = np.asarray(lens, np.int32)
    tables, NB = make_tables(rng, [-(-int(n) // bs) for n in lens])
    dt = DT[t]
    out = dict(q=torch.from_numpy(rng.randn(len(lens), Hk * G, D)).to(dt), tables=tables, lens=lens, NB=NB, Hk=Hk, G=G, D=D,
               bs=bs, t=t, scale=float(np.float32(D ** -0.5)), B=len(lens))
    live = np.zeros((NB, bs), bool)
    for s, L in enumerate(lens):
        for i in range(int(L)):
            live[tables[s, i // bs], i % bs] = True
    for n in "kv":
        u = rng.randint(0, 16, (NB, Hk, bs, D // 64, 64)).astype(np.uint8)
        s = rounded(size * np.exp(rng.uniform(-3, -1, (NB, Hk, bs, D // 64))), dt)
        m = rounded(-7.5 * s + offset * size * rng.randn(NB, Hk, bs, D // 64), dt)
        if garbage:
            s, m = (np.where(live[:, None, :, None], a, np.nan) for a in (s, m))
        out[n + "_parts"] = (u, s, m)
        out[n] = pack(u, s, m, dt)
    return out


def attention_reference(c, k=None, v=None):
    """softmax attention in 64 bits over the case's cache -> out [B, H, D], per
    row the bounds that attention_tolerance needs: of a score's terms, and of a
    value's."""
    (uk, sk, mk), (uv, sv, mv) = (c[n + "_parts"] for n in "kv")
    k, v = numbers(uk, sk, mk), numbers(uv, sv, mv)
    q = c["q"].double().numpy()
    B, H, D = q.shape
    G, bs = c["G"], c["bs"]
    out, score, value = np.zeros((B, H, D)), np.zeros((B, H)), np.zeros((B, H))
    for b in range(B):
        L = int(c["lens"][b])
        if not L:
            continue
        blocks = c["tables"][b, : -(-L // bs)]
        rows = lambda a, h: a[blocks, h].reshape(-1, *a.shape[3:])[:L]  # noqa: E731
        for h in range(c["Hk"]):
            qq = q[b, h * G:(h + 1) * G]
            z = c["scale"] * (qq @ rows(k, h).T)
            p = np.exp(z - z.max(-1, keepdims=True))
            out[b, h * G:(h + 1) * G] = (p / p.sum(-1, keepdims=True)) @ rows(v, h)
            # the largest sum of a score's terms (codes up to 15, minima), and of a value's
            qa = np.abs(qq).reshape(G, -1, 64).sum(-1)
            score[b, h * G:(h + 1) * G] = abs(c["scale"]) * (qa @ (15 * rows(sk, h) + np.abs(rows(mk, h))).T).max(-1)
            value[b, h * G:(h + 1) * G] = (15 * rows(sv, h) + np.abs(rows(mv, h))).max()
    return out, score, value


def attention_tolerance(c, ref, score, value, out_dtype):
    """How far a kernel's row may be from the 64-bit one, element by element.

    A score is a sum of D products in fp32, of codes and of minima, in any
    order: D + 8 additions, on tensor cores cut instead of rounded (2^-23 each),
    so it is off by ds <= (D + 8) 2^-23 of its terms' sum; q brought to f16 by a
    power of two is off by at most 2^-35 of its head's largest, which times D
    terms is below one of those steps.  Every weight is then off by a factor
    within e^(2 ds), and by 2^-20 for the exponential, the division and the two
    f16 parts in which it enters the product with the codes (2^-22, and 2^-32 of
    the largest weight for each token, which L 2^-23 covers).  The sums over L
    tokens are cut at most L + 16 times, each time by 2^-23 of what has been
    summed: at most sum_i w_i (15 s + |m|), where codes and minima are summed
    apart.  A 16-bit output adds half a step of its own."""
    L = np.asarray(c["lens"], float)[:, None]
    rel = np.expm1(2 * (c["D"] + 8) * 2.0 ** -23 * score) + 2.0 ** -20 + (L + 16) * 2.0 ** -23
    tol = np.broadcast_to((rel * value)[..., None], ref.shape)
    if out_dtype != torch.float32:
        tiny = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}[out_dtype]
        tol = tol + (np.abs(ref) + tol) * torch.finfo(out_dtype).eps / 2 + tiny
    return tol
