"""What is measured of the 4-bit cache: cases, inputs, plain forms.

Three operators, reached through the package's Python entry points:

  reshape_and_cache_q4       new tokens' K and V into a cache of 4-bit codes, each group of 64 dimensions of a
                             row with a scale and a minimum of its own
  gather_cache_q4            rows of such a cache back as numbers
  paged_attention_decode_q4  single-query attention over such a cache

A write is measured together with the reading back of what it wrote, which gives its result as numbers.

``own`` false: the plain forms, elementary torch operations.  ``own`` true: the package's calls.
"""
import math

import numpy as np
import torch

own = False

WORKSPACE = 96 << 20     # bytes of scratch a serving program keeps for all its layers
GROUP = 64               # dimensions that share a scale and a minimum

# ------------------------------------------------------------------ cases


def _case(op, dtype, seqs, heads, kv_heads, dim, block, lo, hi):
    return dict(op=op, dtype=dtype, seqs=seqs, heads=heads, kv_heads=kv_heads, dim=dim, block=block, lo=lo, hi=hi)


def listed():
    return [
        # one running request at the start of a chat: latency of a single small call
        dict(_case("decode", "bf16", 1, 32, 8, 128, 16, 700, 700), name="decode, one request"),
        # a batch of 64 requests, 32 heads without sharing, contexts of 128 to 2048 tokens
        dict(_case("decode", "f16", 64, 32, 32, 128, 16, 128, 2048), name="decode, batch of 64"),
        # 16 long contexts of 16K to 32K tokens, 64 query heads on 8 kv heads
        dict(_case("decode", "bf16", 16, 64, 8, 128, 16, 16384, 32768), name="decode, long contexts"),
        # one request over a long document: all parallelism comes from its context
        dict(_case("decode", "bf16", 1, 32, 8, 128, 32, 131071, 131071), name="decode, one long context"),
        # heads of 64, three query heads to a kv head, contexts of any length from one token on
        dict(_case("decode", "f16", 33, 24, 8, 64, 8, 1, 4095), name="decode, heads of 64"),
        # one request's token of a decode step
        dict(_case("write", "bf16", 1, 8, 8, 128, 16, 1, 1), name="write and read, one token"),
        # a decode step's tokens, one per request, of a batch of 256
        dict(_case("write", "bf16", 256, 8, 8, 128, 16, 1, 1), name="write and read, decode step"),
        # prompts of 1K to 2K tokens written after their prefill
        dict(_case("write", "f16", 8, 40, 40, 128, 16, 1024, 2048), name="write and read, prompts"),
        # ragged prompts, heads of 64, an odd number of them
        dict(_case("write", "bf16", 19, 5, 5, 64, 8, 1, 1500), name="write and read, heads of 64"),
        # the cached prefix that one new prompt starts with
        dict(_case("read", "bf16", 1, 8, 8, 128, 16, 1000, 1000), name="read, one prefix"),
        # cached prefixes of 4K to 16K tokens for 16 prompts' prefill
        dict(_case("read", "bf16", 16, 8, 8, 128, 16, 4096, 16384), name="read, prefixes"),
        # ragged prefixes, heads of 64, blocks of 32
        dict(_case("read", "f16", 7, 5, 5, 64, 32, 1, 6001), name="read, heads of 64"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


#: what the largest listed case of each operator holds: cached values (tokens x kv heads x dim) at most
_MOST = {"decode": 16 * 32768 * 8 * 128, "write": 8 * 2048 * 40 * 128, "read": 16 * 16384 * 8 * 128}


def draw(rng):
    op = rng.choice(["decode", "decode", "write", "read"])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8]) if op == "decode" else 1
    kv = rng.choice([1, 2, 4, 5, 8, 10, 16, 32, 40])
    dim = rng.choice([64, 128])
    block = rng.choice([8, 16, 32])
    dtype = rng.choice(["f16", "bf16"])
    seqs = _spread(rng, 1, 256)
    most = max(16, min(131072, _MOST[op] // (seqs * kv * dim)))
    hi = 1 if op == "write" and rng.random() < 0.4 else _spread(rng, 1, most)
    lo = rng.choice([hi, max(1, hi // 2), max(1, hi // 8), 1])
    return _case(op, dtype, seqs, group * kv, kv, dim, block, lo, hi)


# ----------------------------------------------------------------- inputs

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def _keys(gen, nb, hk, bs, d):
    """Keys as a cache holds them: channels of different sizes, neighbours alike."""
    dev = gen.device
    x = torch.randn(nb, hk, bs, d, generator=gen, device=dev).mul_(0.8)
    x += 0.6 * torch.randn(nb, hk, 1, d, generator=gen, device=dev)
    return x.mul_(torch.exp(0.5 * torch.randn(1, hk, 1, d, generator=gen, device=dev)))


def _values(gen, nb, hk, bs, d):
    dev = gen.device
    size = torch.exp(0.5 * torch.randn(nb, hk, 1, 1, generator=gen, device=dev))
    return torch.randn(nb, hk, bs, d, generator=gen, device=dev).mul_(size)


def _places(bs, D, dev):
    """Where a block's record of one kv head holds row r, dimension d: (byte, shift of the nibble), [bs, D] each;
    and the 16-bit words of each row's groups' scales and minima, [bs, D / 64, 2].

    A row is D / 8 words of eight codes: word (D / 64) i + j holds dimensions 64 j + 8 i .. + 7, the lowest in the
    lowest bits.  Rows fill lines of 128 bytes one after another, and the 16-byte pieces of a line are exchanged:
    piece p of line n is stored at p ^ x(n), x = n % 8 for rows of 64 bytes, 0, 4, 2, 6 for n % 4 = 0 .. 3 for rows
    of 32.  Behind the codes come the rows' (scale, minimum) pairs, a pair for each group.
    """
    r, d = torch.arange(bs, device=dev)[:, None], torch.arange(D, device=dev)[None]
    groups = D // GROUP
    at = r * (D // 2) + ((d % GROUP) // 8 * groups + d // GROUP) * 4 + (d % 8) // 2
    line = at // 128
    x = line % 8 if groups == 2 else torch.tensor([0, 4, 2, 6], device=dev)[line % 4]
    return at ^ (x * 16), (d % 2) * 4, (bs * D // 4 + torch.arange(bs * groups * 2, device=dev)).reshape(bs, groups, 2)


def _quantize(x):
    """Rows x [..., D] of a 16-bit type -> codes uint8 [..., D / 64, 64], scales and minima of that type [..., D / 64]."""
    g = x.float().reshape(*x.shape[:-1], -1, GROUP)
    low, high = g.amin(-1), g.amax(-1)
    s = ((high * 0.5 - low * 0.5) / 7.5).to(x.dtype).float()
    s = torch.where(s < 2.0 ** -126, 0.0, s)
    c = torch.where(s > 0, 2.0 / s, 0.0)
    half = g * 0.5 - (low * 0.5)[..., None]
    # in 64 bits, where the product is exact; taken to 16 binary places first, so that a quotient halfway between
    # two codes is seen as one although c is rounded: those are common among 16-bit numbers, and go to the even code
    u = ((half.double() * c.double()[..., None] * 65536.0).round() / 65536.0).round().clamp_max(15.0).to(torch.uint8)
    return u, s.to(x.dtype), low.to(x.dtype)


def _records(x):
    """Blocks x [NB, Hk, bs, D] of a 16-bit type -> their records, uint8 [NB, Hk, bs, D / 2 + D / 16]."""
    NB, Hk, bs, D = x.shape
    byte, shift, words = _places(bs, D, x.device)
    u, s, m = _quantize(x)
    u = u.reshape(NB, Hk, bs, D)
    rec = torch.zeros(NB, Hk, bs * (D // 2 + D // 16), dtype=torch.uint8, device=x.device)
    rec[..., byte[:, 0::2].reshape(-1)] = (u[..., 0::2] | (u[..., 1::2] << 4)).reshape(NB, Hk, -1)
    rec.view(x.dtype)[..., words.reshape(-1)] = torch.stack([s, m], -1).reshape(NB, Hk, -1)
    return rec.reshape(NB, Hk, bs, D // 2 + D // 16)


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    host = np.random.RandomState(int(seed) % (1 << 31))
    B, H, Hk, D, bs = c["seqs"], c["heads"], c["kv_heads"], c["dim"], c["block"]
    t = _TYPES[c["dtype"]]
    # where a row comes out for each token, their number is the same for every seed
    lens = (host if c["op"] == "decode" else np.random.RandomState(B)).randint(c["lo"], c["hi"] + 1, B)
    need = -(-lens // bs)
    NB = int(need.sum()) + 1 + int(need.sum()) // 16
    MB = int(need.max())
    order = host.permutation(NB)
    tables = np.full((B, MB), -1, np.int32)
    at = 0
    for i in range(B):
        tables[i, : need[i]] = order[at: at + need[i]]
        at += need[i]
    s = dict(op=c["op"], B=B, H=H, Hk=Hk, D=D, bs=bs, G=H // Hk, t=t, NB=NB, MB=MB, scale=1.0 / math.sqrt(D),
             block_tables=torch.from_numpy(tables).to(dev), context_lens=torch.from_numpy(lens.astype(np.int32)).to(dev),
             max_len=int(lens.max()), places=_places(bs, D, dev))
    if c["op"] != "decode":
        seq = np.repeat(np.arange(B), lens)
        pos = np.arange(len(seq)) - (np.cumsum(lens) - lens)[seq]
        s["slots"] = torch.from_numpy(tables[seq, pos // bs].astype(np.int64) * bs + pos % bs).to(dev)
        T = s["T"] = len(seq)
        s["out_key"], s["out_value"] = (torch.empty(T, Hk, D, dtype=t, device=dev) for _ in "kv")
    if c["op"] == "write":
        s["k_cache"], s["v_cache"] = (torch.zeros(NB, Hk, bs, D // 2 + D // 16, dtype=torch.uint8, device=dev) for _ in "kv")
        s["key"] = _keys(gen, T, Hk, 1, D)[:, :, 0].to(t).contiguous()
        s["value"] = _values(gen, T, Hk, 1, D)[:, :, 0].to(t).contiguous()
        return s
    s["k_cache"] = _records(_keys(gen, NB, Hk, bs, D).to(t))
    s["v_cache"] = _records(_values(gen, NB, Hk, bs, D).to(t))
    if c["op"] == "decode":
        s["q"] = torch.randn(B, H, D, generator=gen, device=dev).to(t)
        s["out"] = torch.empty(B, H, D, dtype=t, device=dev)
        s["workspace"] = torch.empty(WORKSPACE, dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------ plain forms


def _numbers(rec, places, t):
    """Records [..., bs, D / 2 + D / 16] -> the rows' numbers in 32 bits, [..., bs, D]."""
    byte, shift, words = places
    bs, D = byte.shape
    rec = rec.flatten(-2)
    u = ((rec[..., byte.reshape(-1)] >> shift.expand(bs, D).reshape(-1)) & 15).float().unflatten(-1, (bs, D // GROUP, GROUP))
    pairs = rec.view(t)[..., words.reshape(-1)].float().unflatten(-1, (bs, D // GROUP, 2, 1))
    return (u * pairs[..., 0, :] + pairs[..., 1, :]).flatten(-2)


def _decode(s):
    B, Hk, G, D, bs = s["B"], s["Hk"], s["G"], s["D"], s["bs"]
    phys = s["block_tables"].long().clamp_min(0)
    live = torch.arange(s["MB"] * bs, device=phys.device) < s["context_lens"].long()[:, None]
    rows = lambda name: _numbers(s[name][phys].transpose(1, 2), s["places"], s["t"]).reshape(B, Hk, -1, D)  # noqa: E731
    scores = torch.matmul(s["q"].float().reshape(B, Hk, G, D), rows("k_cache").transpose(-1, -2)) * s["scale"]
    scores = torch.where(live[:, None, None], scores, float("-inf"))
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    v = torch.where(live[:, None, :, None], rows("v_cache"), 0.0)
    return (torch.matmul(p, v) / p.sum(-1, keepdim=True)).reshape(B, Hk * G, D).to(s["t"])


def _write_one(s, cache, x):
    """Codes, scales and minima of the rows x [T, Hk, D] to their slots."""
    Hk, bs, D, NB = s["Hk"], s["bs"], s["D"], s["NB"]
    byte, _, words = s["places"]
    u, scale, low = _quantize(x)
    u = u.flatten(-2)
    block, row = (s["slots"] // bs)[:, None, None], s["slots"] % bs
    heads = torch.arange(Hk, device=x.device)[None, :, None]
    cache.view(NB, Hk, -1)[block, heads, byte[row, 0::2][:, None]] = u[..., 0::2] | (u[..., 1::2] << 4)
    cache.view(s["t"]).view(NB, Hk, -1)[block, heads, words[row].flatten(1)[:, None]] = torch.stack([scale, low], -1).flatten(-2)


def _read_one(s, cache, out):
    """The rows at the slots as numbers of the cache's type."""
    Hk, bs, D, NB = s["Hk"], s["bs"], s["D"], s["NB"]
    byte, _, words = s["places"]
    block, row = (s["slots"] // bs)[:, None, None], s["slots"] % bs
    heads = torch.arange(Hk, device=out.device)[None, :, None]
    two = cache.view(NB, Hk, -1)[block, heads, byte[row, 0::2][:, None]]
    u = torch.stack([two & 15, two >> 4], -1).flatten(-2).float().unflatten(-1, (D // GROUP, GROUP))
    pair = cache.view(s["t"]).view(NB, Hk, -1)[block, heads, words[row].flatten(1)[:, None]].float().unflatten(-1, (D // GROUP, 2, 1))
    out.copy_((u * pair[..., 0, :] + pair[..., 1, :]).flatten(-2))


def run(s):
    if own:
        import paged_kv_cache_311_gb300 as pkv
        if s["op"] == "decode":
            return pkv.paged_attention_decode_q4(s["out"], s["q"], s["k_cache"], s["v_cache"], s["block_tables"],
                                                 s["context_lens"], s["scale"], max_context_len=s["max_len"],
                                                 workspace=s["workspace"])
        if s["op"] == "write":
            pkv.reshape_and_cache_q4(s["key"], s["value"], s["k_cache"], s["v_cache"], s["slots"])
        pkv.gather_cache_q4(s["out_key"], s["out_value"], s["k_cache"], s["v_cache"], s["slots"])
        return {"key": s["out_key"], "value": s["out_value"]}
    if s["op"] == "decode":
        return _decode(s)
    if s["op"] == "write":
        _write_one(s, s["k_cache"], s["key"])
        _write_one(s, s["v_cache"], s["value"])
    _read_one(s, s["k_cache"], s["out_key"])
    _read_one(s, s["v_cache"], s["out_value"])
    return {"key": s["out_key"], "value": s["out_value"]}


# ------------------------------------------------------------ work, and the values in 64 bits


def work(case):
    c = case
    B, H, Hk, D, bs = c["seqs"], c["heads"], c["kv_heads"], c["dim"], c["block"]
    tokens = B * (c["lo"] + c["hi"]) / 2
    held = D // 2 + D // 16                                  # bytes of a row in the cache
    if c["op"] == "decode":
        return {"bytes": 2 * tokens * Hk * held + 4 * B * H * D + 4 * tokens / bs, "flops": 4 * tokens * H * D}
    if c["op"] == "write":                                   # rows in, records and the rows' numbers out
        return {"bytes": 2 * tokens * Hk * (4 * D + held) + 8 * tokens, "flops": 14 * tokens * Hk * D}
    return {"bytes": 2 * tokens * Hk * (2 * D + held) + 8 * tokens, "flops": 4 * tokens * Hk * D}


def _exact_codes(rec, bs, D, t):
    """Records [n, bs * (D / 2 + D / 16)], word by word -> the rows' numbers [n, bs, D] in 64 bits."""
    groups, out = D // 64, torch.empty(len(rec), bs, D, dtype=torch.float64, device=rec.device)
    words = rec[:, : bs * D // 2].contiguous().view(torch.int32)
    pairs = rec[:, bs * D // 2:].contiguous().view(t).double().reshape(len(rec), bs, groups, 2)
    for r in range(bs):
        for i in range(8):
            for j in range(groups):
                w = r * (D // 8) + groups * i + j            # the word, before pieces are exchanged
                line, piece = w // 32, w // 4 % 8
                piece ^= line % 8 if groups == 2 else (0, 4, 2, 6)[line % 4]
                word = words[:, line * 32 + piece * 4 + w % 4, None]
                codes = (word >> torch.arange(0, 32, 4, device=rec.device)) & 15
                out[:, r, 64 * j + 8 * i: 64 * j + 8 * i + 8] = codes.double() * pairs[:, r, j, :1] + pairs[:, r, j, 1:]
    return out


def _exact_row(x):
    """What rows x [..., D] of a 16-bit type become, by the definition in real numbers."""
    t, g = x.dtype, x.double().unflatten(-1, (-1, 64))
    low, span = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True) - g.amin(-1, keepdim=True)
    s = (span / 15).to(t).double()
    u = torch.where(s > 0, ((g - low) / torch.where(s > 0, s, 1.0)).round().clamp(0, 15), 0.0)
    return (s * u + low).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    B, Hk, G, D, bs, t = s["B"], s["Hk"], s["G"], s["D"], s["bs"], s["t"]
    if s["op"] == "write":
        return {"key": _exact_row(s["key"]), "value": _exact_row(s["value"])}
    numbers = {n: _exact_codes(s[n].flatten(0, 1).flatten(1), bs, D, t).reshape(s["NB"], Hk, bs, D) for n in ("k_cache", "v_cache")}
    tables = s["block_tables"].long()
    if s["op"] == "read":
        block, row = s["slots"] // bs, s["slots"] % bs
        return {"key": numbers["k_cache"][block, :, row], "value": numbers["v_cache"][block, :, row]}
    out = torch.zeros(B, Hk, G, D, dtype=torch.float64, device="cuda")
    for b in range(B):
        L = int(s["context_lens"][b])
        phys = tables[b, : -(-L // bs)]
        for h in range(Hk):
            k, v = (numbers[n][phys, h].reshape(-1, D)[:L] for n in ("k_cache", "v_cache"))
            z = s["q"][b, h * G: (h + 1) * G].double() @ k.T * s["scale"]
            out[b, h] = torch.softmax(z, -1) @ v
    return out.reshape(B, Hk * G, D)
