"""What is measured of the 8-bit cache and of the attention over selected blocks: cases, inputs, plain forms.

Five operators, reached through the package's Python entry points:

  append_cache_q8                  new tokens' K and V into a cache of e4m3 values with one power-of-two scale
                                   for each block of tokens and kv head
  paged_attention_decode_q8        single-query attention over such a cache
  summarize_blocks                 per block and kv head, the smallest and largest value of each key dimension
  select_blocks                    for each sequence and kv head, the blocks with the highest upper bound on
                                   the scores of the head's query group, bounded through those summaries
  paged_attention_decode_selected  single-query attention over the selected blocks, of either kind of cache

``own`` false: the plain forms, elementary torch operations.  ``own`` true: the package's calls.
"""
import math

import numpy as np
import torch

own = False

WORKSPACE = 96 << 20     # bytes of scratch a serving program keeps for all its layers
E4M3_MAX = 448.0
MIN_EXP = -126           # the scale of a block that holds only zeros is 2^-126

# ------------------------------------------------------------------ cases


def _case(op, dtype, seqs, heads, kv_heads, dim, block, lo, hi, **more):
    return dict(op=op, dtype=dtype, seqs=seqs, heads=heads, kv_heads=kv_heads, dim=dim, block=block,
                lo=lo, hi=hi, **more)


def listed():
    return [
        # one running request at the start of a chat: latency of a single small call
        dict(_case("decode_q8", "bf16", 1, 32, 8, 128, 16, 700, 700), name="q8 decode, one request"),
        # a batch of 64 requests, 32 heads without sharing, contexts of 128 to 2048 tokens
        dict(_case("decode_q8", "f16", 64, 32, 32, 128, 16, 128, 2048), name="q8 decode, batch of 64"),
        # 16 long contexts of 16K to 32K tokens, 64 query heads on 8 kv heads
        dict(_case("decode_q8", "bf16", 16, 64, 8, 128, 16, 16384, 32768), name="q8 decode, long contexts"),
        # a decode step's new tokens, one per request, of a batch of 256
        dict(_case("append", "bf16", 256, 32, 8, 128, 16, 1, 256, new_lo=1, new_hi=1), name="q8 append, decode step"),
        # prompts of 1K to 2K tokens written after their prefill
        dict(_case("append", "f16", 8, 40, 40, 128, 16, 0, 0, new_lo=1024, new_hi=2048), name="q8 append, prompts"),
        # the summaries of the blocks that a decode step of 256 requests wrote into
        dict(_case("summarize", "bf16", 256, 32, 8, 128, 16, 1, 256, new_lo=1, new_hi=1, q8=False),
             name="summaries, decode step"),
        # the summaries of prompts of 4K to 16K tokens, from the 8-bit cache
        dict(_case("summarize", "bf16", 16, 64, 8, 128, 16, 0, 0, new_lo=4096, new_hi=16384, q8=True),
             name="summaries, prompts in q8"),
        # four requests of 2K to 8K tokens, 64 blocks each
        dict(_case("select", "f16", 4, 32, 8, 128, 16, 2048, 8192, pick=64, first=1, last=2),
             name="select, four requests"),
        # long contexts: 128 blocks (2048 tokens) of 16K to 32K tokens
        dict(_case("select", "bf16", 16, 64, 8, 128, 16, 16384, 32768, pick=128, first=1, last=4),
             name="select, long contexts"),
        # one request with 64 selected blocks of a 16-bit cache
        dict(_case("selected", "f16", 1, 32, 8, 128, 16, 8192, 8192, pick=64, q8=False),
             name="selected, one request"),
        # long contexts: 128 blocks of a 16-bit cache for each of 32 sequences and 8 kv heads
        dict(_case("selected", "bf16", 32, 64, 8, 128, 16, 4096, 16384, pick=128, q8=False),
             name="selected, batch of 32"),
        # the same over the 8-bit cache, blocks of 32 tokens
        dict(_case("selected", "bf16", 32, 64, 8, 128, 32, 4096, 16384, pick=64, q8=True),
             name="selected in q8, batch of 32"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


#: what the largest listed case of each operator holds: cached values (tokens x kv heads x dim) at most
_MOST = {"decode_q8": 16 * 32768 * 8 * 128, "append": 8 * 2048 * 40 * 128, "summarize": 16 * 16384 * 8 * 128,
         "select": 16 * 32768 * 8 * 128, "selected": 32 * 16384 * 8 * 128}


def draw(rng):
    op = rng.choice(["decode_q8", "append", "summarize", "select", "selected"])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    kv = rng.choice([1, 2, 4, 5, 8, 10, 16, 32])
    dim = rng.choice([64, 128])
    block = rng.choice([8, 16, 32])
    dtype = rng.choice(["f16", "bf16"])
    seqs = _spread(rng, 1, 200)
    most = max(16, min(32768, _MOST[op] // (seqs * kv * dim)))
    more = {}
    if op in ("append", "summarize"):
        if rng.random() < 0.5:
            more = dict(new_lo=1, new_hi=1)
            lo, hi = 0, _spread(rng, 1, min(most, 400))
        else:
            new_hi = _spread(rng, 2, max(2, most // 2))
            more = dict(new_lo=rng.choice([0, 1, max(1, new_hi // 3)]), new_hi=new_hi)
            lo, hi = 0, rng.choice([0, min(most // 2, _spread(rng, 1, 100))])
    else:
        hi = _spread(rng, 1, most)
        lo = rng.choice([hi, max(1, hi // 2), max(1, hi // 8), 1])
    if op == "selected":
        more["pick"] = _spread(rng, 4, 300)
    if op == "select":                                      # more blocks than are picked: else there is nothing to select
        hi = max(hi, 32 * block)
        lo = max(lo, hi // 2)
        more.update(pick=_spread(rng, 4, max(4, hi // (4 * block))), first=rng.choice([0, 1]), last=rng.choice([1, 2, 3]))
    if op in ("summarize", "selected"):
        more["q8"] = rng.random() < 0.5
    return _case(op, dtype, seqs, group * kv, kv, dim, block, lo, hi, **more)


# ----------------------------------------------------------------- inputs

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def _exponent(amax):
    """The smallest e, at least MIN_EXP, with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax)                                # amax = m * 2^e, m in [0.5, 1)
    e = torch.where(m <= 0.875, e - 9, e - 8)               # 448 = 0.875 * 2^9
    return torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp_min(MIN_EXP)


def _power(e):
    """2^e in float32, for whole e in [-126, 127]."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


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


def _pad4(n):
    return -(-n // 4) * 4


def _to_q8(x):
    """A cache of e4m3 values and its scales, float32 [blocks, kv heads rounded up to 4]."""
    e = _exponent(x.abs().amax((2, 3)))
    scales = torch.zeros(x.shape[0], _pad4(x.shape[1]), device=x.device)
    scales[:, : x.shape[1]] = _power(e)
    return x.mul_(_power(-e)[:, :, None, None]).to(torch.float8_e4m3fn), scales


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    host = np.random.RandomState(int(seed) % (1 << 31))
    B, H, Hk, D, bs = c["seqs"], c["heads"], c["kv_heads"], c["dim"], c["block"]
    t = _TYPES[c["dtype"]]
    lens = host.randint(c["lo"], c["hi"] + 1, B)
    new = host.randint(c["new_lo"], c["new_hi"] + 1, B) if "new_hi" in c else np.zeros(B, np.int64)
    total = lens + new
    need = -(-total // bs)
    NB = int(need.sum()) + 1 + int(need.sum()) // 16
    if "new_hi" in c:                                       # the pool itself is an output: the same size for every seed
        NB = B * -(-(c["hi"] + c["new_hi"]) // bs) + 1
    MB = int(max(need.max(), 1))
    order = host.permutation(NB)
    tables = np.full((B, MB), -1, np.int32)
    at = 0
    for s in range(B):
        tables[s, : need[s]] = order[at: at + need[s]]
        at += need[s]
    s = dict(op=c["op"], B=B, H=H, Hk=Hk, D=D, bs=bs, G=H // Hk, t=t,
             block_tables=torch.from_numpy(tables).to(dev),
             context_lens=torch.from_numpy(total.astype(np.int32)).to(dev),
             max_len=int(total.max()), max_new=int(new.max()), MB=MB, NB=NB, scale=1.0 / math.sqrt(D),
             spare=int(order[at]), host_new=new)
    if c["op"] in ("append", "summarize"):
        starts = np.concatenate([[0], np.cumsum(new)])
        s["query_start"] = None if c["new_lo"] == c["new_hi"] == 1 else torch.from_numpy(starts.astype(np.int32)).to(dev)
        T = s["num_tokens"] = int(starts[-1])
        token_seq = np.repeat(np.arange(B), new)
        token_pos = (total - new)[token_seq] + np.arange(T) - starts[:-1][token_seq]
        s["token_seq"] = torch.from_numpy(token_seq).to(dev)
        s["token_pos"] = torch.from_numpy(token_pos).to(dev)
    if c["op"] == "append":
        s["k_cache"], s["k_scales"] = _to_q8(_keys(gen, NB, Hk, bs, D))
        s["v_cache"], s["v_scales"] = _to_q8(_values(gen, NB, Hk, bs, D))
        s["key"] = _keys(gen, T, Hk, 1, D)[:, :, 0].to(t).contiguous()
        s["value"] = _values(gen, T, Hk, 1, D)[:, :, 0].to(t).contiguous()
        return s
    if c["op"] in ("decode_q8", "select", "selected"):
        s["q"] = torch.randn(B, H, D, generator=gen, device=dev).to(t)
        s["workspace"] = torch.empty(WORKSPACE, dtype=torch.uint8, device=dev)
    if c["op"] == "select":
        k = _keys(gen, NB, Hk, bs, D).to(t)
        s["summaries"] = torch.stack([k.amin(2), k.amax(2)], 2).contiguous()
        s["selected"] = torch.zeros(B, Hk, c["pick"], dtype=torch.int32, device=dev)
        s["first"], s["last"] = c["first"], c["last"]
        return s
    if c["op"] == "decode_q8" or c["q8"]:
        s["k_cache"], s["k_scales"] = _to_q8(_keys(gen, NB, Hk, bs, D))
        if c["op"] != "summarize":
            s["v_cache"], s["v_scales"] = _to_q8(_values(gen, NB, Hk, bs, D))
    else:
        s["k_cache"], s["k_scales"] = _keys(gen, NB, Hk, bs, D).to(t), None
        if c["op"] != "summarize":
            s["v_cache"], s["v_scales"] = _values(gen, NB, Hk, bs, D).to(t), None
    if c["op"] == "summarize":
        s["summaries"] = torch.zeros(NB, Hk, 2, D, dtype=torch.bfloat16 if c["q8"] else t, device=dev)
        return s
    s["out"] = torch.empty(B, H, D, dtype=t, device=dev)
    if c["op"] == "selected":
        # random blocks of each sequence and kv head, the last one always among them, in ascending order
        n = torch.from_numpy(need).to(dev)
        j = torch.arange(MB, device=dev)
        order = torch.rand(B, Hk, MB, generator=gen, device=dev)
        order = torch.where(j == (n - 1)[:, None, None], -1.0, order)
        order = torch.where(j < n[:, None, None], order, 2.0)
        pick = torch.full((B, Hk, c["pick"]), MB, device=dev)
        top = order.argsort(-1)[..., : c["pick"]]
        pick[..., : top.shape[-1]] = torch.where(order.gather(-1, top) < 1.5, top, MB)
        pick = pick.sort(-1).values
        s["selected"] = torch.where(pick < MB, pick, -1).to(torch.int32)
    return s


# ------------------------------------------------------------ plain forms


def _softmax_sum(scores, v):
    """softmax over the last axis of scores [..., G, N], its row of a fully masked one zero, times v [..., N, D]."""
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isinf(m), 0.0, m))
    den = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(den > 0, den, 1.0)


def _rows(cache, scales, phys, heads):
    """Rows of `cache` as float32: blocks phys [...] at kv heads `heads` (same shape) -> [..., bs, D]."""
    if scales is None:
        return cache[phys, heads].float()
    return cache.view(torch.uint8)[phys, heads].view(torch.float8_e4m3fn).float() * scales[phys, heads][..., None, None]


def _attend(s, logical):
    """Attention over the logical blocks [B, Hk, N] (-1: none)."""
    B, Hk, G, D, bs = s["B"], s["Hk"], s["G"], s["D"], s["bs"]
    N = logical.shape[-1]
    heads = torch.arange(Hk, device=logical.device)[None, :, None].expand(B, Hk, N)
    phys = s["block_tables"].long().clamp_min(0)[:, None].expand(B, Hk, -1).gather(-1, logical.long().clamp_min(0))
    pos = logical.long()[..., None] * bs + torch.arange(bs, device=logical.device)
    live = (logical[..., None] >= 0) & (pos < s["context_lens"].long()[:, None, None, None])
    live = live.reshape(B, Hk, 1, N * bs)
    k = _rows(s["k_cache"], s["k_scales"], phys, heads).reshape(B, Hk, N * bs, D)
    scores = torch.matmul(s["q"].float().reshape(B, Hk, G, D), k.transpose(-1, -2)) * s["scale"]
    del k
    scores = torch.where(live, scores, float("-inf"))
    v = _rows(s["v_cache"], s["v_scales"], phys, heads).reshape(B, Hk, N * bs, D)
    return _softmax_sum(scores, v).reshape(B, Hk * G, D).to(s["t"])


def _touched(s):
    """The blocks that hold new tokens: logical ids [B, N], where one is (bool), and the first new token's position [B]."""
    bs, dev = s["bs"], s["context_lens"].device
    total = s["context_lens"].long()
    new = torch.ones_like(total) if s["query_start"] is None else (s["query_start"][1:] - s["query_start"][:-1]).long()
    start = total - new
    j = start[:, None] // bs + torch.arange((s["max_new"] + bs - 2) // bs + 1, device=dev)
    return j, (j * bs < total[:, None]) & (new > 0)[:, None], start


def _append_one(s, cache, scales, x):
    """The new rows x [T, Hk, D] in the cache's blocks, each block's scale raised to what they need."""
    bs, Hk, NB = s["bs"], s["Hk"], s["NB"]
    tables = s["block_tables"].long()
    cache = cache.view(torch.uint8)
    j, there, start = _touched(s)
    kept = torch.where(there[:, 0], start % bs, 0)          # rows that a sequence's first touched block holds already
    first = torch.where(kept > 0, tables.gather(1, (start // bs).clamp_max(s["MB"] - 1)[:, None])[:, 0], s["spare"])
    block = tables[s["token_seq"], s["token_pos"] // bs]
    amax = torch.zeros(NB, Hk, device=x.device).scatter_reduce_(0, block[:, None].expand(-1, Hk), x.abs().amax(-1), "amax")
    hit = torch.zeros(NB, dtype=torch.bool, device=x.device).index_fill_(0, block, True)
    grown = torch.zeros(NB, dtype=torch.bool, device=x.device).index_fill_(0, first, True)
    old, fresh = scales[:, :Hk], _power(_exponent(amax))
    new = torch.where(hit[:, None], torch.where(grown[:, None], torch.maximum(old, fresh), fresh), old)
    held = cache[first]
    ratio = (old[first] / new[first])[:, :, None, None]
    again = (held.view(torch.float8_e4m3fn).float() * ratio).to(torch.float8_e4m3fn).view(torch.uint8)
    rescaled = (torch.arange(bs, device=x.device) < kept[:, None])[:, None, :, None] & (ratio < 1)
    cache[first] = torch.where(rescaled, again, held)
    cache[block, :, s["token_pos"] % bs] = (x / new[block][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    scales[:, :Hk] = new


def _append(s):
    _append_one(s, s["k_cache"], s["k_scales"], s["key"].float())
    _append_one(s, s["v_cache"], s["v_scales"], s["value"].float())
    return {n: s[n] for n in ("k_cache", "v_cache", "k_scales", "v_scales")}


def _summarize(s):
    bs, Hk = s["bs"], s["Hk"]
    j, there, _ = _touched(s)
    phys = torch.where(there, s["block_tables"].long().gather(1, j.clamp_max(s["MB"] - 1)), s["spare"])
    heads = torch.arange(Hk, device=phys.device)
    rows = _rows(s["k_cache"], s["k_scales"], phys[..., None].expand(-1, -1, Hk), heads.expand(*phys.shape, Hk))
    pos = j[..., None] * bs + torch.arange(bs, device=phys.device)
    live = (pos < s["context_lens"].long()[:, None, None])[:, :, None, :, None]
    low = torch.where(live, rows, float("inf")).amin(-2)
    high = torch.where(live, rows, float("-inf")).amax(-2)
    both = torch.stack([low, high], -2).to(s["summaries"].dtype)
    # every sequence without a j-th touched block writes the spare block, which keeps what it holds
    s["summaries"][phys] = torch.where(there[..., None, None, None], both, s["summaries"][s["spare"]])
    return s["summaries"]


def _select(s):
    B, Hk, G, D, K = s["B"], s["Hk"], s["G"], s["D"], s["selected"].shape[-1]
    phys = s["block_tables"].long().clamp_min(0)
    q = s["q"].double().reshape(B, Hk, G, D)
    up, down = q.clamp_min(0).sum(2), (-q).clamp_min(0).sum(2)
    # per block: the sum over the group's heads of the largest score that its keys' ranges allow; in 64 bits,
    # because two blocks' scores may lie closer together than 32 bits tell
    low, high = s["summaries"][phys].unbind(-2)             # [B, N, Hk, D]
    score = (high.double() * up[:, None]).sum(-1) - (low.double() * down[:, None]).sum(-1)
    n = (s["context_lens"].long() + s["bs"] - 1) // s["bs"]
    j = torch.arange(phys.shape[1], device=phys.device)
    always = (j < s["first"]) | (j >= (n - s["last"])[:, None])
    there = (j < n[:, None])[..., None]
    score = torch.where(there, torch.where(always[..., None], float("inf"), score), float("-inf")).transpose(1, 2)
    best = score.sort(dim=-1, descending=True, stable=True).indices[..., :K]
    best = torch.where(best < n[:, None, None], best, phys.shape[1]).sort(-1).values
    s["selected"].fill_(-1)
    s["selected"][..., : best.shape[-1]] = torch.where(best < phys.shape[1], best, -1).to(torch.int32)
    return s["selected"]


def run(s):
    op = s["op"]
    if own:
        import paged_kv_cache_311_gb300 as pkv
        if op == "decode_q8":
            return pkv.paged_attention_decode_q8(s["out"], s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"],
                                                 s["block_tables"], s["context_lens"], s["scale"],
                                                 max_context_len=s["max_len"], workspace=s["workspace"])
        if op == "append":
            pkv.append_cache_q8(s["key"], s["value"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"],
                                s["block_tables"], s["context_lens"], s["query_start"])
            return {n: s[n] for n in ("k_cache", "v_cache", "k_scales", "v_scales")}
        if op == "summarize":
            return pkv.summarize_blocks(s["k_cache"], s["summaries"], s["block_tables"], s["context_lens"],
                                        s["query_start"], num_tokens=s["num_tokens"], k_scales=s["k_scales"])
        if op == "select":
            return pkv.select_blocks(s["selected"], s["q"], s["summaries"], s["block_tables"], s["context_lens"], s["bs"],
                                     keep_first=s["first"], keep_last=s["last"], max_context_len=s["max_len"])
        return pkv.paged_attention_decode_selected(s["out"], s["q"], s["k_cache"], s["v_cache"], s["block_tables"],
                                                   s["context_lens"], s["selected"], s["scale"], k_scales=s["k_scales"],
                                                   v_scales=s["v_scales"], workspace=s["workspace"])
    if op == "decode_q8":
        j = torch.arange(s["MB"], device=s["q"].device)
        n = (s["context_lens"] + s["bs"] - 1) // s["bs"]
        return _attend(s, torch.where(j < n[:, None], j, -1)[:, None].expand(-1, s["Hk"], -1))
    if op == "selected":
        return _attend(s, s["selected"])
    return {"append": _append, "summarize": _summarize, "select": _select}[op](s)


# ------------------------------------------------------------ work, and the values in 64 bits


def work(case):
    c = case
    B, H, Hk, D, bs = c["seqs"], c["heads"], c["kv_heads"], c["dim"], c["block"]
    held = B * (c["lo"] + c["hi"]) / 2
    if c["op"] == "decode_q8":
        return {"bytes": held * Hk * (2 * D + 8 / bs) + 4 * B * H * D + 4 * held / bs, "flops": 4 * held * H * D}
    if c["op"] == "selected":
        one = 1 if c["q8"] else 2
        mean = (c["lo"] + c["hi"]) / 2
        read = B * min(mean, c["pick"] * bs) * Hk
        return {"bytes": read * (2 * D * one + 8 / bs) + 4 * B * H * D, "flops": 4 * read * (H // Hk) * D}
    if c["op"] == "select":
        blocks = held / bs * Hk
        return {"bytes": blocks * 4 * D + 2 * B * H * D + 4 * B * Hk * c["pick"] + 4 * held / bs, "flops": blocks * 4 * D}
    new = B * (c["new_lo"] + c["new_hi"]) / 2
    blocks = new / bs + B * (1 if c["new_hi"] > 1 else 1 - 1 / bs)
    if c["op"] == "append":
        return {"bytes": new * Hk * D * 2 * 3 + 16 * blocks * Hk, "flops": 6 * new * Hk * D}
    # summaries: the rows of the touched blocks that hold a token, read once; two rows written for each block
    rows = new + B * min(c["hi"], bs) / 2
    return {"bytes": rows * Hk * D * (1 if c["q8"] else 2) + blocks * Hk * D * 4, "flops": 2 * rows * Hk * D}


def _nearest_e4m3(x):
    """x [...] float64, rounded to the nearest e4m3 value (halves to even, at most 448), as float64."""
    a = np.abs(x)
    e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6.0)
    step = np.exp2(e - 3.0)
    return np.sign(x) * np.minimum(np.rint(a / step) * step, 448.0)


def _exact_append(s):
    """Block by block on the host: which rows a block holds, the largest magnitude, the power of two that it needs."""
    tables, total = s["block_tables"].cpu().numpy(), s["context_lens"].cpu().numpy()
    new, bs, Hk = s["host_new"], s["bs"], s["Hk"]
    starts = np.concatenate([[0], np.cumsum(new)])
    got = {}
    for name, x in (("k", s["key"]), ("v", s["value"])):
        cache = s[name + "_cache"].float().cpu().numpy()
        scales = s[name + "_scales"].cpu().numpy().astype(np.float64)
        x = x.double().cpu().numpy()
        for q in range(s["B"]):
            lo, hi = int(total[q] - new[q]), int(total[q])
            for j in range(lo // bs, -(-hi // bs) if hi > lo else 0):
                a, b, blk = max(lo, j * bs), min(hi, (j + 1) * bs), tables[q, j]
                rows = x[starts[q] + a - lo: starts[q] + b - lo]                 # [n, Hk, D]
                big = np.abs(rows).max((0, 2))
                scale = np.exp2(np.maximum(np.ceil(np.log2(np.where(big > 0, big, 1e-300) / 448.0)), -126.0))
                held = a - j * bs
                if held:
                    scale = np.maximum(scale, scales[blk, :Hk])
                    cache[blk, :, :held] = _nearest_e4m3(cache[blk, :, :held].astype(np.float64) * (scales[blk, :Hk] / scale)[:, None, None])
                scales[blk, :Hk] = scale
                cache[blk, :, held: held + b - a] = _nearest_e4m3(rows / scale[None, :, None]).transpose(1, 0, 2)
        got[name + "_cache"], got[name + "_scales"] = cache, scales
    return got


def _e4m3_values():
    """The value of each e4m3 bit pattern: sign, 4 bits of exponent (bias 7), 3 of mantissa."""
    bits = np.arange(256)
    mag, e = bits & 7, (bits >> 3) & 15
    x = np.where(e > 0, (8 + mag) * np.exp2(e - 10.0), mag * np.exp2(-9.0)) * np.where(bits >= 128, -1.0, 1.0)
    return torch.from_numpy(x).cuda()


def _exact_rows(s, name, phys, h, e4m3):
    if s[name + "_scales"] is None:
        return s[name + "_cache"][phys, h].double()
    return e4m3[s[name + "_cache"].view(torch.uint8)[phys, h].long()] * s[name + "_scales"][phys, h].double()[:, None, None]


def _exact_attention(s, heads_blocks):
    """One sequence and kv head after another; heads_blocks(b, h) -> logical block ids (int64, on the GPU)."""
    B, Hk, G, D, bs = s["B"], s["Hk"], s["G"], s["D"], s["bs"]
    out, e4m3 = torch.zeros(B, Hk, G, D, dtype=torch.float64, device="cuda"), _e4m3_values()
    for b in range(B):
        L = int(s["context_lens"][b])
        for h in range(Hk if L else 0):
            blocks = heads_blocks(b, h, -(-L // bs))
            phys = s["block_tables"][b].long()[blocks]
            pos = (blocks[:, None] * bs + torch.arange(bs, device="cuda")).reshape(-1)
            k, v = (_exact_rows(s, n, phys, h, e4m3).reshape(-1, D)[pos < L] for n in ("k", "v"))
            z = s["q"][b, h * G: (h + 1) * G].double() @ k.T * s["scale"]
            out[b, h] = torch.softmax(z, -1) @ v
    return out.reshape(B, Hk * G, D)


def _exact_summaries(s):
    got = s["summaries"].double().cpu().numpy()
    tables, total = s["block_tables"].cpu().numpy(), s["context_lens"].cpu().numpy()
    k = s["k_cache"].float().cpu().numpy()
    scales = None if s["k_scales"] is None else s["k_scales"].cpu().numpy()
    for b in range(s["B"]):
        lo, hi = int(total[b] - s["host_new"][b]), int(total[b])
        for j in range(lo // s["bs"], -(-hi // s["bs"]) if hi > lo else 0):
            blk = tables[b, j]
            rows = k[blk, :, : min(s["bs"], hi - j * s["bs"])].astype(np.float64)
            if scales is not None:
                rows = rows * scales[blk, : s["Hk"], None, None]
            got[blk, :, 0], got[blk, :, 1] = rows.min(1), rows.max(1)
    return got


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "append":
        return _exact_append(s)
    if s["op"] == "summarize":
        return _exact_summaries(s)
    if s["op"] == "select":
        return None       # whole numbers: the plain form is computed in 64 bits
    if s["op"] == "decode_q8":
        return _exact_attention(s, lambda b, h, n: torch.arange(n, device="cuda"))
    picked = s["selected"].long()
    return _exact_attention(s, lambda b, h, n: picked[b, h][picked[b, h] >= 0])
