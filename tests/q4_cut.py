"""How paged_attention_decode_q4 divides its work, restated on the host: the
shares of the line of all rows' units, and the chunks in which a CTA looks up
the blocks of its share.  And rows in which every piece tells: values of a
level of their own in each stretch of tokens, so that an output without one of
them is another."""
from __future__ import annotations

import torch

UNIT, ROW_COST, CHUNK, WARPS, CTAS = 32, 8, 128, 4, 3


def shares(lens, kv_heads: int, count: int):
    """[(sequence, head, first unit, units)] of each of `count` CTAs: the line is cut by cost, a row (a sequence's kv
    head) costing its units and ROW_COST in front of them; units of later rows follow those of the first."""
    rows = [(s, h, -(-n // UNIT)) for s, n in enumerate(lens) for h in range(kv_heads) if n > 0]
    total = sum(n + ROW_COST for _, _, n in rows)
    ends = [total * i // count for i in range(count + 1)]
    place, at, k = [], 0, 0                                 # of each end: row, unit in it
    for e in ends:
        while k < len(rows) and e >= at + rows[k][2] + ROW_COST:
            at += rows[k][2] + ROW_COST
            k += 1
        place.append((k, max(0, e - at - ROW_COST) if k < len(rows) else 0))
    first = [0]
    for _, _, n in rows:
        first.append(first[-1] + n)
    out = []
    for (k, u), (k1, u1) in zip(place, place[1:]):
        left = first[k1] + u1 - first[k] - u
        out.append((*rows[k][:2], u, left) if k < len(rows) else (0, 0, 0, 0))
    return out, rows


def chunks(share, rows):
    """A share's chunks, each a list of pieces (sequence, head, first unit, units), and how each ended: "" at CHUNK units
    or the share's end, "row" in front of a row that would leave too few units to the next chunk, "four" with WARPS units
    of a row left for the next."""
    s, h, u, left = share
    if left == 0:
        return []
    k = next(i for i, r in enumerate(rows) if r[:2] == (s, h))
    out = []
    while left:
        size, at, pieces, how = min(left, CHUNK), 0, [], ""
        kk, uu = k, u
        while at < size:
            n = min(rows[kk][2] - uu, size - at)
            if at + n == size:
                rest = min(rows[kk][2] - uu - n, left - size)
                if 0 < rest < WARPS:
                    if at > 0:
                        size, how = at, "row"
                        break
                    size, how, n = size - WARPS, "four", n - WARPS
            pieces.append((*rows[kk][:2], uu, n))
            at += n
            uu += n
            if uu == rows[kk][2]:
                kk, uu = kk + 1, 0
        out.append((pieces, how))
        k, u, left = kk, uu, left - size
    return out


def all_chunks(lens, kv_heads: int, sms: int):
    """[chunks of each share] of a streamed call."""
    cut, rows = shares(lens, kv_heads, CTAS * sms)
    return [chunks(c, rows) for c in cut]


class Rows:
    """Sequences on the GPU whose K and V went through reshape_and_cache_q4: keys that make scores of a few units, values
    of a level of its own for each `stretch` tokens and dimension.  Queries have eight dimensions of 1/8, so a score's
    terms add up to no more than a key's largest number."""

    def __init__(self, pkv, seed, lens, *, dtype, Hk, G, D, bs, stretch=UNIT):
        dev = "cuda"
        self.pkv, self.lens, self.Hk, self.G, self.D, self.bs, self.dtype = pkv, list(lens), Hk, G, D, bs, dtype
        g = torch.Generator(device=dev).manual_seed(seed)
        need = [-(-n // bs) for n in lens]
        order = torch.randperm(sum(need) + 2, generator=g, device=dev).to(torch.int32)
        self.NB, MB = sum(need) + 2, max(need)
        self.tables = torch.full((len(need), MB), -1, dtype=torch.int32, device=dev)
        at = 0
        for s, n in enumerate(need):
            self.tables[s, :n] = order[at: at + n]
            at += n
        self.context = torch.tensor(self.lens, dtype=torch.int32, device=dev)
        self.q = torch.zeros(len(need), Hk * G, D, dtype=dtype, device=dev)
        for h in range(Hk * G):                             # another eight dimensions for each head
            d = torch.randperm(D, generator=g, device=dev)[:8]
            self.q[:, h, d] = torch.where(torch.rand(8, generator=g, device=dev) < 0.5, -0.125, 0.125).to(dtype)
        self.k, self.v = (pkv.q4_cache(self.NB, Hk, bs, D, dev) for _ in "kv")
        self.rows, self.size, self.most = [], [], []        # numbers as the cache has them; 15 s + |m| of V; the most of K
        for s, n in enumerate(self.lens):
            if n == 0:
                self.rows.append(None)
                self.size.append(None)
                self.most.append(0.0)
                continue
            key = 0.7 * torch.randn(n, Hk, D, generator=g, device=dev) + 0.4 * torch.randn(n, Hk, 1, generator=g, device=dev)
            level = torch.rand(-(-n // stretch), Hk, D, generator=g, device=dev) + 1.0
            value = level.repeat_interleave(stretch, 0)[:n] + 0.2 * torch.randn(n, Hk, D, generator=g, device=dev)
            pos = torch.arange(n, device=dev)
            slots = self.tables[s].long()[pos // bs] * bs + pos % bs
            key, value = key.to(dtype), value.to(dtype)
            pkv.reshape_and_cache_q4(key, value, self.k, self.v, slots)
            back = [torch.empty(n, Hk, D, device=dev) for _ in "kv"]
            pkv.gather_cache_q4(*back, self.k, self.v, slots, dtype=dtype)
            self.rows.append(back)
            groups = [x.float().unflatten(-1, (-1, 64)) for x in (key, value)]
            # a scale is a fifteenth of the range, rounded to 2^-8 of itself at most
            low, span = zip(*((x.amin(-1), (x.amax(-1) - x.amin(-1)) * (1 + 2.0 ** -8)) for x in groups))
            self.most.append(float((span[0] + low[0].abs()).max()))
            self.size.append((span[1] + low[1].abs()).amax(0).repeat_interleave(64, -1))   # [Hk, D]

    def decode(self, most=None, P=0, tables=None):
        out = torch.full(self.q.shape, float("nan"), device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        t = self.tables if tables is None else tables
        if most:
            t = torch.nn.functional.pad(t, (0, max(0, -(-most // self.bs) - t.shape[1])), value=-1)
        self.pkv.paged_attention_decode_q4(out, self.q, self.k, self.v, t, self.context, 1.0, max_context_len=most or max(self.lens),
                                           partition_size=P, device_status=st)
        return out.view(len(self.lens), self.Hk, self.G, self.D), int(st.item())

    def sums(self, s):
        """Sequence s in 64 bits, unit by unit: sums of weights [Hk, G, units] and of values [Hk, G, units, D]."""
        k, v = (x.double().transpose(0, 1) for x in self.rows[s])
        z = torch.matmul(self.q[s].double().view(self.Hk, self.G, self.D), k.transpose(1, 2))
        p = torch.exp(z - z.amax(-1, keepdim=True))
        n = self.lens[s]
        pad = -n % UNIT
        p = torch.nn.functional.pad(p, (0, pad)).unflatten(-1, (-1, UNIT))
        v = torch.nn.functional.pad(v, (0, 0, 0, pad)).unflatten(1, (-1, UNIT))
        return p.sum(-1), torch.einsum("hgut,hutd->hgud", p, v)

    def tolerance(self, s, additions):
        """How far an fp32 output of sequence s may be: [Hk, 1, D].

        A score has eight products of codes, cut at 2^-23 of their sum (on tensor cores; sums of zeros are exact), the
        minima's product and the sums that join them: 24 such steps of no more than the key's most.  Each weight is then
        off by e^(2 ds), by 2^-20 for exponential, parts and division, and a sum (of numbers of one sign, or taken from
        either side by turns, where a part may be twice the value's size) by 2^-23 for each of `additions`, those that
        one lane makes of a row and those of the joins."""
        ds = 24 * 2.0 ** -23 * self.most[s]
        return ((2 * ds + 2.0 ** -20 + additions * 2.0 ** -23) * 2 * self.size[s].double())[:, None]
