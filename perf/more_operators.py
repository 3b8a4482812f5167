"""Rotary positions, the 8-bit key-value cache, the attention over it and eviction from it, as
they are measured.

  rope     queries and keys rotated by their positions (or gradients rotated back);
  append   K and V rows added to sequences in a paged cache of 8 bits, and read back;
  attn     softmax attention of the last tokens of each sequence over the cache;
  weigh    the same, adding each key's attention weight to a running sum;
  evict    the keys of largest weight (and the last ones) kept, copied to pages of their own.

Rotary positions: pair i of a row turns by position * w_i and is multiplied by a gain; pairs are
(i, i + rot / 2) or, interleaved, (2 i, 2 i + 1) of the first rot features; the others are copied.
w_i = base^(-2 i / rot), for long contexts changed by a factor f: "linear" w_i / f; "base" with the
base times f^(rot / (rot - 2)); "parts" w_i (g + (1 - g) / f), where g goes from 0 to 1 as the turns
of the pair over the trained length, trained * w_i / 2 pi, go from slow to fast, and the gain is
0.1 ln f + 1.

The cache: 16 positions of a sequence that share a block hold, for each head and for K and V, a
scale 2^e and codes in e4m3 of x / 2^e, ties to even.  e is the smallest with every |x| <= 448 * 2^e,
at least -100.  Rows added to a block that has earlier ones make e the larger of what was there and
what they need, and the earlier codes are rounded again at it.  Eviction gives a block the largest e
that its rows come with.

`own` chooses what `run` does: false, elementary torch operations in 32 bits; true, the calls a
user makes of the library.
"""
import math

import torch

own = False

BLOCK = 16
LOWEST = -100  # of e
BASE = 10000.0
FAST, SLOW = 32.0, 1.0
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def _rope(name, B, N, Hq, Hk, d, rot, dtype="bf16", interleaved=False, scaling="none", factor=1.0,
          trained=4096, back=False, pos0=0):
    return dict(name=name, op="rope", B=B, N=N, Hq=Hq, Hk=Hk, d=d, rot=rot, dtype=dtype,
                interleaved=interleaved, scaling=scaling, factor=factor, trained=trained,
                back=back, pos0=pos0)


def _append(name, B, N, H, d, page, old, dtype="bf16"):
    """old: tokens that each sequence has before."""
    return dict(name=name, op="append", B=B, N=N, H=H, d=d, page=page, dtype=dtype,
                old=",".join(str(n) for n in old))


def _attn(name, B, Nq, Hq, Hkv, d, page, lens, mask="causal", window=0, op="attn"):
    return dict(name=name, op=op, B=B, Nq=Nq, Hq=Hq, Hkv=Hkv, d=d, page=page,
                lens=",".join(str(n) for n in lens), mask=mask, window=window)


def _evict(name, B, Hkv, d, page, lens, keep, recent):
    return dict(name=name, op="evict", B=B, Hkv=Hkv, d=d, page=page, keep=keep, recent=recent,
                lens=",".join(str(n) for n in lens))


RAGGED = [8192, 1, 513, 4095, 7000, 64, 65, 1999, 3001, 8190, 12, 6144, 2500, 777, 5120, 128]


def listed():
    return [
        # a decode step of 16 sequences, shared key heads: latency
        _rope("rope_step_b16", 16, 1, 32, 8, 128, 128, pos0=4096),
        # fp32 rows of odd number, half of each head rotated, positions read far out
        _rope("rope_partial_f32", 3, 1001, 20, 20, 96, 48, "f32", False, "linear", 4.0, pos0=120000),
        # gradients of a long training sequence, interleaved pairs, scaled by parts
        _rope("rope_bwd_32k", 1, 32768, 32, 8, 128, 128, "bf16", True, "parts", 8.0, 4096, True),
        # a decode step of 32 sequences of 80 pseudo-heads: latency
        _append("append_step_b32", 32, 1, 80, 128, 64, [17 + 131 * i for i in range(32)]),
        # a whole prompt after its prefill
        _append("append_prompt_8k", 1, 8192, 80, 128, 64, [0]),
        # one sequence, short context: the smallest attention call
        _attn("decode_b1_777", 1, 1, 80, 80, 128, 64, [777]),
        # a ragged batch with shared key heads, 4 drafted tokens each, sequences just begun
        _attn("draft_gqa_b16", 16, 4, 32, 8, 128, 64, RAGGED),
        # one long context
        _attn("decode_long_131071", 1, 1, 80, 80, 128, 64, [131071]),
        # a ragged batch whose weights are summed for a later eviction
        _attn("weigh_gqa_b16", 16, 1, 32, 8, 128, 64, RAGGED, op="weigh"),
        # long contexts of unshared heads, weights summed
        _attn("weigh_b4_32k", 4, 1, 20, 20, 128, 64, [32768, 30004, 16384, 400], op="weigh"),
        # a small batch brought back to its budget
        _evict("evict_b4_1k", 4, 8, 128, 64, [1100, 1025, 1024, 1531], 1000, 64),
        # a long context cut to a quarter
        _evict("evict_32k", 1, 80, 128, 64, [32768], 8192, 512),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn", "weigh", "evict"])
    if op == "rope":
        d = rng.choice([32, 64, 80, 96, 128, 256])
        rot = rng.choice([d, d, d // 2, 2 * rng.randint(2, d // 2)])
        Hq, Hk = rng.choice([(80, 80), (32, 8), (20, 20), (8, 1), (4, 0), (7, 7)])
        T = _log(rng, 1, 32768 * 40 * 128 // ((Hq + Hk) * d))
        B = min(T, _log(rng, 1, 64))
        return dict(op=op, B=B, N=max(1, T // B), Hq=Hq, Hk=Hk, d=d, rot=rot,
                    dtype=rng.choice(["bf16", "bf16", "f32"] if T < 16000 else ["bf16"]),
                    interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "base", "parts"]),
                    factor=rng.choice([2.0, 4.0, 7.5, 32.0]), trained=rng.choice([2048, 4096, 8192]),
                    back=rng.random() < 0.4, pos0=rng.choice([0, rng.randrange(0, 1000000)]))
    d = rng.choice([32, 64, 96, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        H = rng.choice([1, 4, 8, 20, 80])
        T = _log(rng, 1, min(16384, 8192 * 80 * 128 // (H * d)))
        B = min(T, _log(rng, 1, 64))
        return dict(op=op, B=B, N=max(1, T // B), H=H, d=d, page=page,
                    dtype=rng.choice(["bf16", "bf16", "f32"]) if T < 5000 else "bf16",
                    old=",".join(str(rng.choice([0, rng.randrange(0, 5000)])) for _ in range(B)))
    if op == "evict":
        Hkv = rng.choice([80, 40, 20, 8, 8, 1])
        B = _log(rng, 1, 32)
        top = max(64, min(131072, 32768 * 80 * 128 // (B * Hkv * d)))
        cap = _log(rng, 40, top)
        lens = [rng.randint(max(1, cap // 4), cap) for _ in range(B)]
        keep = _log(rng, 16, max(16, min(cap, 8192)))
        return dict(op=op, B=B, Hkv=Hkv, d=d, page=page, lens=",".join(str(n) for n in lens),
                    keep=keep, recent=rng.choice([0, 1, keep // 4, keep]))
    Hkv, G = rng.choice([(80, 1), (40, 1), (20, 1), (8, 1), (8, 4), (8, 8), (4, 7), (2, 16), (1, 8)])
    B = _log(rng, 1, 64)
    Nq = rng.choice([1, 1, 1, 2, 4, 5, 8, 16])
    if op == "weigh":
        Nq = min(Nq, 64 // G)
    top = max(64, min(131072, 16384 * 80 * 128 // (B * Hkv * d * max(1, Nq * G // 32))))
    cap = _log(rng, 16, top)
    lens = [rng.randint(max(1, cap // 8), cap) for _ in range(B)]
    if B > 2 and rng.random() < 0.5:
        lens[rng.randrange(B)] = 0  # a slot of the batch that holds no sequence
    mask = rng.choice(["causal", "causal", "none", "window"])
    return dict(op=op, B=B, Nq=Nq, Hq=Hkv * G, Hkv=Hkv, d=d, page=page,
                lens=",".join(str(n) for n in lens), mask=mask,
                window=_log(rng, 1, 4096) if mask == "window" else 0)


# ------------------------------------------------------------------ inputs, from the seed alone
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 29)
    return g


def _normal(g, shape, dtype=torch.bfloat16, gain=None, mean=None):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    if gain is not None:
        x *= gain
    if mean is not None:
        x += mean
    return x.to(dtype)


def _kv(g, shape, dtype):
    """Keys with channels of unequal size and offset, as trained keys have; plain values."""
    H, d = shape[-2:]
    gain = torch.exp(0.5 * torch.randn((H, d), generator=g, device="cuda"))
    mean = 0.5 * torch.randn((H, d), generator=g, device="cuda")
    return _normal(g, shape, dtype, gain, mean), _normal(g, shape, dtype)


def _ints(text):
    return [int(n) for n in text.split(",")]


def _heads(c):
    return c["H"] if c["op"] == "append" else c["Hkv"]


def _tables(g, lens, page, spare=2):
    """A table of pages in any order for sequences of these lengths, how many pages there are,
    and the pages that no sequence has."""
    per = [-(-n // page) for n in lens]
    n_pages = sum(per) + spare
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((len(lens), max(1, max(per))), device="cuda", dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    return table, n_pages, order[at:]


def _slots_of(table, b, first, last, page):
    j = torch.arange(first, last, device="cuda")
    return table[b, j // page].long() * page + j % page


def _inputs(c, seed):
    g = _gen(seed)
    s = {}
    if c["op"] == "rope":
        B, N, d = c["B"], c["N"], c["d"]
        s["q"] = _normal(g, (B, N, c["Hq"], d), DT[c["dtype"]])
        s["k"] = _normal(g, (B, N, c["Hk"], d), DT[c["dtype"]]) if c["Hk"] else None
        start = c["pos0"] + 37 * torch.arange(B, device="cuda", dtype=torch.int32)
        s["pos"] = (start[:, None] + torch.arange(N, device="cuda", dtype=torch.int32)).contiguous()
        return s
    H, d, page = _heads(c), c["d"], c["page"]
    if c["op"] == "append":
        B, N, old = c["B"], c["N"], _ints(c["old"])
        s["table"], s["n_pages"], _ = _tables(g, [n + N for n in old], page)
        s["lens"] = torch.tensor([n + N for n in old], device="cuda", dtype=torch.int32)
        s["old_lens"] = torch.tensor(old, device="cuda", dtype=torch.int32)
        s["had"] = torch.tensor([n % BLOCK for n in old], device="cuda", dtype=torch.int32)
        k, v = _kv(g, (B, BLOCK - 1 + N, H, d), DT[c["dtype"]])
        # the rows that the first block of each sequence has already, the last had[b] of 15
        s["k0"], s["v0"] = k[:, :BLOCK - 1].contiguous(), v[:, :BLOCK - 1].contiguous()
        s["k"], s["v"] = k[:, BLOCK - 1:].contiguous(), v[:, BLOCK - 1:].contiguous()
        # read back: each block that has a new row, from its start
        first = [n - n % BLOCK for n in old]
        s["back"] = torch.cat([_slots_of(s["table"], b, first[b], old[b] + N, page)
                               for b in range(B)]).to(torch.int32).reshape(1, -1).contiguous()
        return s
    B, lens = c["B"], _ints(c["lens"])
    if c["op"] == "evict":
        kept = [min(n, c["keep"]) for n in lens]
        width = max(1, -(-max(kept) // page))
        s["table"], s["n_pages"], free = _tables(g, lens, page, B * width + 1)
        s["dest"] = free[:B * width].reshape(B, width).contiguous()
        # weights as attention leaves them: a few keys have most, some have none
        w = torch.exp(2.0 * torch.randn((B, H, s["table"].shape[1] * page), generator=g,
                                        device="cuda"))
        w *= torch.rand(w.shape, generator=g, device="cuda") < 0.9
        s["weights"] = w
        s["back"] = torch.cat([_slots_of(s["dest"], b, 0, n, page)
                               for b, n in enumerate(kept)]).to(torch.int32).reshape(1, -1)
    else:
        s["table"], s["n_pages"], _ = _tables(g, lens, page)
        s["q"] = _normal(g, (B, c["Nq"], c["Hq"], d))
        if c["op"] == "weigh":
            s["weights"] = torch.rand((B, H, s["table"].shape[1] * page), generator=g,
                                      device="cuda")
    s["lens"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
    s["k"], s["v"] = _kv(g, (1, sum(lens), H, d), torch.bfloat16)
    return s


# ------------------------------------------------------------------ plain forms, 32 bits
def _two(e):
    """2^e, as the bits of a float; below 2^-126 that (which leaves no code but 0)."""
    return ((e.clamp(min=-126).to(torch.int32) + 127) << 23).view(torch.float32)


def _need(x):
    """e that rows x [blocks, tokens, H, d] need, for each block and head."""
    f, k = torch.frexp(x.abs().amax((1, 3)))
    e = torch.where(f <= 0.875, k - 9, k - 8)
    return torch.where(f == 0.0, LOWEST, e).clamp(min=LOWEST).to(torch.int32)


def _code(x, e):
    """x / 2^e as the nearest codes, held as bytes; e broadcasts over [..., H]."""
    return (x * _two(-e).unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8)


def _decode(codes):
    return codes.view(torch.float8_e4m3fn).float()


class _Plain:
    """The cache in plain tensors: codes of each slot, e of each block."""

    def __init__(self, n_pages, page, H, d):
        rows = n_pages * page
        self.codes = [torch.zeros((rows, H, d), dtype=torch.uint8, device="cuda")
                      for _ in range(2)]
        self.e = [torch.full((rows // BLOCK, H), LOWEST, dtype=torch.int32, device="cuda")
                  for _ in range(2)]

    def values(self, which, slots):
        e = self.e[which][slots // BLOCK]
        return _decode(self.codes[which][slots]) * _two(e).unsqueeze(-1)

    def append(self, xs, slots, first):
        """Rows of one sequence, from position `first` on, go to these slots."""
        for which, x in enumerate(xs):
            codes, es = self.codes[which], self.e[which]
            at, pos, n = 0, first, x.shape[0]
            if pos % BLOCK:  # the block that is there already
                m = min(BLOCK - pos % BLOCK, n)
                self._grow(which, x[:m].float(), slots[:m], pos % BLOCK)
                at, pos = m, pos + m
            while at < n:  # whole blocks, and what is left
                m = min((n - at) // BLOCK * BLOCK or n - at, 16384)
                y = x[at:at + m].float()
                y = y.reshape(-1, min(m, BLOCK), *y.shape[1:])
                to = slots[at:at + m]
                e = _need(y)
                es[to.reshape(y.shape[0], -1)[:, 0] // BLOCK] = e
                codes[to] = _code(y, e[:, None]).reshape(m, *y.shape[2:])
                at += m

    def _grow(self, which, x, slots, had):
        codes, es = self.codes[which], self.e[which]
        blk = slots[:1] // BLOCK
        old = blk * BLOCK + torch.arange(had, device="cuda")
        before = es[blk]
        e = torch.maximum(before, _need(x[None]))
        codes[old] = _code(_decode(codes[old]), e - before)
        codes[slots] = _code(x, e)
        es[blk] = e

    def load(self, slots, dtype):
        flat = slots.reshape(-1).long()
        return [torch.cat([self.values(w, flat[a:a + 16384]).to(dtype)
                           for a in range(0, flat.numel(), 16384)])
                .reshape(*slots.shape, *self.codes[w].shape[1:]) for w in range(2)]


def _turns(c):
    """w_i, and the gain."""
    rot, f = c["rot"], c["factor"]
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    base, gain = BASE, 1.0
    if c["scaling"] == "base":
        base = BASE * f ** (rot / (rot - 2))
    w = base ** (-2.0 * i / rot)
    if c["scaling"] == "linear":
        w = w / f
    if c["scaling"] == "parts":
        g = ((c["trained"] * w / (2 * math.pi) - SLOW) / (FAST - SLOW)).clamp(0.0, 1.0)
        w = w * (g + (1.0 - g) / f)
        gain = 0.1 * math.log(f) + 1.0
    return w, gain


def _plain_rope(c, s):
    w, gain = _turns(c)
    a = s["pos"].double()[..., None, None] * w  # far positions: the angle in 64 bits
    cos, sin = (gain * torch.cos(a)).float(), (gain * torch.sin(a)).float()
    if c["back"]:
        sin = -sin
    rot, half = c["rot"], c["rot"] // 2
    out = []
    for x in (s["q"], s["k"]):
        if x is None:
            continue
        y = x.clone()
        lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if c["interleaved"] else \
            (slice(0, half), slice(half, rot))
        x0, x1 = x[..., lo].float(), x[..., hi].float()
        y[..., lo] = (x0 * cos - x1 * sin).to(x.dtype)
        y[..., hi] = (x1 * cos + x0 * sin).to(x.dtype)
        out.append(y)
    return out


def _visible(c, n, dev):
    """[Nq, n] truth values: which keys of a sequence of n each of its last Nq positions sees."""
    Nq = c["Nq"]
    j = torch.arange(n, device=dev)
    if c["mask"] == "none":
        return torch.ones((Nq, n), dtype=torch.bool, device=dev)
    i = n - Nq + torch.arange(Nq, device=dev)
    vis = j[None, :] <= i[:, None]
    if c["mask"] == "window":
        vis &= i[:, None] - j[None, :] < c["window"]
    return vis


def _plain_attn(c, s):
    B, Nq, Hq, Hkv, d, page = (c[n] for n in ("B", "Nq", "Hq", "Hkv", "d", "page"))
    G = Hq // Hkv
    o = torch.zeros((B, Nq, Hq, d), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, Hq, Nq), -math.inf, device="cuda")
    weights = s["weights"].clone() if c["op"] == "weigh" else None
    for b, n in enumerate(_ints(c["lens"])):
        lo = max(0, n - Nq + 1 - c["window"]) if c["mask"] == "window" else 0
        if n == 0:
            continue
        rows = _slots_of(s["table"], b, lo, n, page)
        k, v = s["cache"].values(0, rows), s["cache"].values(1, rows)
        q = s["q"][b].float().reshape(Nq, Hkv, G, d).permute(1, 2, 0, 3).reshape(Hkv, G * Nq, d)
        x = torch.matmul(q, k.permute(1, 2, 0)) * (1.0 / math.sqrt(d))
        vis = _visible(c, n, "cuda")[:, lo:].repeat(G, 1)
        x = torch.where(vis, x, -math.inf)
        m = x.amax(-1, keepdim=True)
        m = torch.where(m > -math.inf, m, 0.0)
        p = torch.exp(x - m)
        l = p.sum(-1, keepdim=True)
        p = p / torch.where(l > 0, l, 1.0)
        r = torch.matmul(p, v.permute(1, 0, 2))
        o[b] = r.reshape(Hkv, G, Nq, d).permute(2, 0, 1, 3).reshape(Nq, Hq, d).to(torch.bfloat16)
        lse[b] = (m + torch.log(l)).reshape(Hq, Nq)
        if weights is not None:
            weights[b, :, lo:n] += p.sum(1)
    return [o, lse] if weights is None else [o, lse, weights]


def _plain_evict(c, s):
    B, H, page, keep, recent = (c[n] for n in ("B", "Hkv", "page", "keep", "recent"))
    cache = s["cache"]
    kept = torch.full((B, H, keep), -1, dtype=torch.int32, device="cuda")
    weights = torch.zeros((B, H, s["dest"].shape[1] * page), device="cuda")
    heads = torch.arange(H, device="cuda")
    for b, n in enumerate(_ints(c["lens"])):
        m = min(n, keep)
        if n <= keep:
            ids = torch.arange(n, device="cuda").expand(H, n)
        else:
            top = torch.sort(s["weights"][b, :, :n - recent], dim=1, descending=True,
                             stable=True).indices[:, :keep - recent]
            last = torch.arange(n - recent, n, device="cuda").expand(H, recent)
            ids = torch.cat((torch.sort(top, dim=1).values, last), 1)
        kept[b, :, :m] = ids.to(torch.int32)
        weights[b, :, :m] = torch.gather(s["weights"][b], 1, ids)
        src = s["table"][b, ids // page].long() * page + ids % page  # [H, m]
        dst = _slots_of(s["dest"], b, 0, m, page)
        for which in range(2):
            e = cache.e[which][src // BLOCK, heads[:, None]]  # [H, m]
            fill = torch.nn.functional.pad(e, (0, -m % BLOCK), value=LOWEST)
            block = fill.reshape(H, -1, BLOCK).amax(2)  # [H, blocks]
            to = block.repeat_interleave(BLOCK, 1)[:, :m]
            row = _decode(cache.codes[which][src, heads[:, None]])
            cache.codes[which][dst] = _code(row, to - e).transpose(0, 1)
            cache.e[which][dst[::BLOCK] // BLOCK] = block.T
    return kept, weights


# ------------------------------------------------------------------ what a program keeps, one pass
def prepare(c, seed):
    s = _inputs(c, seed)
    s["case"] = c
    if own:
        import transformer_attention_iha_gb300 as iha
    if c["op"] == "rope":
        if own:
            s["rope"] = iha.Rope(c["rot"], base=BASE, interleaved=c["interleaved"],
                                 scaling=None if c["scaling"] == "none" else c["scaling"],
                                 factor=c["factor"], trained=c["trained"], fast=FAST, slow=SLOW)
        return s
    H, d, page = _heads(c), c["d"], c["page"]
    if own:
        s["cache"] = torch.zeros((s["n_pages"], iha.kv8_page_bytes(page, H, d)),
                                 dtype=torch.uint8, device="cuda")
    else:
        s["cache"] = _Plain(s["n_pages"], page, H, d)
    # the cache as earlier steps left it
    if c["op"] == "append":
        if own:
            iha.kv8_append(s["k0"], s["v0"], s["table"], s["old_lens"], s["cache"], page,
                           counts=s["had"])
        else:
            for b, n in enumerate(_ints(c["old"])):
                had = n % BLOCK
                if had:
                    s["cache"].append([s["k0"][b, BLOCK - 1 - had:], s["v0"][b, BLOCK - 1 - had:]],
                                      _slots_of(s["table"], b, n - had, n, page), n - had)
        del s["k0"], s["v0"]
        return s
    at = 0
    for b, n in enumerate(_ints(c["lens"])):
        if n and own:
            iha.kv8_append(s["k"][:, at:at + n], s["v"][:, at:at + n], s["table"][b:b + 1],
                           s["lens"][b:b + 1], s["cache"], page)
        elif n:
            s["cache"].append([s["k"][0, at:at + n], s["v"][0, at:at + n]],
                              _slots_of(s["table"], b, 0, n, page), 0)
        at += n
    del s["k"], s["v"]
    if own and c["op"] in ("attn", "weigh"):
        s["workspace"] = torch.zeros(
            iha.mha_fwd_kv8_workspace_bytes(
                c["B"], c["Nq"], c["Hq"], H, d,
                s["table"].shape[1] * page if c["op"] == "weigh" else 0),
            dtype=torch.uint8, device="cuda")
    return s


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import transformer_attention_iha_gb300 as iha
        if op == "rope":
            call = iha.rope_bwd if c["back"] else iha.rope_fwd
            return [y for y in call(s["q"], s["k"], s["pos"], s["rope"]) if y is not None]
        page = c["page"]
        if op == "append":
            iha.kv8_append(s["k"], s["v"], s["table"], s["lens"], s["cache"], page)
            return list(iha.kv8_load(s["cache"], s["back"], c["H"], c["d"], page,
                                     dtype=DT[c["dtype"]]))
        if op == "evict":
            lens, kept, weights = iha.kv8_evict(s["cache"], s["table"], s["lens"], s["weights"],
                                                s["dest"], c["Hkv"], c["d"], page, c["keep"],
                                                c["recent"])
            return [lens, kept, weights] + list(iha.kv8_load(s["cache"], s["back"], c["Hkv"],
                                                             c["d"], page))
        mask = {"none": iha.MASK_NONE, "causal": iha.MASK_CAUSAL,
                "window": iha.MASK_CAUSAL_WINDOW}[c["mask"]]
        return list(iha.mha_fwd_kv8(s["q"], s["cache"], s["table"], s["lens"], c["Hkv"], page,
                                    mask=mask, window=c["window"], return_lse=True,
                                    weights=s.get("weights"), workspace=s["workspace"]))
    if op == "rope":
        return _plain_rope(c, s)
    if op == "append":
        for b, n in enumerate(_ints(c["old"])):
            s["cache"].append([s["k"][b], s["v"][b]],
                              _slots_of(s["table"], b, n, n + c["N"], c["page"]), n)
        return s["cache"].load(s["back"], DT[c["dtype"]])
    if op == "evict":
        kept, weights = _plain_evict(c, s)
        return [torch.clamp(s["lens"], max=c["keep"]), kept, weights] + \
            s["cache"].load(s["back"], torch.bfloat16)
    return _plain_attn(c, s)


# ------------------------------------------------------------------ what a pass cannot do without
def work(c):
    d = c["d"]
    if c["op"] == "rope":
        T, H = c["B"] * c["N"], c["Hq"] + c["Hk"]
        es = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": T * (2 * H * d * es + 4), "flops": 3 * T * H * c["rot"]}
    row8 = 2 * d + 0.5  # K and V of a token and head, codes and scales (a byte each a block and 16)
    if c["op"] == "append":
        H, N = c["H"], c["N"]
        full = 2 * d * (2 if c["dtype"] == "bf16" else 4)
        old = sum(n % BLOCK for n in _ints(c["old"]))
        new = c["B"] * N
        # new rows in, codes out; codes of the blocks in, rows out, and their slots
        return {"bytes": int(new * H * (full + row8) + (new + old) * (H * (row8 + full) + 4)),
                "flops": 6 * (new + old) * H * d}
    lens = _ints(c["lens"])
    if c["op"] == "evict":
        H = c["Hkv"]
        kept = sum(min(n, c["keep"]) for n in lens)
        wide = c["B"] * -(-max(min(n, c["keep"]) for n in lens) // c["page"]) * c["page"]
        # weights read, written with the ids; rows moved; then read back as bf16
        return {"bytes": int(H * (4 * sum(lens) + 4 * wide + 4 * c["B"] * c["keep"]) +
                             kept * (H * (3 * row8 + 4 * d) + 4)),
                "flops": H * sum(lens)}
    Nq, Hq, Hkv = c["Nq"], c["Hq"], c["Hkv"]
    keys = pairs = 0
    for n in lens:
        w = c["window"] if c["mask"] == "window" else n + Nq
        if c["mask"] == "none":
            pairs += Nq * n
        else:
            pairs += sum(max(0, min(n - Nq + t + 1, w)) for t in range(Nq))
        keys += min(n, w + Nq - 1)
    more = 8 * c["B"] * Hkv * -(-max(1, max(lens)) // c["page"]) * c["page"]
    return {"bytes": int(keys * Hkv * row8 + c["B"] * Nq * Hq * (d * 2 * 2 + 4) + 4 * c["B"] +
                         (more if c["op"] == "weigh" else 0)),
            "flops": 4 * d * pairs * Hq}


# ------------------------------------------------------------------ the definition, in 64 bits
def _nearest8(y):
    """The nearest number with 3 fraction bits and exponent >= -6, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3.0)
    return torch.round(y / step) * step


def _log_scale(top):
    """The smallest whole e >= -100 with top <= 448 * 2^e, and 2^e."""
    e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -120) / 448.0)).clamp(min=-100.0)
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where((top <= 448.0 * torch.exp2(e - 1)) & (e > -100.0), e - 1, e)
    return torch.exp2(e)


def _held(x):
    """Values that rows x [n, H, d], positions from 0 on, have in the cache; scales by row."""
    n, H, d = x.shape
    held = torch.empty((n, H, d), dtype=torch.float64, device=x.device)
    scale = torch.empty((n, H), dtype=torch.float64, device=x.device)
    for a in range(0, n, 16384):
        part = x[a:a + 16384].double()
        m = part.shape[0]
        grid = torch.zeros((-(-m // 16) * 16, H, d), dtype=torch.float64, device=x.device)
        grid[:m] = part
        grid = grid.reshape(-1, 16, H, d)
        t = _log_scale(torch.amax(torch.abs(grid), dim=(1, 3), keepdim=True))
        held[a:a + m] = (_nearest8(grid / t) * t).reshape(-1, H, d)[:m]
        scale[a:a + m] = t.expand(-1, 16, -1, -1).reshape(-1, H)[:m]
    return held, scale


def _exact_rope(c, s):
    rot, f = c["rot"], c["factor"]
    freq, gain = [], 1.0
    for i in range(rot // 2):
        w = BASE ** (-2.0 * i / rot)
        if c["scaling"] == "linear":
            w /= f
        elif c["scaling"] == "base":
            w = (BASE * f ** (rot / (rot - 2.0))) ** (-2.0 * i / rot)
        elif c["scaling"] == "parts":
            g = min(1.0, max(0.0, (c["trained"] * w / (2 * math.pi) - SLOW) / (FAST - SLOW)))
            w = g * w + (1.0 - g) * w / f
            gain = 1.0 + 0.1 * math.log(f)
        freq.append(w)
    freq = torch.tensor(freq, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.full((), gain, device="cuda", dtype=torch.float64),
                       s["pos"].double()[..., None] * freq)[:, :, None, :]
    if c["back"]:
        turn = turn.conj()
    res = []
    for x in (s["q"], s["k"]):
        if x is None:
            continue
        y = x.double()
        pairs = y[..., :rot].unflatten(-1, (-1, 2) if c["interleaved"] else (2, -1))
        if not c["interleaved"]:
            pairs = pairs.transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        if not c["interleaved"]:
            z = z.transpose(-1, -2)
        res.append(torch.cat((z.flatten(-2), y[..., rot:]), -1))
    return res


def _exact_append(c, s):
    res = []
    for x0, x in ((s["k0"], s["k"]), (s["v0"], s["v"])):
        parts = []
        for b, n in enumerate(_ints(c["old"])):
            had = n % BLOCK
            first = BLOCK - had if had else 0  # new rows in the block that has earlier ones
            if had:
                old, t0 = _held(x0[b, 15 - had:])
                new = x[b, :first].double()
                t = torch.maximum(t0[0], _log_scale(new.abs().amax((0, 2))))[None, :, None]
                parts += [_nearest8(old / t) * t, _nearest8(new / t) * t]
            if c["N"] > first:
                parts.append(_held(x[b, first:])[0])
        res.append(torch.cat(parts)[None])
    return res


def _exact_evict(c, s):
    B, H, page, keep, recent = (c[n] for n in ("B", "Hkv", "page", "keep", "recent"))
    kept = torch.full((B, H, keep), -1, dtype=torch.int64, device="cuda")
    weights = torch.zeros((B, H, s["dest"].shape[1] * page), dtype=torch.float64, device="cuda")
    rows = ([], [])
    at = 0
    for b, n in enumerate(_ints(c["lens"])):
        m = min(n, keep)
        w = s["weights"][b, :, :n].double()
        if n > keep:
            # rank of a key: how many come before it, the larger first, then the earlier
            rank = w[:, :n - recent].neg().argsort(dim=1, stable=True).argsort(dim=1)
            stay = torch.ones((H, n), dtype=torch.bool, device="cuda")
            stay[:, :n - recent] = rank < keep - recent
        else:
            stay = torch.ones((H, n), dtype=torch.bool, device="cuda")
        ids = stay.nonzero()[:, 1].reshape(H, m)
        kept[b, :, :m] = ids
        weights[b, :, :m] = w.gather(1, ids)
        for x, to in ((s["k"], rows[0]), (s["v"], rows[1])):
            held, scale = _held(x[0, at:at + n])
            y = torch.stack([held[ids[h], h] for h in range(H)], 1)
            t = torch.stack([scale[ids[h], h] for h in range(H)], 1)
            for a in range(0, m, 16):
                t[a:a + 16] = t[a:a + 16].amax(0)
            to.append(_nearest8(y / t[..., None]) * t[..., None])
        at += n
    return [s["lens"].clamp(max=keep), kept, weights] + [torch.cat(r)[None] for r in rows]


def exact(c, seed):
    s = _inputs(c, seed)
    if c["op"] == "rope":
        return _exact_rope(c, s)
    if c["op"] == "append":
        return _exact_append(c, s)
    if c["op"] == "evict":
        return _exact_evict(c, s)
    B, Nq, Hq, Hkv, d = (c[n] for n in ("B", "Nq", "Hq", "Hkv", "d"))
    G = Hq // Hkv
    o = torch.zeros((B, Nq, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64, device="cuda")
    weights = s["weights"].double() if c["op"] == "weigh" else None
    at = 0
    for b, n in enumerate(_ints(c["lens"])):
        if n == 0:
            continue
        k, v = _held(s["k"][0, at:at + n])[0], _held(s["v"][0, at:at + n])[0]
        for t in range(Nq):
            last = n if c["mask"] == "none" else n - Nq + t + 1
            first = max(0, last - c["window"]) if c["mask"] == "window" else 0
            if last <= first:
                continue
            q = s["q"][b, t].double().reshape(Hkv, G, d)
            z = torch.einsum("jhf,hgf->hgj", k[first:last], q) / math.sqrt(d)
            p = torch.softmax(z, 2)
            lse[b, :, t] = torch.logsumexp(z, 2).reshape(-1)
            o[b, t] = torch.einsum("hgj,jhf->hgf", p, v[first:last]).reshape(Hq, d)
            if weights is not None:
                weights[b, :, first:last] += p.sum(1)
        at += n
    return [o, lse] if weights is None else [o, lse, weights]
