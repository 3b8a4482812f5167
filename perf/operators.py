"""The serving operators of an IHA layer with a 4-bit key-value cache, as they are measured.

Four operators of one decode step:
  premix   the premix of Q, K and V of new tokens at given positions (RoPE on Q and K);
  store    K and V rows quantised to 4 bits as they are written to a paged cache, and read back;
  load     rows of the cache read back to bf16 or float32, in any order;
  attn     softmax attention of new queries over the 4-bit paged cache.

Definition of a row held in 4 bits: values count as bf16 (float32 is rounded to it); a row of d
features is d / 32 groups of 32 neighbours; a group's scale is s = bf16(max |x| / 7) and its codes
are c = round(x / s), ties to even, -7 <= c <= 7; a group stands for s * c.  A slot is a token's
place in the cache, page * page_size + offset; slot -1 is padding: not stored, read back as zeros.

`own` chooses what `run` does: false, elementary torch operations in 32 bits; true, the calls a
user makes of the library.
"""
import math

import torch

own = False

GROUP = 32
ROPE_BASE = 10000.0
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def _store(name, B, N, H, d, page, dtype="bf16", pad=0.0):
    return dict(name=name, op="store", B=B, N=N, H=H, d=d, page=page, dtype=dtype, pad=pad)


def _load(name, B, N, H, d, page, dtype="bf16"):
    return dict(name=name, op="load", B=B, N=N, H=H, d=d, page=page, dtype=dtype, pad=0.0)


def _attn(name, B, Nq, Hq, Hkv, d, page, lens, mask="causal", window=0):
    return dict(name=name, op="attn", B=B, Nq=Nq, Hq=Hq, Hkv=Hkv, d=d, page=page,
                lens=",".join(str(n) for n in lens), mask=mask, window=window)


def _premix(name, B, N, H, P, d, pos0):
    return dict(name=name, op="premix", B=B, N=N, H=H, P=P, d=d, pos0=pos0)


def listed():
    return [
        # one decode step of 8 sequences: 80 pseudo-heads of 20 heads x P = 4, latency
        _store("store_step_b8", 8, 1, 80, 128, 64),
        # a whole prompt written after its prefill
        _store("store_prompt_8k", 1, 8192, 80, 128, 64),
        # float32 rows of a padded batch (slot -1), small pages, odd length
        _store("store_padded_f32", 3, 333, 8, 64, 16, "f32", 0.2),
        # a long prefix read back for a prefill that goes on from it, rows in any order
        _load("load_prefix_16k", 1, 16384, 80, 128, 64),
        # a few rows of heads of 96, as float32
        _load("load_rows_d96_f32", 2, 117, 20, 96, 32, "f32"),
        # one sequence, short context: the smallest attention call
        _attn("decode_b1_777", 1, 1, 80, 80, 128, 64, [777]),
        # a ragged batch with shared key-value heads, one sequence just begun
        _attn("decode_gqa_b16", 16, 1, 32, 8, 128, 64,
              [8192, 1, 513, 4095, 7000, 64, 65, 1999, 3001, 8190, 12, 6144, 2500, 777, 5120, 128]),
        # one long context
        _attn("decode_long_131071", 1, 1, 80, 80, 128, 64, [131071]),
        # sliding-window layers: 1024 keys of each sequence, whatever its length
        _attn("decode_window_b32", 32, 1, 80, 80, 128, 64,
              [1 + (i * 2654435761) % 16000 for i in range(32)], "window", 1024),
        # the joint-softmax variant: the P = 4 pseudo-tokens of a new token, 20 heads
        _attn("decode_joint_b4", 4, 4, 20, 20, 128, 64, [32768, 30004, 16384, 400]),
        # premix of one new token of 16 sequences
        _premix("premix_step_b16", 16, 1, 20, 4, 128, 4096),
        # premix of a chunk that continues a prompt
        _premix("premix_chunk_2k", 1, 2048, 20, 4, 128, 14336),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["store", "load", "attn", "attn", "attn", "premix"])
    if op == "premix":
        H = rng.choice([4, 8, 16, 20, 32])
        P = rng.choice([p for p in (1, 2, 3, 4) if p * H <= 128])
        d = rng.choice([64, 128])
        T = _log(rng, 1, 4096 * 2560 // (H * d) if H * d > 2560 else 4096)
        B = min(T, _log(rng, 1, 64))
        return dict(op=op, B=B, N=max(1, T // B), H=H, P=P, d=d, pos0=rng.randrange(0, 120000))
    d = rng.choice([32, 64, 96, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    if op in ("store", "load"):
        H = rng.choice([1, 4, 8, 20, 80])
        T = _log(rng, 1, min(16384, 8192 * 80 * 128 // (H * d)))
        B = min(T, _log(rng, 1, 32))
        return dict(op=op, B=B, N=max(1, T // B), H=H, d=d, page=page,
                    dtype=rng.choice(["bf16", "bf16", "f32"]),
                    pad=rng.choice([0.0, 0.3]) if op == "store" else 0.0)
    Hkv, G = rng.choice([(80, 1), (40, 1), (20, 1), (8, 1), (8, 4), (8, 8), (4, 7), (2, 16), (1, 8)])
    B = _log(rng, 1, 64)
    Nq = rng.choice([1, 1, 1, 2, 4, 5, 8, 16])
    top = max(64, min(131072, 16384 * 80 * 128 // (B * Hkv * d)))
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
    g.manual_seed(1000003 * seed + 17)
    return g


def _normal(g, shape, dtype=torch.bfloat16, std=1.0, mean=None, gain=None):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    if std != 1.0:
        x *= std
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
    return _normal(g, shape, dtype, 1.0, mean, gain), _normal(g, shape, dtype)


def _lens(c):
    return [int(n) for n in c["lens"].split(",")]


def _inputs(c, seed):
    g = _gen(seed)
    s = {}
    if c["op"] == "premix":
        B, N, H, P, d = (c[n] for n in "BNHPd")
        s["xs"] = [_normal(g, (B, N, H, d)) for _ in range(3)]
        s["ws"] = [_normal(g, (H, P, H), torch.float32, H ** -0.5) for _ in range(3)]
        start = c["pos0"] + 37 * torch.arange(B, device="cuda", dtype=torch.int32)
        s["pos"] = (start[:, None] + torch.arange(N, device="cuda", dtype=torch.int32)).contiguous()
        return s
    if c["op"] in ("store", "load"):
        B, N, H, d, page = c["B"], c["N"], c["H"], c["d"], c["page"]
        T = B * N
        s["n_pages"] = -(-T // page) + 3
        if c["op"] == "load":
            s["k"], s["v"] = _kv(g, (1, T, H, d), torch.bfloat16)
        else:
            s["k"], s["v"] = _kv(g, (B, N, H, d), DT[c["dtype"]])
        if T <= 4096 or c["op"] == "load":  # rows in any order
            perm = torch.randperm(s["n_pages"] * page, generator=g, device="cuda")[:T]
        else:  # a prompt: pages in any order, rows in order inside them
            pages = torch.randperm(s["n_pages"], generator=g, device="cuda")
            perm = (pages[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:T]
        s["slots"] = perm.to(torch.int32).reshape(B, N)
        if c["pad"]:
            drop = torch.rand((B, N), generator=g, device="cuda") < c["pad"]
            s["slots"] = torch.where(drop, -1, s["slots"]).to(torch.int32)
        return s
    B, Nq, Hq, Hkv, d, page = (c[n] for n in ("B", "Nq", "Hq", "Hkv", "d", "page"))
    lens = _lens(c)
    per = [-(-n // page) for n in lens]
    s["n_pages"] = sum(per) + 2
    order = torch.randperm(s["n_pages"], generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((B, max(1, max(per))), device="cuda", dtype=torch.int32)
    at = 0
    slots = []
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        rows = (order[at:at + n, None] * page +
                torch.arange(page, device="cuda", dtype=torch.int32)).reshape(-1)[:lens[b]]
        slots.append(rows)
        at += n
    s["table"] = table
    s["slots"] = torch.cat(slots).reshape(1, -1).contiguous()
    s["lens"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
    s["k"], s["v"] = _kv(g, (1, s["slots"].shape[1], Hkv, d), torch.bfloat16)
    s["q"] = _normal(g, (B, Nq, Hq, d))
    return s


# ------------------------------------------------------------------ plain forms, 32 bits
def _quantise(x):
    """x [..., d] -> codes two to a byte [..., d / 2], scales bf16 [..., d / 32]."""
    xg = x.to(torch.bfloat16).float().unflatten(-1, (-1, GROUP))
    s = (xg.abs().amax(-1) / 7.0).to(torch.bfloat16)
    sf = s.float().unsqueeze(-1)
    c = torch.where(sf > 0, torch.round(xg / sf), 0.0)
    c = (c + 8.0).to(torch.uint8).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), s


def _values(codes, s):
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8.0
    return (c.unflatten(-1, (-1, GROUP)) * s.float().unsqueeze(-1)).flatten(-2)


def _plain_cache(rows, H, d):
    """Codes and scales; one row more than there are slots takes what padding writes."""
    return [torch.zeros((rows + 1, H, d // 2), dtype=torch.uint8, device="cuda"),
            torch.zeros((rows + 1, H, d // GROUP), dtype=torch.bfloat16, device="cuda")]


def _plain_store(caches, xs, slots):
    flat = slots.reshape(-1).long()
    at = torch.where(flat >= 0, flat, caches[0][0].shape[0] - 1)
    for (codes, scales), x in zip(caches, xs):
        c, s = _quantise(x.flatten(0, 1))
        codes[at] = c
        scales[at] = s


def _plain_load(caches, slots, dtype):
    flat = slots.reshape(-1)
    out = []
    for codes, scales in caches:
        at = flat.clamp(min=0).long()
        x = _values(codes[at], scales[at])
        x = torch.where((flat >= 0)[:, None, None], x, 0.0)
        out.append(x.to(dtype).unflatten(0, slots.shape))
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
    for b, n in enumerate(_lens(c)):
        lo = max(0, n - Nq + 1 - c["window"]) if c["mask"] == "window" else 0
        if n == 0:
            continue
        j = torch.arange(lo, n, device="cuda")
        rows = s["table"][b, j // page].long() * page + j % page
        k = _values(s["caches"][0][0][rows], s["caches"][0][1][rows])
        v = _values(s["caches"][1][0][rows], s["caches"][1][1][rows])
        q = s["q"][b].float().reshape(Nq, Hkv, G, d).permute(1, 2, 0, 3).reshape(Hkv, G * Nq, d)
        x = torch.matmul(q, k.permute(1, 2, 0)) * (1.0 / math.sqrt(d))
        vis = _visible(c, n, "cuda")[:, lo:].repeat(G, 1)
        x = torch.where(vis, x, -math.inf)
        m = x.amax(-1, keepdim=True)
        m = torch.where(m > -math.inf, m, 0.0)
        p = torch.exp(x - m)
        l = p.sum(-1, keepdim=True)
        r = torch.matmul(p, v.permute(1, 0, 2)) / torch.where(l > 0, l, 1.0)
        o[b] = r.reshape(Hkv, G, Nq, d).permute(2, 0, 1, 3).reshape(Nq, Hq, d).to(torch.bfloat16)
        lse[b] = (m + torch.log(l)).reshape(Hq, Nq)
    return o, lse


def _plain_premix(c, s):
    d, half = c["d"], c["d"] // 2
    inv = ROPE_BASE ** (-2.0 * torch.arange(half, device="cuda", dtype=torch.float64) / d)
    a = s["pos"].double()[:, :, None, None] * inv  # far positions: the angle in 64 bits
    cos, sin = torch.cos(a).float(), torch.sin(a).float()
    out = []
    for t in range(3):
        H, P, _ = s["ws"][t].shape
        y = torch.matmul(s["ws"][t].reshape(H * P, H), s["xs"][t].float())
        if t < 2:
            y0, y1 = y[..., :half], y[..., half:]
            y = torch.cat((y0 * cos - y1 * sin, y1 * cos + y0 * sin), -1)
        out.append(y.to(torch.bfloat16))
    return out


# ------------------------------------------------------------------ what a program keeps, one pass
def prepare(c, seed):
    s = _inputs(c, seed)
    s["case"] = c
    if c["op"] == "premix":
        return s
    H = c["Hkv"] if c["op"] == "attn" else c["H"]
    d, page = c["d"], c["page"]
    if own:
        import transformer_attention_iha_gb300 as iha
        s["cache"] = torch.zeros((s["n_pages"], iha.kv4_page_bytes(page, H, d)),
                                 dtype=torch.uint8, device="cuda")
        if c["op"] == "attn":
            s["workspace"] = torch.zeros(
                iha.mha_fwd_kv4_workspace_bytes(c["B"], c["Nq"], c["Hq"], H, d),
                dtype=torch.uint8, device="cuda")
    else:
        s["caches"] = [_plain_cache(s["n_pages"] * page, H, d) for _ in range(2)]
    if c["op"] != "store":  # the cache as earlier steps left it
        slots = s["slots"].reshape(1, -1).contiguous()
        if own:
            iha.kv4_store(s["k"], s["v"], slots, s["cache"], page)
        else:
            for at in range(0, slots.shape[1], 16384):
                part = slice(at, at + 16384)
                _plain_store(s["caches"], (s["k"][:, part], s["v"][:, part]), slots[:, part])
        del s["k"], s["v"]
    return s


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import transformer_attention_iha_gb300 as iha
        if op == "premix":
            return list(iha.premix_fwd_qkv_at(s["xs"], s["ws"], c["P"], s["pos"],
                                              rope_base=ROPE_BASE))
        if op == "store":
            iha.kv4_store(s["k"], s["v"], s["slots"], s["cache"], c["page"])
            return list(iha.kv4_load(s["cache"], s["slots"], c["H"], c["d"], c["page"],
                                     dtype=DT[c["dtype"]]))
        if op == "load":
            return list(iha.kv4_load(s["cache"], s["slots"], c["H"], c["d"], c["page"],
                                     dtype=DT[c["dtype"]]))
        mask = {"none": iha.MASK_NONE, "causal": iha.MASK_CAUSAL,
                "window": iha.MASK_CAUSAL_WINDOW}[c["mask"]]
        return list(iha.mha_fwd_kv4(s["q"], s["cache"], s["table"], s["lens"], c["Hkv"], c["page"],
                                    mask=mask, window=c["window"], return_lse=True,
                                    workspace=s["workspace"]))
    if op == "premix":
        return _plain_premix(c, s)
    if op == "store":
        _plain_store(s["caches"], (s["k"], s["v"]), s["slots"])
        return _plain_load(s["caches"], s["slots"], DT[c["dtype"]])
    if op == "load":
        return _plain_load(s["caches"], s["slots"], DT[c["dtype"]])
    return list(_plain_attn(c, s))


# ------------------------------------------------------------------ what a pass cannot do without
def work(c):
    d = c["d"]
    if c["op"] == "premix":
        T, H, HP = c["B"] * c["N"], c["H"], c["H"] * c["P"]
        return {"bytes": 3 * (T * (H + HP) * d * 2 + HP * H * 4) + 4 * T,
                "flops": 3 * 2 * T * HP * H * d + 2 * 3 * T * HP * d}
    row4 = 2 * (d // 2 + d // GROUP * 2)  # K and V of a token and head, codes and scales
    if c["op"] in ("store", "load"):
        T, H = c["B"] * c["N"], c["H"]
        full = 2 * d * (2 if c["dtype"] == "bf16" else 4)
        kept = T * (1.0 - c["pad"])
        if c["op"] == "load":
            return {"bytes": int(T * (H * (row4 + full) + 4)), "flops": 2 * T * H * d}
        # rows in, codes out, codes in, rows out
        return {"bytes": int(kept * H * (full + 2 * row4) + T * (H * full + 8)),
                "flops": int(kept * 10 * H * d)}
    Nq, Hq, Hkv = c["Nq"], c["Hq"], c["Hkv"]
    keys = pairs = 0
    for n in _lens(c):
        w = c["window"] if c["mask"] == "window" else n + Nq
        if c["mask"] == "none":
            pairs += Nq * n
        else:
            pairs += sum(max(0, min(n - Nq + t + 1, w)) for t in range(Nq))
        keys += min(n, w + Nq - 1)
    return {"bytes": keys * Hkv * row4 + c["B"] * Nq * Hq * (d * 2 * 2 + 4) + 4 * c["B"],
            "flops": 4 * d * pairs * Hq}


# ------------------------------------------------------------------ the definition, in 64 bits
def _held(x):
    """The values that x [rows, H, d] has once it is held in 4 bits, from the definition."""
    rows, H, d = x.shape
    y = x.to(torch.bfloat16).double().reshape(rows, H, d // 32, 32)
    top = torch.maximum(y.max(3, keepdim=True).values, -y.min(3, keepdim=True).values)
    step = (top / 7).to(torch.bfloat16).double()
    safe = torch.where(step == 0, torch.ones_like(step), step)
    return (torch.round(y / safe) * step).reshape(rows, H, d)


def exact(c, seed):
    s = _inputs(c, seed)
    if c["op"] == "premix":
        half = c["d"] // 2
        freq = torch.exp(torch.arange(half, device="cuda", dtype=torch.float64) *
                         (-2.0 / c["d"] * math.log(ROPE_BASE)))
        turn = torch.polar(torch.ones((), device="cuda", dtype=torch.float64),
                           s["pos"].double()[..., None] * freq)[:, :, None, :]
        res = []
        for t, (x, w) in enumerate(zip(s["xs"], s["ws"])):
            y = torch.einsum("hps,bnsf->bnhpf", w.double(), x.double()).flatten(2, 3)
            if t != 2:
                z = torch.complex(y[..., :half].contiguous(), y[..., half:].contiguous()) * turn
                y = torch.cat((z.real, z.imag), -1)
            res.append(y)
        return res
    if c["op"] in ("store", "load"):
        B, N, H, d = c["B"], c["N"], c["H"], c["d"]
        pad = (s["slots"] < 0).reshape(B, N, 1, 1)
        return [_held(x.reshape(B * N, H, d)).reshape(B, N, H, d).masked_fill(pad, 0.0)
                for x in (s["k"], s["v"])]
    B, Nq, Hq, Hkv, d = (c[n] for n in ("B", "Nq", "Hq", "Hkv", "d"))
    o = torch.zeros((B, Nq, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b, n in enumerate(_lens(c)):
        for t in range(Nq if n else 0):
            last = n if c["mask"] == "none" else n - Nq + t + 1
            first = max(0, last - c["window"]) if c["mask"] == "window" else 0
            if last <= first:
                continue
            k = _held(s["k"][0, at + first:at + last]).repeat_interleave(Hq // Hkv, 1)
            z = (k * s["q"][b, t].double()).sum(-1).T / math.sqrt(d)
            del k
            lse[b, :, t] = torch.logsumexp(z, 1)
            v = _held(s["v"][0, at + first:at + last]).repeat_interleave(Hq // Hkv, 1)
            o[b, t] = (torch.softmax(z, 1).T[..., None] * v).sum(0)
            del v
        at += n
    return [o, lse]
