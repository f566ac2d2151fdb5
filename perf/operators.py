"""What the 4-bit key/value cache of mxq is measured on: attention over the paged cache, appending
tokens to it (with reading them back as bf16), branching sequences that share pages, and compacting
the pages in use.

The sizes are those of the attention projection of the benchmark's problems (hidden size 5120, 7168
projection rows = 40 query heads + 2 x 8 key/value heads of 128), and generic ones beside it.

Layout of the cache.  A layer is uint8 [pages, kv_heads, page_size / 16, unit]: a unit holds 16 tokens
of one key/value head as  K codes (8 D bytes) | V codes (8 D bytes) | K scales | V scales  with D the
head size and nb = D / 32 (MXFP4) or D / 16 (NVFP4) scale bytes a token and side.  Two E2M1 codes a
byte, the even element in the low nibble ("row bytes" below: byte i = elements 2i, 2i + 1).
  K codes   the row's bytes are dealt to four quarters t = 0..3 of D / 8 bytes: NVFP4 quarter t is
            row bytes [t D/8, (t+1) D/8); MXFP4 quarter t is the 32-bit words t, t + 4, t + 8, ... of
            the row.  Quarters are cut in pieces of min(16, D / 8) bytes, stored [piece][token][t].
  V codes   row byte 8 j + g goes to lane (g, t) of its group of eight tokens, t = (token % 8) / 2, as
            byte (token % 2) D/16 + j of that lane's record of D / 8 bytes; records are cut in pieces of
            min(16, D / 8) bytes, stored [token / 8][piece][4 g + t].
  K scales  [token][nb].        V scales  [token / 2][nb][token % 2].
"""
import math
import random  # noqa: F401  (the type of draw's argument)

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ------------------------------------------------------------------------------------------ cases

def _attn(name, fmt, heads, kv_heads, dim, page, batch, shortest, longest, q=1, ragged_q=False, window=0):
    return dict(name=name, op="attention", fmt=fmt, heads=heads, kv_heads=kv_heads, dim=dim, page=page, batch=batch,
                shortest=shortest, longest=longest, q=q, ragged_q=ragged_q, window=window)


def listed():
    return [
        # one chat at an early turn, one new token: the latency of a single call
        _attn("decode 1 x 1009", "nvfp4", 40, 8, 128, 16, 1, 1009, 1009),
        # a serving batch in mid-flight: sequences of very different lengths, one new token each
        _attn("decode 32 x 500..16000", "mxfp4", 40, 8, 128, 64, 32, 500, 16000),
        # one long document, one new token: the cache has to be split over the whole GPU
        _attn("decode 1 x 131061", "nvfp4", 40, 8, 128, 64, 1, 131061, 131061),
        # four drafted tokens a sequence are verified at once
        _attn("verify 16 x 4 of 4100", "nvfp4", 40, 8, 128, 32, 16, 3000, 4100, q=4),
        # wide heads with a sliding window: the tail of a long sequence alone is read
        _attn("window 2048, heads of 256", "mxfp4", 24, 4, 256, 16, 24, 90, 9000, window=2048),
        # the next turns of two chats: chunks of new tokens over what the cache holds
        _attn("chunk 700 of 8300", "nvfp4", 40, 8, 128, 64, 2, 4200, 8300, q=700, ragged_q=True),
        # one decode step's new tokens of a batch, scattered over pages
        dict(name="append 64", op="append", fmt="nvfp4", kv_heads=8, heads=40, dim=128, page=16, tokens=64, run=1),
        # a prefill of several prompts, keys and values taken out of the fused projection's rows
        dict(name="append 8192", op="append", fmt="mxfp4", kv_heads=8, heads=40, dim=128, page=64, tokens=8192, run=977),
        # parallel samples of a few prompts: children share the prompt's pages, then write a token of their own
        dict(name="branch 4 x 3, 8 layers", op="branch", fmt="mxfp4", kv_heads=8, dim=128, page=16, layers=8, parents=4,
             children=3, length=1003, spare=64),
        # a beam step over long prompts and all layers: many tail pages are copied
        dict(name="branch 32 x 7, 24 layers", op="branch", fmt="nvfp4", kv_heads=8, dim=128, page=64, layers=24, parents=32,
             children=7, length=777, spare=40),
        # a small pool after some sequences ended
        dict(name="compact 600 pages", op="compact", fmt="nvfp4", kv_heads=8, dim=128, page=16, layers=4, pages=600, live=250,
             sequences=9),
        # a large pool, two thirds in use, is packed so that its end can be given back
        dict(name="compact 3000 pages", op="compact", fmt="mxfp4", kv_heads=8, dim=128, page=32, layers=16, pages=2987,
             live=1993, sequences=37),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    fmt = rng.choice(["mxfp4", "nvfp4"])
    page = rng.choice([16, 32, 64, 128])
    dim = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    op = rng.choice(["attention"] * 5 + ["append"] * 2 + ["branch", "compact"])
    if op == "attention":
        group = rng.choice([1, 2, 4, 5, 8, 12, 16])
        kind = rng.choice(["decode", "decode", "verify", "chunk"])
        batch = _log(rng, 1, 64 if kind != "chunk" else 4)
        most = min(131061, 200000000 // (batch * kv * dim))
        longest = _log(rng, 1, most if kind != "chunk" else 6000)
        shortest = _log(rng, 1, longest)
        q = 1 if kind == "decode" else rng.randint(2, 8) if kind == "verify" else _log(rng, 9, max(9, 9000 * 128 // (group * kv * dim * batch)))
        window = _log(rng, 5, 4096) if rng.random() < 0.3 else 0
        case = _attn("", fmt, kv * group, kv, dim, page, batch, shortest, longest, q, q > 1 and rng.random() < 0.5, window)
        del case["name"]
        return case
    if op == "append":
        tokens = _log(rng, 1, 8192)
        return dict(op=op, fmt=fmt, kv_heads=kv, heads=kv * rng.choice([1, 4, 5]), dim=dim, page=page, tokens=tokens,
                    run=_log(rng, 1, max(1, tokens)))
    if op == "branch":
        return dict(op=op, fmt=fmt, kv_heads=kv, dim=dim, page=page, layers=rng.randint(1, 8), parents=_log(rng, 1, 24),
                    children=rng.randint(1, 6), length=_log(rng, 1, 1500), spare=rng.randint(0, 50))
    pages = _log(rng, 2, 1500)
    live = rng.randint(1, pages)
    return dict(op=op, fmt=fmt, kv_heads=kv, dim=dim, page=page, layers=rng.randint(1, 8), pages=pages, live=live,
                sequences=rng.randint(1, min(live, 40)))


# ------------------------------------------------------------------------------ sizes of a case

def _nb(c):
    return c["dim"] // (32 if c["fmt"] == "mxfp4" else 16)


def _unit(c):
    return 16 * c["dim"] + 32 * _nb(c)


def _page_bytes(c):
    return c["kv_heads"] * (c["page"] // 16) * _unit(c)


def _lens(c):
    """Lengths between shortest and longest, evenly spread over their logarithm, in a fixed mixed order."""
    b, lo, hi = c["batch"], c["shortest"], c["longest"]
    return [int(round(lo * (hi / lo) ** (((i * 7 + 3) % b if b % 7 else i) / (b - 1)))) if b > 1 else hi for i in range(b)]


def _qlens(c):
    """New tokens of each sequence; they are the last ones of its length (fewer rows where it is shorter)."""
    return [max(1, c["q"] * (i + 1) // c["batch"]) if c["ragged_q"] else c["q"] for i in range(c["batch"])]


def _spans(c):
    """For each query token: first and end position that it attends to."""
    spans = []
    for n, q in zip(_lens(c), _qlens(c)):
        for j in range(q):
            end = max(0, n - q + j + 1)
            spans.append((max(0, end - c["window"]) if c["window"] else 0, end))
    return spans


def work(case):
    c = case
    if c["op"] == "attention":
        read = 0
        at, spans = 0, _spans(c)
        for q in _qlens(c):
            mine = spans[at:at + q]
            read += max(0, max(e for _, e in mine) - min(s for s, _ in mine))
            at += q
        pairs = sum(max(0, e - s) for s, e in spans)
        rows = len(spans) * c["heads"]
        return {"bytes": read * c["kv_heads"] * (c["dim"] + 2 * _nb(c)) + rows * (4 * c["dim"] + 4) + read // c["page"] * 4,
                "flops": 4.0 * pairs * c["heads"] * c["dim"]}
    if c["op"] == "append":  # read in bf16, written in 4 bits, then read in 4 bits and written in bf16
        values = 2 * c["tokens"] * c["kv_heads"] * c["dim"]
        return {"bytes": 2 * values * (2 + 0.5 + _nb(c) / c["dim"]), "flops": 4.0 * values}
    if c["op"] == "branch":
        n = c["parents"] * c["children"]
        used = -(-c["length"] // c["page"])
        copied = n if c["length"] % c["page"] else 0
        return {"bytes": 2 * copied * c["layers"] * _page_bytes(c) + 4 * n * (4 * used + 8), "flops": 0}
    used = 4 * (2 * c["live"] + c["pages"])
    return {"bytes": 2 * _moved(c) * c["layers"] * _page_bytes(c) + used, "flops": 0}


def _moved(c):
    """Pages to move: those in use at or behind the number in use, in the fixed pattern of _live."""
    return sum(1 for p in _live(c) if p >= c["live"])


def _live(c):
    """Which pages are in use: a fixed pattern, spread over the pool."""
    r = random.Random(c["pages"] * 31 + c["live"])
    return sorted(r.sample(range(c["pages"]), c["live"]))


# --------------------------------------------------------------------------- plain quantizer, layout

def _quantize(x, fmt, g):
    """x [..., D] fp32 -> codes [..., D] (uint8, 0..15) and scale bytes [..., nb]: block amax, MXFP4 scale by
    the CEIL rule (least power of two with amax <= 6 * scale), NVFP4 scale e4m3(amax / 6 / g), elements to
    the nearest E2M1 value, ties to the even code."""
    bs = 32 if fmt == "mxfp4" else 16
    b = x.float().unflatten(-1, (-1, bs))
    amax = b.abs().amax(-1)
    if fmt == "mxfp4":
        m, e = torch.frexp(amax)
        e = torch.where(amax > 0, e - 3 + (m > 0.75).int(), -127).clamp(-127, 127)
        sf = (e + 127).to(torch.uint8)
        v = torch.ldexp(b, (-e).unsqueeze(-1))
    else:
        s = (amax / 6.0 / g).clamp(max=448.0).to(torch.float8_e4m3fn)
        sf = s.view(torch.uint8)
        d = s.float() * g
        v = b * torch.where(d > 0, 1.0 / d, 0.0).unsqueeze(-1)
    a = v.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.round(a / step) * step
    code = torch.where(q < 2, q * 2, torch.where(q < 4, q + 2, q / 2 + 4)).to(torch.uint8)
    return (code + 8 * torch.signbit(b).to(torch.uint8)).flatten(-2), sf


def _pack(k, v, ks, vs, fmt):
    """Codes [..., 16, D] and scale bytes [..., 16, nb] of both sides -> units [..., unit]."""
    lead, D, nb = k.shape[:-2], k.shape[-1], ks.shape[-1]
    P, w = max(1, D // 128), min(16, D // 8)
    kb = (k[..., 0::2] + 16 * k[..., 1::2]).view(*lead, 16, D // 2)
    vb = (v[..., 0::2] + 16 * v[..., 1::2]).view(*lead, 2, 4, 2, D // 16, 8)
    if fmt == "mxfp4":
        kb = kb.view(*lead, 16, nb, 4, 4).transpose(-3, -2)
    kb = kb.reshape(*lead, 16, 4, P, w).movedim(-2, -4).reshape(*lead, 8 * D)
    vb = vb.movedim(-1, -4).reshape(*lead, 2, 32, P, w)       # [group][g, t][parity, j] in pieces
    vb = vb.movedim(-2, -3).reshape(*lead, 8 * D)
    vs = vs.view(*lead, 8, 2, nb).transpose(-1, -2).reshape(*lead, 16 * nb)
    return torch.cat([kb, vb, ks.reshape(*lead, 16 * nb), vs], -1)


def _unpack(u, fmt, D):
    """Units [..., unit] -> row bytes [..., 16, D / 2] and scale bytes [..., 16, nb] of keys, then of values."""
    lead, nb = u.shape[:-1], D // (32 if fmt == "mxfp4" else 16)
    P, w = max(1, D // 128), min(16, D // 8)
    kb, vb, ks, vs = u.split([8 * D, 8 * D, 16 * nb, 16 * nb], -1)
    kb = kb.reshape(*lead, P, 16, 4, w).movedim(-4, -2).reshape(*lead, 16, 4, D // 8)
    if fmt == "mxfp4":
        kb = kb.reshape(*lead, 16, 4, nb, 4).transpose(-3, -2)
    kb = kb.reshape(*lead, 16, D // 2)
    vb = vb.reshape(*lead, 2, P, 32, w).movedim(-3, -2).reshape(*lead, 2, 8, 4, 2, D // 16)
    vb = vb.movedim(-4, -1).reshape(*lead, 16, D // 2)
    return kb, ks.reshape(*lead, 16, nb), vb, vs.reshape(*lead, 8, nb, 2).transpose(-1, -2).reshape(*lead, 16, nb)


def _values(rows, sf, fmt, g):
    """Row bytes [..., D / 2] and scale bytes -> fp32 values [..., D]."""
    lut = torch.tensor(E2M1, device=rows.device)
    e = torch.stack([lut[(rows & 15).int()], lut[(rows >> 4).int()]], -1).flatten(-2)
    if fmt == "mxfp4":
        s = torch.ldexp(torch.ones_like(sf, dtype=torch.float32), sf.int() - 127)
    else:
        s = sf.view(torch.float8_e4m3fn).float() * g
    return (e.unflatten(-1, (sf.shape[-1], -1)) * s.unsqueeze(-1)).flatten(-2)


# ------------------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _kv(gen, c, tokens):
    """Keys with a few strong channels, values of unit spread, bf16 [tokens, kv_heads, dim] each."""
    shape = (tokens, c["kv_heads"], c["dim"])
    k = torch.randn(shape, generator=gen, device=DEV)
    k = k * (1 + 4 * (torch.rand((c["kv_heads"], c["dim"]), generator=gen, device=DEV) > 0.95))
    return k.to(torch.bfloat16), torch.randn(shape, generator=gen, device=DEV).to(torch.bfloat16)


def _scales(c):
    """NVFP4 per-tensor scales in the decode direction, as a calibrated model carries them (amax / 2688)."""
    if c["fmt"] == "mxfp4":
        return None, None
    return torch.tensor([27.1828 / 2688], device=DEV), torch.tensor([6.0973 / 2688], device=DEV)


def _filled(gen, c, pages):
    """A layer of `pages` full pages of quantized random keys and values."""
    cache = torch.empty((pages, c["kv_heads"], c["page"] // 16, _unit(c)), dtype=torch.uint8, device=DEV)
    gk, gv = _scales(c)
    at = max(1, (1 << 26) // (c["page"] * c["kv_heads"] * c["dim"]))
    for p in range(0, pages, at):
        n = min(at, pages - p)
        k, v = _kv(gen, c, n * c["page"])
        (k, ks), (v, vs) = _quantize(k, c["fmt"], gk), _quantize(v, c["fmt"], gv)
        cut = lambda x: x.view(n, c["page"] // 16, 16, c["kv_heads"], -1).permute(0, 3, 1, 2, 4)  # noqa: E731
        cache[p:p + n] = _pack(cut(k), cut(v), cut(ks), cut(vs), c["fmt"])
    return cache


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c, gen = case, _gen(seed)
    s = {"case": c}
    s["gk"], s["gv"] = _scales(c)
    if c["op"] == "attention":
        lens, ql = _lens(c), _qlens(c)
        used = [-(-n // c["page"]) for n in lens]
        total = max(1, sum(used))
        s["cache"] = _filled(gen, c, total)
        order = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
        table = torch.full((c["batch"], max(1, max(used))), -1, dtype=torch.int32, device=DEV)
        at = 0
        for i, n in enumerate(used):
            table[i, :n] = order[at:at + n]
            at += n
        s["table"], s["lens"] = table, _ints(lens)
        starts = [0]
        for q in ql:
            starts.append(starts[-1] + q)
        s["max_q"] = max(ql)
        s["q_start"] = _ints(starts)
        s["q"] = torch.randn((starts[-1], c["heads"], c["dim"]), generator=gen, device=DEV).to(torch.bfloat16)
        s["scale"] = c["dim"] ** -0.5
        if own:
            from nvfp4_block_scaled_mx_b200 import mxq
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty((starts[-1], c["heads"]), dtype=torch.float32, device=DEV)
            s["workspace"] = torch.empty(mxq.kv_attention_workspace(c["batch"], s["max_q"], c["heads"], c["kv_heads"],
                                                                    c["dim"]), dtype=torch.uint8, device=DEV)
    elif c["op"] == "append":
        T, H, D = c["tokens"], c["kv_heads"], c["dim"]
        k, v = _kv(gen, c, T)
        rows = torch.zeros((T, c["heads"] + 2 * H, D), dtype=torch.bfloat16, device=DEV)  # the fused projection's rows
        rows[:, c["heads"]:c["heads"] + H], rows[:, c["heads"] + H:] = k, v
        s["k"], s["v"] = rows[:, c["heads"]:c["heads"] + H], rows[:, c["heads"] + H:]
        # runs of `run` tokens, each in fresh pages that start at some offset
        runs = -(-T // c["run"])
        each = -(-c["run"] // c["page"]) + 1
        pages = runs * each
        order = torch.randperm(pages, generator=gen, device=DEV)
        i = torch.arange(T, device=DEV)
        off = torch.randint(0, c["page"], (runs,), generator=gen, device=DEV)[i // c["run"]] + i % c["run"]
        s["slots"] = (order[i // c["run"] * each + off // c["page"]] * c["page"] + off % c["page"]).to(torch.int32)
        s["cache"] = torch.zeros((pages, H, c["page"] // 16, _unit(c)), dtype=torch.uint8, device=DEV)
    elif c["op"] == "branch":
        n, kids, used = c["parents"], c["parents"] * c["children"], -(-c["length"] // c["page"])
        pages = n * used + kids * 2 + c["spare"]
        s["cache"] = _bytes(gen, c, pages)
        order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)[:n * used]
        s["table"] = torch.full((n + kids, used + 1), -1, dtype=torch.int32, device=DEV)
        s["table"][:n, :used] = order.view(n, used)
        s["lens"] = _ints([c["length"]] * n + [0] * kids)
        s["refs"] = torch.zeros(pages, dtype=torch.int32, device=DEV)
        s["refs"][order.long()] = 1
        s["kids"] = torch.arange(n, n + kids, dtype=torch.int32, device=DEV)
        s["of"] = (s["kids"] - n) // c["children"]
        s["zero"], s["one"] = _ints([0] * kids), _ints([1] * kids)
        if own:
            s["slots"], s["info"] = _ints([0] * kids), _ints([0, 0])
    else:
        used = _live(c)
        s["cache"] = _bytes(gen, c, c["pages"])
        live = _ints(used)[torch.randperm(c["live"], generator=gen, device=DEV)]
        n = c["sequences"]
        cuts = sorted(random.Random(c["live"]).sample(range(1, c["live"]), n - 1)) if n > 1 else []
        counts = [b - a for a, b in zip([0] + cuts, cuts + [c["live"]])]
        table = torch.full((n, max(counts)), -1, dtype=torch.int32, device=DEV)
        at = 0
        for i, m in enumerate(counts):
            table[i, :m] = live[at:at + m]
            at += m
        s["table0"], s["lens"] = table, _ints([m * c["page"] - (i * 5) % c["page"] for i, m in enumerate(counts)])
        s["refs0"] = torch.zeros(c["pages"], dtype=torch.int32, device=DEV)
        s["refs0"][live.long()] = 1
        s["table"], s["refs"] = table.clone(), s["refs0"].clone()
        if own:
            from nvfp4_block_scaled_mx_b200 import mxq
            s["info"] = _ints([0, 0])
            s["workspace"] = torch.empty(mxq.kv_compact_workspace(c["pages"]), dtype=torch.uint8, device=DEV)
    return s


def _bytes(gen, c, pages):
    """Layers of pages whose contents do not matter to what is done with them."""
    shape = (c["layers"], pages, c["kv_heads"], c["page"] // 16, _unit(c))
    return torch.randint(0, 120, shape, generator=gen, device=DEV, dtype=torch.uint8)


# ------------------------------------------------------------------------------------------ passes

def run(state):
    s = state
    c = s["case"]
    return {"attention": _attention, "append": _append, "branch": _branch, "compact": _compact}[c["op"]](s, c)


def _attention(s, c):
    if own:
        from nvfp4_block_scaled_mx_b200 import mxq
        return mxq.kv_attention(s["q"], s["cache"], s["table"], s["lens"], c["fmt"], q_start=s["q_start"], max_q=s["max_q"],
                                scale=s["scale"], window=c["window"], g_k=s["gk"], g_v=s["gv"], out=s["out"], lse=s["lse"],
                                workspace=s["workspace"])
    B, H, G, D = c["batch"], c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"]
    u = s["cache"][s["table"].clamp(min=0).long()]                       # [B, pages, H, units, unit]
    u = u.permute(0, 2, 1, 3, 4).flatten(2, 3)                           # [B, H, units, unit]
    kb, ks, vb, vs = _unpack(u, c["fmt"], D)
    k = _values(kb, ks, c["fmt"], s["gk"]).flatten(2, 3)                 # [B, H, L, D]
    v = _values(vb, vs, c["fmt"], s["gv"]).flatten(2, 3)
    pos = torch.arange(k.shape[2], device=DEV)
    v = torch.where((pos < s["lens"].view(-1, 1)).view(B, 1, -1, 1), v, 0.0)
    # the queries of each sequence, padded to max_q rows
    ql = s["q_start"][1:] - s["q_start"][:-1]
    j = torch.arange(s["max_q"], device=DEV)
    real = j < ql.view(-1, 1)                                            # [B, Q]
    at = torch.where(real, s["q_start"][:-1].view(-1, 1) + j, 0).long()
    q = s["q"].float()[at].unflatten(2, (H, G)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [B, H, Q G, D]
    end = s["lens"].view(-1, 1) - ql.view(-1, 1) + j + 1                 # [B, Q]
    seen = pos < end.unsqueeze(-1)
    if c["window"]:
        seen = seen & (pos >= (end - c["window"]).unsqueeze(-1))
    seen = seen.repeat_interleave(G, 1).unsqueeze(1)                     # [B, 1, Q G, L]
    x = torch.where(seen, q @ k.transpose(2, 3) * s["scale"], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total)).squeeze(-1)
    o = o.unflatten(2, (-1, G)).permute(0, 2, 1, 3, 4).flatten(2, 3)     # [B, Q, heads, D]
    lse = lse.unflatten(2, (-1, G)).permute(0, 2, 1, 3).flatten(2, 3)
    return o[real].to(torch.bfloat16), lse[real]


def _append(s, c):
    if own:
        from nvfp4_block_scaled_mx_b200 import mxq
        mxq.kv_append(s["k"], s["v"], s["cache"], s["slots"], c["fmt"], rule="ceil", g_k=s["gk"], g_v=s["gv"])
        return mxq.kv_read(s["cache"], s["slots"], c["fmt"], c["dim"], g_k=s["gk"], g_v=s["gv"])
    slot = s["slots"].long()
    page, unit, row = slot // c["page"], slot % c["page"] // 16, slot % 16
    (k, ks), (v, vs) = _quantize(s["k"], c["fmt"], s["gk"]), _quantize(s["v"], c["fmt"], s["gv"])
    # where each token's bytes lie in a unit: the layout applied to the bytes' own numbers
    T, H, D, nb = k.shape[0], c["kv_heads"], c["dim"], ks.shape[-1]
    number = torch.arange(_unit(c), device=DEV)
    kat, ksat, vat, vsat = (x.reshape(16, -1)[row].unsqueeze(1) for x in _unpack(number, c["fmt"], D))   # [T, 1, bytes]
    pack = lambda x: x[..., 0::2] + 16 * x[..., 1::2]  # noqa: E731
    data = torch.cat([pack(k), ks, pack(v), vs], -1)
    at = torch.cat([kat, ksat, vat, vsat], -1).expand_as(data)
    head = torch.arange(H, device=DEV).view(1, H, 1)
    s["cache"][page.view(-1, 1, 1), head, unit.view(-1, 1, 1), at] = data
    # and back
    got = s["cache"][page.view(-1, 1, 1), head, unit.view(-1, 1, 1), at]
    kb, ks, vb, vs = got.split([D // 2, nb, D // 2, nb], -1)
    return (_values(kb.contiguous(), ks.contiguous(), c["fmt"], s["gk"]).to(torch.bfloat16),
            _values(vb.contiguous(), vs.contiguous(), c["fmt"], s["gv"]).to(torch.bfloat16))


def _branch(s, c):
    """The last step's children are dropped, new ones share their parents' pages, and each gets room for a token."""
    if own:
        from nvfp4_block_scaled_mx_b200 import mxq
        mxq.kv_truncate(s["kids"], s["zero"], s["table"], s["lens"], s["refs"], c["page"], info=s["info"])
        mxq.kv_fork(s["of"], s["kids"], s["table"], s["lens"], s["refs"], c["page"], info=s["info"])
        mxq.kv_reserve(s["kids"], s["one"], s["table"], s["lens"], s["refs"], s["cache"], c["page"], slots=s["slots"],
                       info=s["info"])
        return s["table"], s["lens"], s["refs"], s["slots"], s["cache"]
    table, lens, refs, cache, ps = s["table"], s["lens"], s["refs"], s["cache"], c["page"]
    kids, of = s["kids"].long(), s["of"].long()
    col = torch.arange(table.shape[1], device=DEV)
    pages = lambda n: (n + ps - 1) // ps  # noqa: E731
    # drop
    held = col < pages(lens[kids]).unsqueeze(1)
    gone = table[kids][held].long()
    refs.index_put_((gone,), torch.full_like(gone, -1, dtype=torch.int32), accumulate=True)
    table[kids] = torch.where(held, -1, table[kids])
    lens[kids] = 0
    # share
    n = lens[of]
    held = col < pages(n).unsqueeze(1)
    mine = torch.where(held, table[of], -1)
    table[kids] = mine
    lens[kids] = n
    shared = mine[held].long()
    refs.index_put_((shared,), torch.ones_like(shared, dtype=torch.int32), accumulate=True)
    # room for one token: a tail page that is shared and not full is copied, a full one is followed by a new page
    last = (n - 1).clamp(min=0) // ps
    tail = torch.where(n > 0, mine.gather(1, last.long().unsqueeze(1)).squeeze(1), 0).long()
    copy = (n % ps != 0) & (refs[tail] > 1)
    need = copy | (n % ps == 0)
    free = torch.nonzero(refs == 0).squeeze(1)
    fresh = free[(torch.cumsum(need, 0) - 1).clamp(min=0)]
    cache[:, fresh[copy]] = cache[:, tail[copy]]
    refs.index_put_((tail[copy],), torch.full_like(tail[copy], -1, dtype=torch.int32), accumulate=True)
    refs[fresh[need]] = 1
    table[kids[need], (n // ps).long()[need]] = fresh[need].to(torch.int32)
    lens[kids] = n + 1
    slots = table[kids, (n // ps).long()] * ps + n % ps
    return table, lens, refs, slots, cache


def _compact(s, c):
    """The pool as it was left is packed: pages in use behind the first `live` ones move into the holes among them."""
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    if own:
        from nvfp4_block_scaled_mx_b200 import mxq
        mxq.kv_compact(s["table"], s["lens"], s["refs"], s["cache"], c["page"], info=s["info"], workspace=s["workspace"])
        return s["table"], s["refs"], s["info"], s["cache"]
    table, refs, cache = s["table"], s["refs"], s["cache"]
    used = refs > 0
    live = used.sum()
    at = torch.arange(refs.numel(), device=DEV)
    src, dst = torch.nonzero(used & (at >= live)).squeeze(1), torch.nonzero(~used & (at < live)).squeeze(1)
    to = at.to(torch.int32)
    to[src] = dst.to(torch.int32)
    held = torch.arange(table.shape[1], device=DEV) < ((s["lens"] + c["page"] - 1) // c["page"]).unsqueeze(1)
    s["table"] = torch.where(held, to[table.clamp(min=0).long()], table)
    cache[:, dst] = cache[:, src]
    refs[dst] = refs[src]
    refs[src] = 0
    return s["table"], refs, torch.stack([torch.zeros_like(live), live]).to(torch.int32), cache


# -------------------------------------------------------------------------- definition in 64 bits

def _decode64(codes, scales, fmt, g):
    """One row of bytes after another: codes [n, D / 2], scales [n, nb] -> float64 [n, D]."""
    byte = torch.tensor([[E2M1[b & 15], E2M1[b >> 4]] for b in range(256)], dtype=torch.float64, device=DEV)
    e = byte[codes.long()].reshape(codes.shape[0], -1)
    if fmt == "mxfp4":
        s = torch.exp2(scales.double() - 127)
    else:
        exp, man = (scales >> 3).double(), (scales & 7).double()
        s = torch.where(exp == 0, man * 2.0 ** -9, (1 + man / 8) * torch.exp2(exp - 7)) * g.double()
    return e * s.repeat_interleave(e.shape[1] // s.shape[1], 1)


def _where64(c):
    """Byte positions in a unit of each token's row bytes and scales, by the words of the layout alone."""
    D, nb, P = c["dim"], _nb(c), min(16, c["dim"] // 8)
    kc, vc, ks, vs = [], [], [], []
    for r in range(16):
        row = [0] * (D // 2)
        for i in range(D // 2):
            if c["fmt"] == "mxfp4":
                word, t = i // 4 // 4, i // 4 % 4
                inside = word * 4 + i % 4
            else:
                t, inside = divmod(i, D // 8)
            row[i] = (inside // P) * 64 * P + (r * 4 + t) * P + inside % P
        kc.append(row)
        row = [0] * (D // 2)
        for i in range(D // 2):
            j, g = divmod(i, 8)
            inside = (r % 2) * (D // 16) + j
            row[i] = 8 * D + (r // 8) * 4 * D + (inside // P) * 32 * P + (4 * g + (r % 8) // 2) * P + inside % P
        vc.append(row)
        ks.append([16 * D + r * nb + b for b in range(nb)])
        vs.append([16 * D + 16 * nb + (r // 2) * 2 * nb + 2 * b + r % 2 for b in range(nb)])
    return [torch.tensor(x, device=DEV) for x in (kc, ks, vc, vs)]


def exact(case, seed):
    c = case
    if c["op"] in ("branch", "compact"):
        return None  # whole numbers and bytes
    s = prepare(c, seed)
    if c["op"] == "append":
        out = []
        for x, g in ((s["k"], s["gk"]), (s["v"], s["gv"])):
            b = x.double().reshape(-1, 32 if c["fmt"] == "mxfp4" else 16)
            amax = b.abs().amax(1, keepdim=True)
            if c["fmt"] == "mxfp4":
                sc = torch.exp2(torch.ceil(torch.log2(amax / 6)))
                sc = torch.where(amax <= 3 * sc, sc / 2, torch.where(amax > 6 * sc, sc * 2, sc))
            else:
                u = (amax / 6 / g.double()).clamp(max=448.0)
                step = torch.exp2(torch.floor(torch.log2(u.clamp(min=2.0 ** -6))) - 3)
                sc = torch.round(u / step) * step * g.double()
            v = torch.where(sc > 0, b / sc, 0.0)
            a = v.abs().clamp(max=6.0)
            step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
            out.append((torch.round(a / step) * step * torch.sign(v) * sc).reshape(x.shape))
        return tuple(out)
    kat, ksat, vat, vsat = _where64(c)
    gk, gv = s["gk"], s["gv"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    G, at, spans = c["heads"] // c["kv_heads"], 0, _spans(c)
    for b, (n, q) in enumerate(zip(_lens(c), _qlens(c))):
        mine = spans[at:at + q]
        lo = torch.tensor([x for x, _ in mine], device=DEV).view(-1, 1, 1)
        hi = torch.tensor([x for _, x in mine], device=DEV).view(-1, 1, 1)
        rows = s["q"][at:at + q].double()
        live = [i for i, (x, y) in enumerate(mine) if y > x]
        if live:
            pages = s["table"][b, :-(-n // c["page"])].long()
            for h in range(c["kv_heads"]):
                u = s["cache"][pages, h].reshape(-1, _unit(c))
                k = _decode64(u[:, kat].reshape(-1, c["dim"] // 2), u[:, ksat].reshape(-1, _nb(c)), c["fmt"], gk)[:n]
                v = _decode64(u[:, vat].reshape(-1, c["dim"] // 2), u[:, vsat].reshape(-1, _nb(c)), c["fmt"], gv)[:n]
                x = rows[:, h * G:(h + 1) * G] @ k.T * s["scale"]
                pos = torch.arange(n, device=DEV)
                x = torch.where((pos >= lo) & (pos < hi), x, -math.inf)
                z = torch.logsumexp(x, -1)
                lse[at:at + q, h * G:(h + 1) * G] = z
                p = torch.exp(x - torch.where(z == -math.inf, 0.0, z).unsqueeze(-1))
                o[at:at + q, h * G:(h + 1) * G] = p @ v
        at += q
    return o, lse
