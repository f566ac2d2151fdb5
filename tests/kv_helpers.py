"""Shared helpers of the key/value cache tests: the cache's layout from its description, tokens quantized
by the oracle, attention in 64 bits, and the page bookkeeping as plain Python."""
import numpy as np
import torch

import oracle

FMT = {"mxfp4": oracle.MXFP4, "nvfp4": oracle.NVFP4}
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6])


def nb_of(D, fmt):
    return D // (32 if fmt == "mxfp4" else 16)


def unit_bytes(D, fmt):
    return 16 * D + 32 * nb_of(D, fmt)


def positions(D, fmt):
    """Byte positions in a unit: K codes [16, D/2], K scales [16, nb], V codes, V scales."""
    nb, W = nb_of(D, fmt), min(16, D // 8)
    kc = np.zeros((16, D // 2), np.int64)
    vc = np.zeros((16, D // 2), np.int64)
    for r in range(16):
        for i in range(D // 2):
            if fmt == "mxfp4":
                t, inside = i // 4 % 4, i // 16 * 4 + i % 4
            else:
                t, inside = i // (D // 8), i % (D // 8)
            kc[r, i] = inside // W * 64 * W + (r * 4 + t) * W + inside % W
            j, g = i // 8, i % 8
            inside = r % 2 * (D // 16) + j
            vc[r, i] = 8 * D + r // 8 * 4 * D + inside // W * 32 * W + (4 * g + r % 8 // 2) * W + inside % W
    r, b = np.arange(16)[:, None], np.arange(nb)[None]
    return kc, 16 * D + r * nb + b, vc, 16 * D + 16 * nb + r // 2 * 2 * nb + 2 * b + r % 2


def quantize(x, fmt, rule, g):
    """x [n, H, D] bf16 -> codes [n, H, D/2], scales [n, H, nb] by the oracle."""
    n, H, D = x.shape
    flat = x.detach().cpu().reshape(n * H, D).contiguous()
    q, sf = oracle.quantize(flat, FMT[fmt], {"even": oracle.EVEN, "ceil": oracle.CEIL}[rule], 1.0 if g is None else g)
    return np.asarray(q).reshape(n, H, D // 2), np.asarray(sf).reshape(n, H, nb_of(D, fmt))


def append(cache, k, v, slots, fmt, rule, gk, gv):
    """The cache (numpy uint8 [P, H, units, U]) with the tokens written, in place."""
    D, page = k.shape[2], 16 * cache.shape[2]
    pos = positions(D, fmt)
    parts = quantize(k, fmt, rule, gk) + quantize(v, fmt, rule, gv)
    for i, s in enumerate(slots):
        if s < 0:
            continue
        u = cache[s // page, :, s % page // 16]
        for p, d in zip(pos, parts):
            u[:, p[s % 16]] = d[i]


def values(codes, scales, fmt, g):
    """Row bytes [..., D/2] and scales [..., nb] -> float64 [..., D] (nan scales stay nan)."""
    e = np.stack([E2M1[codes & 15], E2M1[codes >> 4]], -1).reshape(codes.shape[:-1] + (2 * codes.shape[-1],))
    s = scales.astype(np.float64)
    if fmt == "mxfp4":
        s = np.exp2(s - 127)
    else:
        exp, man = scales >> 3, scales & 7
        s = np.where(exp == 0, man * 2.0 ** -9, (1 + man / 8) * np.exp2(exp.astype(np.float64) - 7)) * float(g)
    return e * np.repeat(s, e.shape[-1] // s.shape[-1], -1)


def tokens(cache, table_row, n, D, fmt, gk, gv):
    """Keys and values of the first n tokens of a sequence: float64 [n, H, D] each."""
    page = 16 * cache.shape[2]
    pos = positions(D, fmt)
    s = np.arange(n)
    u = cache[np.asarray(table_row)[s // page], :, s % page // 16]       # [n, H, U]
    at = [np.take_along_axis(u, np.broadcast_to(p[s % 16][:, None], u.shape[:2] + (p.shape[1],)), 2) for p in pos]
    return values(at[0], at[1], fmt, gk), values(at[2], at[3], fmt, gv)


def attention(q, cache, table, lens, q_start, fmt, scale, causal, window, gk, gv):
    """out, lse, sum of p |v|, the largest sum of |scale q k|, and tokens times the largest |v|, in float64;
    rows of no sequence are nan."""
    T, Hq, D = q.shape
    H = cache.shape[1]
    G = Hq // H
    out = np.full((T, Hq, D), np.nan)
    lse = np.full((T, Hq), np.nan)
    absv = np.zeros((T, Hq, D))
    floor = np.zeros((T, Hq, 1))
    mass = np.zeros((T, Hq))
    for b, n in enumerate(lens):
        n = max(int(n), 0)
        k, v = tokens(cache, table[b], n, D, fmt, gk, gv)
        for i in range(q_start[b], q_start[b + 1]):
            seen = n - (q_start[b + 1] - q_start[b]) + (i - q_start[b]) + 1
            end = max(seen, 0) if causal else n
            first = max(seen - window, 0) if window else 0
            for h in range(Hq):
                if end <= first:
                    out[i, h], lse[i, h] = 0, -np.inf
                    continue
                kk, vv = k[first:end, h // G], v[first:end, h // G]
                x = kk @ q[i, h] * scale
                top = x.max()
                p = np.exp(x - top)
                total = p.sum()
                out[i, h] = p @ vv / total
                lse[i, h] = top + np.log(total)
                absv[i, h] = p @ np.abs(vv) / total
                floor[i, h] = len(vv) * np.abs(vv).max()
                mass[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
    return out, lse, absv, mass, floor


def check_attention(out, lse, ref, what=""):
    """Tolerances.  A score is a sum of exact products in fp32: it is off by at most 2^-20 of the sum of
    their magnitudes (D <= 256 additions of 2^-24 each, twice, for the tensor cores' truncation, and the
    power-of-two scaling of q, whose smallest elements may lose 2^-31 of the largest), and 2^-22 of its
    own size for the scaling and the exponential.  With d that bound, a probability is off by 2 d (its
    own score and the denominator's), by 2^-11 + 2^-12 for its rounding to f16 and its product's with
    the scale, and by 2^-16 for what fp32 sums of up to 2^16 terms lose.  Below f16's normal range the
    two roundings are absolute: half of 2^-24, of a probability times 2^4 or more and of its product, which
    is at most 2^11 times that for the block's largest scale -- in all at most 2^-28 of the largest value a
    token.  bf16 adds half a step of the result, 2^-8; a result of 0 is exact."""
    r, l, absv, mass, floor = ref
    o, z = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(z), np.isneginf(l)), "%s: rows without tokens" % what
    f = np.isfinite(l)
    d = (2.0 ** -20 + 2.0 ** -22) * mass + 2.0 ** -22 * np.abs(np.where(f, l, 0))
    err = np.abs(z[f] - l[f])
    assert (err <= (d + 2.0 ** -18)[f]).all(), "%s: lse off by %g" % (what, err.max())
    half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
    tol = half * np.abs(r) + (2 * d[..., None] + 2.0 ** -11 + 2.0 ** -12 + 2.0 ** -16) * absv * (1 + half) + 2.0 ** -28 * floor
    err = np.abs(o - r)
    assert (err <= tol).all(), "%s: out off by up to %g of its tolerance" % (what, np.nanmax(err / np.maximum(tol, 1e-300)))


class Pool:
    """Block tables, lengths and reference counts as plain Python."""

    def __init__(self, rows, cols, pages, page):
        self.table = [[-1] * cols for _ in range(rows)]
        self.lens, self.refs, self.page, self.cols = [0] * rows, [0] * pages, page, cols

    def pages_for(self, n):
        return -(-n // self.page)

    def _rows_ok(self, rows):
        return len(set(rows)) == len(rows) and all(0 <= r < len(self.lens) for r in rows)

    def reserve(self, seqs, add, slots_cap=None):
        """(status, pages, slots, copies)"""
        if not self._rows_ok(seqs):
            return -1, 0, None, []
        if any(a < 0 or self.lens[s] + a > self.cols * self.page for s, a in zip(seqs, add)):
            return -2, 0, None, []
        if slots_cap is not None and sum(add) > slots_cap:
            return -2, 0, None, []
        free = [p for p, r in enumerate(self.refs) if r == 0]
        wanted, copies = [], []
        for s, a in zip(seqs, add):
            n = self.lens[s]
            cells = list(range(self.pages_for(n), self.pages_for(n + a)))
            if a and n % self.page and self.refs[self.table[s][n // self.page]] > 1:
                cells.insert(0, n // self.page)
                copies.append((s, n // self.page))
            wanted += [(s, c) for c in cells]
        if len(wanted) > len(free):
            return -3, 0, None, []
        moved = []
        for (s, c), p in zip(wanted, free):
            if (s, c) in copies:
                moved.append((self.table[s][c], p))
            self.table[s][c] = p
            self.refs[p] = 1
        for old, _ in moved:
            self.refs[old] -= 1
        slots = []
        for s, a in zip(seqs, add):
            slots += [self.table[s][p // self.page] * self.page + p % self.page for p in range(self.lens[s], self.lens[s] + a)]
            self.lens[s] += a
        return 0, len(wanted), slots, moved

    def fork(self, parents, children):
        if not self._rows_ok(children) or any(self.lens[c] for c in children) or \
                any(not 0 <= p < len(self.lens) or p in children for p in parents):
            return -1, 0
        n = 0
        for p, c in zip(parents, children):
            k = self.pages_for(self.lens[p])
            self.table[c][:k] = self.table[p][:k]
            for x in self.table[p][:k]:
                self.refs[x] += 1
            self.lens[c] = self.lens[p]
            n += k
        return 0, n

    def truncate(self, seqs, to):
        if not self._rows_ok(seqs):
            return -1, 0
        if any(not 0 <= n <= self.lens[s] for s, n in zip(seqs, to)):
            return -2, 0
        dropped = 0
        for s, n in zip(seqs, to):
            for k in range(self.pages_for(n), self.pages_for(self.lens[s])):
                self.refs[self.table[s][k]] -= 1
                self.table[s][k] = -1
                dropped += 1
            self.lens[s] = n
        return 0, dropped

    def compact(self):
        """(pages in use, moves)"""
        live = sum(r > 0 for r in self.refs)
        src = [p for p, r in enumerate(self.refs) if r > 0 and p >= live]
        dst = [p for p, r in enumerate(self.refs) if r == 0 and p < live]
        to = dict(zip(src, dst))
        for row, n in zip(self.table, self.lens):
            for k in range(self.pages_for(n)):
                row[k] = to.get(row[k], row[k])
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        return live, list(to.items())
