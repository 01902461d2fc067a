"""Plain 64-bit forms of the decoding step's operators, on the CPU, written
from their definitions: paged cache rows, the e4m3 form of a row, attention of
one new token, and a beam-search step.  They share no code with the library.
"""
import math

import torch

NINF = -math.inf


def e4m3_values():
    """The 256 values of an e4m3 code, from its bit fields."""
    out = []
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        if e == 15 and m == 7:
            v = math.nan
        else:
            v = (m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        out.append(-v if s else v)
    return torch.tensor(out, dtype=torch.float64)


_VALUES = e4m3_values()


def decode_rows(data, scale):
    """Values of cache rows [..., d] in 64 bits."""
    if scale is None:
        return data.double()
    return _VALUES[data.view(torch.uint8).long()] * scale.double()[..., None]


def quantise_row(x):
    """(values the stored codes stand for without the scale, scale) of one row
    of bf16 values: smallest power of two 2^e, e >= -127, with max|x| <= 448 * 2^e,
    and the nearest code (the even one of two) of every x / 2^e."""
    x = x.double()
    if not torch.isfinite(x).all():
        return torch.full_like(x, math.nan), math.nan
    top = float(x.abs().max())
    e = 0
    if top > 0:
        e = -127
        while top > 448 * 2.0 ** e:
            e += 1
    grid = _VALUES[:127]  # 0 .. 448, increasing; a code's last bit is its index's parity
    y = (x.abs() / 2.0 ** e)
    hi = torch.searchsorted(grid, y).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - y, y - grid[lo]
    pick_lo = (down < up) | ((down == up) & (lo % 2 == 0))
    return torch.copysign(torch.where(pick_lo, grid[lo], grid[hi]), x), 2.0 ** e


def sequence_rows(cache, scale, table_row, tokens, head):
    """Rows [len(tokens), d] of one sequence's head; None where the page does not exist."""
    pages, _, page, _ = cache.shape
    got = []
    for t in tokens:
        at = int(table_row[t // page])
        if 0 <= at < pages:
            got.append(decode_rows(cache[at, head, t % page], None if scale is None else scale[at, head, t % page]))
    d = cache.shape[3]
    return torch.stack(got) if got else torch.zeros(0, d, dtype=torch.float64)


def attention(q, k_cache, v_cache, table, lens, scale, k_scale=None, v_scale=None, positions=None):
    """(out, lse, bound on sum p|V| per output, largest |q||k| scale per head), 64 bits, CPU tensors."""
    batch, heads, d = q.shape
    kv_heads, page = k_cache.shape[1:3]
    capacity = table.shape[1] * page
    out = torch.zeros(batch, heads, d, dtype=torch.float64)
    mass = torch.zeros_like(out)
    lse = torch.full((batch, heads), NINF, dtype=torch.float64)
    size = torch.zeros(batch, heads, dtype=torch.float64)
    cached = {}
    for b in range(batch):
        n = min(max(int(lens[b]), 0), capacity)
        for h in range(heads):
            kv = h // (heads // kv_heads)
            if positions is None:
                tokens = tuple(range(n))
            else:
                lists = positions.shape[1]
                tokens = tuple(t for t in positions[b, h // (heads // lists)].tolist() if 0 <= t < n)
            if (b, kv, tokens) not in cached:
                cached = {(b, kv, tokens): (sequence_rows(k_cache, k_scale, table[b], tokens, kv),
                                            sequence_rows(v_cache, v_scale, table[b], tokens, kv))}
            k, v = cached[(b, kv, tokens)]
            if k.shape[0] == 0:
                continue
            t = (k @ q[b, h].double()) * scale
            if bool((t == NINF).all()):
                continue
            size[b, h] = abs(scale) * float(q[b, h].double().norm() * k.norm(dim=1).max())
            lse[b, h] = torch.logsumexp(t, 0)
            p = torch.exp(t - t.max()) if not torch.isnan(t).any() else t
            p = p / p.sum()
            out[b, h] = p @ v
            mass[b, h] = p @ v.abs()
    return out, lse, mass, size


def beam_step(logits, scores, k):
    """The k best continuations of one sentence: [(value, beam, token)], best first."""
    beams, _ = logits.shape
    found = []
    for i in range(beams):
        s = float(scores[i])
        if s == NINF:
            continue
        x = logits[i].double()
        bad = bool(torch.isnan(x).any() or (x == math.inf).any())
        off = math.nan if bad else s - float(torch.logsumexp(x, 0))
        live = torch.nonzero(x != NINF).flatten().tolist()
        xs = x.tolist()
        row = sorted(live, key=lambda t: (0 if math.isnan(xs[t]) else 1, -xs[t] if not math.isnan(xs[t]) else 0.0, t))
        found += [(off + xs[t], i, t) for t in row[:k]]
    order = sorted(range(len(found)), key=lambda j: (0 if math.isnan(found[j][0]) else 1,
                                                     0.0 if math.isnan(found[j][0]) else -found[j][0], found[j][1], j))
    return [found[j] for j in order[:k]]
