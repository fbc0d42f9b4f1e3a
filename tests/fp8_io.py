"""Plain 64-bit forms of the routing and 8-bit operators, for their tests:
numpy only, written from the formulas in include/averis.h."""

import numpy as np


# ---------------------------------------------------------------------------
# E4M3 and the block rule
# ---------------------------------------------------------------------------
def e4m3_decode(codes):
    c = np.asarray(codes, dtype=np.uint8).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((e == 15) & (m == 7), np.nan, v)
    return np.where(c & 128, -v, v)


def e4m3_round(y):
    """Nearest E4M3 value (ties to even) of |y| <= 448, in fp64."""
    _, x = np.frexp(y)
    step = np.ldexp(1.0, np.maximum(x - 1, -6) - 3)
    return np.round(y / step) * step


def block_exponent(amax):
    """Smallest integer e >= -127 with amax <= 448 * 2^e, by search from below."""
    e = np.full(np.shape(amax), -127, dtype=np.int64)
    for _ in range(260):
        e = np.where(np.asarray(amax, dtype=np.float64) > 448.0 * 2.0 ** e.astype(np.float64), e + 1, e)
    return e


def quant(x, block=(1, 128)):
    """(values of the codes, scale bytes per block) of x [a, b] in fp64; a
    value times 2^(byte - 127) of its block is the quantized element."""
    x = np.asarray(x, dtype=np.float64)
    a, b = x.shape
    A, B = block
    na, nb = -(-a // A), -(-b // B)
    full = np.zeros((na * A, nb * B))
    full[:a, :b] = x
    v = full.reshape(na, A, nb, B)
    e = block_exponent(np.abs(v).max(axis=(1, 3)))
    q = e4m3_round(v * 2.0 ** -e.astype(np.float64)[:, None, :, None]).reshape(na * A, nb * B)[:a, :b]
    return q, (e + 127).astype(np.uint8)


def dequant(q, scales, block=(1, 128)):
    A, B = block
    e = scales.astype(np.float64) - 127
    return q * (2.0 ** e).repeat(A, 0).repeat(B, 1)[: q.shape[0], : q.shape[1]]


def deq(x, block=(1, 128)):
    return dequant(*quant(x, block), block)


def atoms(s):
    """Scale bytes [rows, blocks] in the atom layout, byte by byte."""
    r, c = s.shape
    na = -(-c // 4)
    out = np.zeros(-(-r // 128) * na * 512, dtype=np.uint8)
    R, C = np.meshgrid(np.arange(r), np.arange(c), indexing="ij")
    out[((R // 128) * na + C // 4) * 512 + 16 * (R % 32) + 4 * (R % 128 // 32) + C % 4] = s
    return out


def from_atoms(flat, r, c):
    na = -(-c // 4)
    R, C = np.meshgrid(np.arange(r), np.arange(c), indexing="ij")
    return np.asarray(flat)[((R // 128) * na + C // 4) * 512 + 16 * (R % 32) + 4 * (R % 128 // 32) + C % 4]


def tensor_value(t):
    """The fp64 value of an api.FP8Tensor."""
    q = e4m3_decode(t.codes.cpu().numpy())
    return dequant(q, from_atoms(t.scales.cpu().numpy(), t.rows, -(-t.K // 128)))


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------
def route(logits, k, norm):
    """(ids, weights): the k largest finite logits, lower index first."""
    T, E = logits.shape
    ids, w = np.full((T, k), -1, dtype=np.int32), np.zeros((T, k))
    for t in range(T):
        l = logits[t].astype(np.float64)
        if not np.all(l < np.inf):
            continue
        order = sorted((e for e in range(E) if l[e] > -np.inf), key=lambda e: (-l[e], e))[:k]
        if not order:
            continue
        over = l[order] if norm else l[l > -np.inf]
        den = np.exp(over - l.max()).sum()
        ids[t, : len(order)] = order
        w[t, : len(order)] = np.exp(l[order] - l.max()) / den
    return ids, w


def route_bwd(logits, norm, ids, w, dw):
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        j = np.nonzero(ids[t] >= 0)[0]
        s = float((w[t, j].astype(np.float64) * dw[t, j]).sum())
        for i in j:
            out[t, ids[t, i]] += float(w[t, i]) * (float(dw[t, i]) - (s if norm else 0.0))
        if not norm:
            l = logits[t].astype(np.float64)
            if np.any(l > -np.inf):
                p = np.exp(l - l.max())
                out[t] -= p / p.sum() * s
    return out


def sort(ids, E):
    """(counts, row, first row of each expert, rows in use)."""
    flat = np.asarray(ids).reshape(-1)
    flat = np.where((flat < 0) | (flat >= E), -1, flat)
    counts = np.array([(flat == e).sum() for e in range(E)], dtype=np.int64)
    off = np.concatenate([[0], np.cumsum(-(-counts // 128) * 128)])
    row = np.full(flat.shape, -1, dtype=np.int64)
    for e in range(E):
        at = np.nonzero(flat == e)[0]
        row[at] = off[e] + np.arange(at.size)
    return counts, row.reshape(np.shape(ids)), off[:-1], int(off[-1])
