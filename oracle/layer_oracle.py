"""Float64 oracle of the 4-bit expert layer: routing with gate weights, microscaled 4-bit quantization,
products over routed segments, combination. Plain numpy, written from the definitions; shares no code
with the GPU path. Every decision (block scale, code, expert order) is made in float64, where the
compared quantities are exact or 29 bits away from the borders of float32 inputs.
"""
import numpy as np

BLOCK = {"e8m0_32": 32, "e4m3_16": 16}
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# every finite non-negative e4m3 number in code order (0x00 .. 0x7e)
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:-1])


def nearest_code(a, levels):
    """Index of the level nearest to each a >= 0, ties to the even index, the last level for anything above."""
    a = np.asarray(a, np.float64)
    hi = np.clip(np.searchsorted(levels, a), 1, len(levels) - 1)
    lo = hi - 1
    below, above = a - levels[lo], levels[hi] - a
    even = np.where(lo % 2 == 0, lo, hi)
    code = np.where(below < above, lo, np.where(below > above, hi, even))
    return np.where(a >= levels[-1], len(levels) - 1, code)


def fp4_quantize(x, fmt, g=1.0):
    """(codes uint8 [R, d], scale bytes uint8 [R, d / block]) of x [R, d]; g: matrix scale, scalar or per row."""
    x = np.asarray(x, np.float64)
    R, d = x.shape
    g = np.broadcast_to(np.asarray(g, np.float64).reshape(-1, 1), (R, 1))
    v = x.reshape(R, -1, BLOCK[fmt])
    top = np.abs(v).max(2) / g
    if fmt == "e8m0_32":
        e = np.where(top > 0, np.frexp(top)[1] - 1 - 2, -127)
        byte = np.clip(e, -127, 127) + 127
        s = np.ldexp(1.0, byte - 127)
    else:
        byte = np.where(top > 0, np.maximum(nearest_code(top / 6, E4M3), 1), 0)
        s = E4M3[byte]
    D = (s * g)[:, :, None]
    a = np.divide(np.abs(v), D, out=np.zeros_like(v), where=D > 0)
    c = nearest_code(a, E2M1) + np.where(np.signbit(v), 8, 0)
    return c.reshape(R, d).astype(np.uint8), byte.astype(np.uint8)


def fp4_values(codes, byte, fmt, g=1.0):
    """Float64 values [R, d] of codes [R, d] and scale bytes [R, d / block]."""
    R, d = codes.shape
    byte = byte.astype(np.int64)
    s = np.ldexp(1.0, byte - 127) if fmt == "e8m0_32" else E4M3[byte]
    q = np.where(codes >= 8, -1.0, 1.0) * E2M1[codes & 7]
    g = np.broadcast_to(np.asarray(g, np.float64).reshape(-1, 1), (R, 1))
    return (q.reshape(R, -1, BLOCK[fmt]) * s[:, :, None]).reshape(R, d) * g


def pack_codes4(codes):
    """uint8 [R, d / 2], the even column in the low four bits."""
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def tile_scales(byte):
    """The tiled scale layout, flat: 512-byte tiles of 128 rows x 4 blocks, row-major, zero padded."""
    R, nb = byte.shape
    rt, kt = -(-R // 128), -(-nb // 4)
    out = np.zeros(rt * kt * 512, np.uint8)
    r, b = np.indices((R, nb))
    out[((r // 128) * kt + b // 4) * 512 + 16 * (r % 32) + 4 * ((r % 128) // 32) + b % 4] = byte
    return out


def silu(x):
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore"):
        return x / (1.0 + np.exp(-x))


def expert_products(x, w, seg=None):
    """Y [rows, N] of x [rows, K] and w [E, N, K]; with seg (starts [E + 1], counts [E]) each expert's rows meet
    its own matrix and every other row is zero."""
    if seg is None:
        return x @ w[0].T
    E = w.shape[0]
    y = np.zeros((x.shape[0], w.shape[1]))
    for e in range(E):
        r = slice(int(seg[e]), int(seg[e] + seg[E + 1 + e]))
        y[r] = x[r] @ w[e].T
    return y


def route_gated(logits, k, score="softmax", bias=None, n_groups=1, top_groups=1, group_rank="max", renormalise=True,
                scale=1.0):
    """(ids [n, k], weights float64 [n, k], counts [E])."""
    l = np.asarray(logits, np.float64)
    n, E = l.shape
    if score == "softmax":
        s = np.exp(l - l.max(1, keepdims=True))
        s /= s.sum(1, keepdims=True)
    else:
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-l))
    by_logit = bias is None and (n_groups == 1 or group_rank == "max")
    c = l.copy() if by_logit else s + (0.0 if bias is None else np.asarray(bias, np.float64))
    ids = np.zeros((n, k), np.int64)
    size = E // n_groups
    for t in range(n):
        groups = c[t].reshape(n_groups, size)
        best = np.sort(groups, 1)[:, ::-1]
        rank = best[:, 0] if group_rank == "max" or size == 1 else best[:, 0] + best[:, 1]
        keep = sorted(range(n_groups), key=lambda g: (-rank[g], g))[:top_groups]
        live = [e for g in keep for e in range(g * size, (g + 1) * size)]
        ids[t] = sorted(live, key=lambda e: (-c[t, e], e))[:k]
    w = np.take_along_axis(s, ids, 1)
    if renormalise:
        total = w.sum(1, keepdims=True)
        w = np.where(total > 0, np.divide(w, total, out=np.zeros_like(w), where=total > 0), 1.0 / k)
    return ids, w * scale, np.bincount(ids.ravel(), minlength=E)


def combine(z, ids, weights, seg, perm, E, add=None):
    """Y [n, d] = add + sum_j weights[:, j] z[row of the token in the segment of expert ids[:, j]]."""
    n, k = ids.shape
    y = np.zeros((n, z.shape[1])) if add is None else np.asarray(add, np.float64).copy()
    for t in range(n):
        for j in range(k):
            e = int(ids[t, j])
            lo, cnt = int(seg[e]), int(seg[E + 1 + e])
            row = lo + int(np.nonzero(perm[lo:lo + cnt] == t)[0][0])
            y[t] += (1.0 if weights is None else weights[t, j]) * z[row]
    return y
