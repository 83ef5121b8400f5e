"""Plain references, in 64 bits, of the routed-token, norm, quantizer and 8-bit product calls."""

import numpy as np


def moe_capacity(T, top_k, E, align):
    n = T * top_k
    return (n + min(E, n) * (align - 1)) // align * align


def moe_tables(ids, E, align, capacity):
    """(m_indptr [E + 1], idx [T, top_k], inv [capacity]) by walking the slots in order."""
    ids = np.asarray(ids)
    segs = [[] for _ in range(E)]
    for i, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < E:
            segs[e].append(i)
    indptr = np.zeros(E + 1, dtype=np.int64)
    idx = np.full(ids.size, -1, dtype=np.int64)
    inv = np.full(capacity, -1, dtype=np.int64)
    for e in range(E):
        for r, i in enumerate(segs[e]):
            idx[i] = indptr[e] + r
            inv[indptr[e] + r] = i
        indptr[e + 1] = indptr[e] + -(-len(segs[e]) // align) * align
    return indptr, idx.reshape(ids.shape), inv


def moe_sum(rows, idx, w=None):
    """sum_j w[t, j] * rows[idx[t, j]] over the slots with an index >= 0."""
    T, k = idx.shape
    out = np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(k):
            if idx[t, j] >= 0:
                out[t] += rows[idx[t, j]] * (1.0 if w is None else w[t, j])
    return out


def moe_unpermute_grads(g, y, idx, w, grad_rows, used, inv):
    """(gy, gw): gy starts from `grad_rows`, with zeros in the padding rows below `used`."""
    gy = np.array(grad_rows, dtype=np.float64)
    gy[:used][inv[:used] < 0] = 0.0
    gw = np.zeros(idx.shape)
    for t in range(idx.shape[0]):
        for j in range(idx.shape[1]):
            p = idx[t, j]
            if p >= 0:
                gy[p] = g[t] * (1.0 if w is None else w[t, j])
                if w is not None:
                    gw[t, j] = g[t] @ y[p]
    return gy, gw


def _e4m3_values():
    """The values of the 256 E4M3 bytes (no infinities; 0x7F and 0xFF are NaN)."""
    v = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[b] = np.nan if b & 127 == 127 else (-x if b & 128 else x)
    return v


E4M3 = _e4m3_values()


def e4m3_encode(x):
    """Bytes of x rounded to the nearest E4M3 value, ties to the even byte, saturating at 448."""
    x = np.asarray(x, dtype=np.float64)
    pos = E4M3[:127]                                  # 0 .. 448, ascending
    mag = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(pos, mag), 1, 126)
    lo = hi - 1
    dl, dh = mag - pos[lo], pos[hi] - mag
    code = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    code = np.where(np.isnan(x), 127, code)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def fp8_quantize(x, block_rows=1):
    """(bytes, scales): the rule in float32, every operation rounded once."""
    x = np.asarray(x, dtype=np.float32)
    T, H = x.shape
    R, G = -(-T // block_rows), -(-H // 128)
    q = np.empty((T, H), dtype=np.uint8)
    s = np.empty((R, G), dtype=np.float32)
    for r in range(R):
        for g in range(G):
            at = np.s_[r * block_rows:(r + 1) * block_rows, g * 128:(g + 1) * 128]
            amax = np.float32(max(np.abs(x[at]).max(), 2.0 ** -100))
            s[r, g] = amax / np.float32(448)
            q[at] = e4m3_encode(x[at] * (np.float32(448) / amax))
    return q, s


def add_rmsnorm(x, residual, weight, eps):
    """(h, y) of the norm, in 64 bits."""
    h = np.asarray(x, dtype=np.float64) + (0.0 if residual is None else residual)
    return h, h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * weight


def mm_fp8(a, b, sa, sb, bias=None):
    """(out, magnitude): the product of dequantized operands in 64 bits, and the sum of its terms' sizes."""
    K, N = a.shape[1], b.shape[0]
    av = E4M3[a] * np.repeat(np.asarray(sa, dtype=np.float64), 128, axis=1)[:, :K]
    bv = E4M3[b] * np.repeat(np.repeat(np.asarray(sb, dtype=np.float64), 128, axis=1)[:, :K], 128, axis=0)[:N]
    out = av @ bv.T
    return (out if bias is None else out + bias), np.abs(av) @ np.abs(bv).T
