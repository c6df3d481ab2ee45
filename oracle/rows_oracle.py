"""Float64 oracle of the row operators: rows to expert order and back, their gradients,
and products of rows quantized to 8 bits.

TEST INFRASTRUCTURE, like oracle/moe_oracle.py.  Plain numpy, slot by slot; it shares no
code with the CUDA path.  A slot that is not routed has inv -1 (and expert id -1).
"""
import numpy as np


def expert_order(topk_idx, E):
    """counts [E], offsets [E + 1], the routed slots in expert order, and inv [T, k]."""
    flat = np.asarray(topk_idx).reshape(-1)
    order = [i for e in range(E) for i in np.flatnonzero(flat == e)]
    counts = np.array([(flat == e).sum() for e in range(E)], dtype=np.int64)
    inv = np.full(flat.shape, -1, dtype=np.int64)
    inv[np.array(order, dtype=np.int64)] = np.arange(len(order))
    return (counts, np.concatenate([[0], np.cumsum(counts)]), np.array(order, dtype=np.int64),
            inv.reshape(np.shape(topk_idx)))


def dispatch(x, inv, x_perm):
    """x_perm with row inv[t, j] replaced by x[t]."""
    out = np.array(x_perm, dtype=np.float64)
    for j in range(inv.shape[1]):
        on = inv[:, j] >= 0
        out[inv[on, j]] = x[on]
    return out


def to_tokens(rows, inv, weight=None, scale=1.0, add=None):
    """scale sum_j weight[t, j] rows[inv[t, j]] + add[t], and the same sum of magnitudes."""
    T, k = inv.shape
    y = np.zeros((T, rows.shape[1]))
    mag = np.zeros_like(y)
    for j in range(k):
        on = inv[:, j] >= 0
        term = rows[inv[on, j]] * (1.0 if weight is None else scale * weight[on, j, None])
        y[on] += term
        mag[on] += np.abs(term)
    if add is not None:
        y, mag = y + add, mag + np.abs(add)
    return y, mag


def combine_backward(dy, o, inv, weight, scale):
    """d_o (rows that no slot names: NaN), d_weight and the sum of magnitudes of its terms."""
    d_o = np.full(o.shape, np.nan)
    d_w = np.zeros(inv.shape)
    mag = np.zeros(inv.shape)
    for j in range(inv.shape[1]):
        on = inv[:, j] >= 0
        r = inv[on, j]
        d_o[r] = scale * weight[on, j, None] * dy[on]
        d_w[on, j] = scale * (dy[on] * o[r]).sum(1)
        mag[on, j] = abs(scale) * np.abs(dy[on] * o[r]).sum(1)
    return d_o, d_w, mag


def sigmoid(v):
    return np.where(v >= 0, 1 / (1 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1 + np.exp(-np.abs(v))))


def route_weights(logits, topk_idx, norm):
    """The weights of the selected experts (0 where not routed)."""
    on = topk_idx >= 0
    l = np.take_along_axis(logits, np.where(on, topk_idx, 0), 1)
    s = np.where(on, sigmoid(l), 0.0)
    return s / np.where(on.any(1), s.sum(1), 1)[:, None] if norm else s


def route_backward(logits, topk_idx, d_w, norm):
    """d_logits: the Jacobian of route_weights applied to d_w, entry by entry."""
    T, k = topk_idx.shape
    out = np.zeros(logits.shape)
    for t in range(T):
        js = [j for j in range(k) if topk_idx[t, j] >= 0]
        if not js:
            continue
        s = sigmoid(logits[t, topk_idx[t, js]])
        r = sigmoid(-logits[t, topk_idx[t, js]])  # 1 - s, which cancels near s = 1
        S = s.sum()
        for b, jb in enumerate(js):
            slope = s[b] * r[b]
            if norm:
                g = sum(d_w[t, ja] * ((a == b) / S - s[a] / S ** 2) for a, ja in enumerate(js))
            else:
                g = d_w[t, jb]
            out[t, topk_idx[t, jb]] += g * slope
    return out


def quantize_int8(x):
    """Codes and scales of float32 rows: every step one rounding to float32."""
    x = np.asarray(x, dtype=np.float32)
    with np.errstate(all="ignore"):
        amax = np.abs(x).max(1)
        s = np.maximum(amax / np.float32(127), np.float32(2.0 ** -126)).astype(np.float32)
        s = np.where(amax == 0, np.float32(1), s)
        bad = ~np.isfinite(x).all(1)
        q = np.rint((x * (np.float32(1) / s)[:, None]).astype(np.float32))
    q[bad] = 0
    return q.astype(np.int8), np.where(bad, np.float32("nan"), s)


def matmul_int8(a, sa, b, sb, offsets=None, swiglu=False):
    """out [M, N] in float64 (rows outside every group: NaN); for swiglu also gate and up.
    b [G, rows, K], sb [G, rows]."""
    M = a.shape[0]
    G, rows, _ = b.shape
    offsets = [0, M] if offsets is None else offsets
    z = np.full((M, rows), np.nan)
    for g in range(G):
        r = slice(int(offsets[g]), int(offsets[g + 1]))
        # float64 products of 8-bit integers add up exactly below 2^53
        z[r] = (a[r].astype(np.float64) @ b[g].astype(np.float64).T) * \
            np.asarray(sa, dtype=np.float64)[r, None] * np.asarray(sb[g], dtype=np.float64)
    if not swiglu:
        return z
    gate, up = z[:, :rows // 2], z[:, rows // 2:]
    return gate * sigmoid(gate) * up, gate, up
