"""Float64 oracle of attention over packed sequences and of projections with per-segment low-rank adapters, written
from their formulas (numpy, row by row, no code shared with the kernels)."""
import numpy as np


def packed_attention(q, k, v, q_start, k_start, causal, scale=None):
    """(o [H, Tq, d], lse [H, Tq], weight [H, Tq, d], spread [H, Tq]) for q [H, Tq, d], k, v [Hk, Tk, d]; rows in no
    sequence are NaN. weight: sum of the softmax weights times |v|; spread: the largest of scale * sum |q k| over the
    keys a row sees (both for error bounds)."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    H, Tq, d = q.shape
    g = H // k.shape[0]
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    o, w = np.full((H, Tq, d), np.nan), np.full((H, Tq, d), np.nan)
    lse, spread = np.full((H, Tq), np.nan), np.full((H, Tq), np.nan)
    for s in range(len(q_start) - 1):
        a, b, ka, kb = q_start[s], q_start[s + 1], k_start[s], k_start[s + 1]
        nq, nk = b - a, kb - ka
        for i in range(nq):
            n = max(0, min(nk, i + nk - nq + 1)) if causal else nk
            for h in range(H):
                if n == 0:
                    o[h, a + i], w[h, a + i], lse[h, a + i], spread[h, a + i] = 0, 0, -np.inf, 0
                    continue
                kk, vv = k[h // g, ka:ka + n], v[h // g, ka:ka + n]
                z = scale * (kk @ q[h, a + i])
                m = z.max()
                e = np.exp(z - m)
                lse[h, a + i] = m + np.log(e.sum())
                e /= e.sum()
                o[h, a + i], w[h, a + i] = e @ vv, e @ np.abs(vv)
                spread[h, a + i] = scale * (np.abs(kk) @ np.abs(q[h, a + i])).max()
    return o, lse, w, spread


def adapted_projection(x, w, bias, start, which, down, up, scale):
    """x w^T + bias + scale_a (x down_a^T) up_a^T for rows x [M, in]; segment s holds rows start[s] .. start[s + 1] - 1
    and takes adapter a = which[s] (none if negative). Also the sums of absolute products (for error bounds): of the
    projection, and of the adapters with every sum inside taken over absolute values."""
    x, w, down, up = (np.asarray(t, dtype=np.float64) for t in (x, w, down, up))
    y, size = x @ w.T, np.abs(x) @ np.abs(w).T
    extra = np.zeros_like(y)
    if bias is not None:
        y = y + np.asarray(bias, dtype=np.float64)
    for s, a in enumerate(which):
        if a < 0:
            continue
        r = slice(start[s], start[s + 1])
        y[r] += float(scale[a]) * ((x[r] @ down[a].T) @ up[a].T)
        extra[r] = abs(float(scale[a])) * ((np.abs(x[r]) @ np.abs(down[a]).T) @ np.abs(up[a]).T)
    return y, size, extra
