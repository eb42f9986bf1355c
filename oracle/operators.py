"""fp64 CPU definitions of the layer's norms and of the operators over a state cache (test
infrastructure only): the gated norm and the residual norm with their gradients, drafted trees, ragged
runs from slot to slot, and copies between slots.  Plain sequential numpy; nothing of the CUDA path.
"""
import numpy as np


def _act(gate, act):
    s = 1.0 / (1.0 + np.exp(-gate))
    return (gate * s, s + gate * s * (1.0 - s)) if act == "silu" else (s, s * (1.0 - s))


def gated_norm(o, gate, weight, act="silu", eps=1e-6):
    """y = o / sqrt(mean(o^2) + eps) * weight * act(gate)."""
    o, gate, weight = (np.asarray(x, np.float64) for x in (o, gate, weight))
    return o / np.sqrt((o * o).mean(-1, keepdims=True) + eps) * weight * _act(gate, act)[0]


def gated_norm_backward(o, gate, weight, dy, act="silu", eps=1e-6):
    """(do, dgate, dweight) of sum(dy * gated_norm(...))."""
    o, gate, weight, dy = (np.asarray(x, np.float64) for x in (o, gate, weight, dy))
    a, slope = _act(gate, act)
    r = 1.0 / np.sqrt((o * o).mean(-1, keepdims=True) + eps)
    dn = dy * a
    do = r * dn * weight - o * r ** 3 * (dn * weight * o).mean(-1, keepdims=True)
    return do, dy * o * r * weight * slope, (dn * o * r).reshape(-1, o.shape[-1]).sum(0)


def add_norm(x, residual, scale, weight, eps=1e-6):
    """(y, h): h = residual + scale * x, y = h / sqrt(mean(h^2) + eps) * weight."""
    h = np.asarray(x, np.float64) * (1.0 if scale is None else np.asarray(scale, np.float64))
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    return h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64), h


def add_norm_backward(h, x, scale, weight, dy, dh=None, eps=1e-6):
    """(dresidual, dx, dscale, dweight) of sum(dy * y) + sum(dh * h) at the given h."""
    h, weight, dy = (np.asarray(t, np.float64) for t in (h, weight, dy))
    width = h.shape[-1]
    r = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    dres = r * dy * weight - h * r ** 3 * (dy * weight * h).mean(-1, keepdims=True)
    if dh is not None:
        dres = dres + np.asarray(dh, np.float64)
    dweight = (dy * h * r).reshape(-1, width).sum(0)
    if scale is None:
        return dres, dres, None, dweight
    scale, x = np.asarray(scale, np.float64), np.asarray(x, np.float64)
    return dres, scale * dres, (dres * x).reshape(-1, width).sum(0), dweight


def step(S, q, k, v, alpha, b, w):
    """One token of the recurrence for every head: S [H, d_k, d_v] -> (S, o)."""
    S = alpha[..., None] * S
    delta = w * v - np.einsum("hkv,hk->hv", S, b * k)
    S = S + k[..., None] * delta[:, None, :]
    return S, np.einsum("hkv,hk->hv", S, q)


def _f64(*xs):
    return [np.asarray(x, np.float64) for x in xs]


def tree(q, k, v, alpha, b, w, pool, slots, cu, parents):
    """o [total, H, d_v] of every node (zero where no tree owns the row); pool [slots, H, d_k, d_v]."""
    q, k, v, alpha, b, w, pool = _f64(q, k, v, alpha, b, w, pool)
    o = np.zeros(v.shape)
    for i in range(len(slots)):
        root = pool[slots[i]] if slots[i] >= 0 else np.zeros(pool.shape[1:])
        states = []
        for t in range(cu[i], cu[i + 1]):
            S = root if parents[t] < 0 else states[parents[t]]
            S, o[t] = step(S, q[t], k[t], v[t], alpha[t], b[t], w[t])
            states.append(S)
    return o


def recurrent(q, k, v, alpha, b, w, pool, slots_in, slots_out, cu, index=None):
    """(o [total, H, d_v], pool after the call); entries of no sequence are zero."""
    q, k, v, alpha, b, w, pool = _f64(q, k, v, alpha, b, w, pool)
    total = len(q) if index is None else len(index)
    o, after = np.zeros((total,) + v.shape[1:]), pool.copy()
    for i in range(len(slots_in)):
        S = pool[slots_in[i]] if slots_in[i] >= 0 else np.zeros(pool.shape[1:])
        for t in range(cu[i], cu[i + 1]):
            r = t if index is None else index[t]
            S, o[t] = step(S, q[r], k[r], v[r], alpha[r], b[r], w[r])
        if slots_out[i] >= 0:
            after[slots_out[i]] = S
    return o, after


def state_copy(dst, src, dst_index, src_index):
    """The destination cache after the pairs, every source read first, the last of equal destinations."""
    src, out = np.array(src), np.array(dst)
    for d, s in zip(dst_index, src_index):
        if d >= 0:
            out[d] = src[s] if s >= 0 else 0.0
    return out
