"""The training operators' formulas in 64 bits, in plain numpy: what the GPU tests compare with."""
import numpy as np


def embed(idx, W, scale, rows):
    idx = np.asarray(idx)
    ok = (idx >= 0) & (idx < rows)
    out = np.zeros(idx.shape + (W.shape[1],))
    out[ok] = W[idx[ok]].astype(np.float64) * np.float64(np.float32(scale))
    return out


def embed_grad(idx, dout, rows, scale):
    """(distinct row ids ascending, their sums, the sums of the magnitudes, how often each occurs)"""
    idx = np.asarray(idx).reshape(-1)
    g = np.asarray(dout, np.float64).reshape(idx.size, -1)
    ok = (idx >= 0) & (idx < rows)
    ids, which, times = np.unique(idx[ok], return_inverse=True, return_counts=True)
    s, m = np.zeros((ids.size, g.shape[1])), np.zeros((ids.size, g.shape[1]))
    np.add.at(s, which, g[ok])
    np.add.at(m, which, np.abs(g[ok]))
    f = np.float64(np.float32(scale))
    return ids, s * f, m * abs(f), times


def gate(x, kv, q, k, mask, eps):
    """out_i = h_i + gate_i * value"""
    T, hc, dim = x.shape
    kv = kv.reshape(T, hc + 1, dim)
    key, v = kv[:, :hc], kv[:, hc:]
    r = 1 / np.sqrt(((x * x).mean(-1) + eps) * ((key * key).mean(-1) + eps) * dim)
    dot = (x * q * k * key).sum(-1) * r
    z = np.copysign(np.sqrt(np.maximum(np.abs(dot), 1e-6)), dot)
    g = np.where(mask[:, None], 1 / (1 + np.exp(-z)), 0.0)
    return x + g[..., None] * v


def gate_grad(x, kv, q, k, dout, mask, eps):
    """The formula of engram_gate_grad's contract; also the scalars (ddot, dot) of every copy."""
    T, hc, dim = x.shape
    kv = kv.reshape(T, hc + 1, dim)
    key, v = kv[:, :hc], kv[:, hc:]
    A, B = (x * x).mean(-1, keepdims=True) + eps, (key * key).mean(-1, keepdims=True) + eps
    r = 1 / np.sqrt(A * B * dim)
    w = q * k
    dot = (x * w * key).sum(-1, keepdims=True) * r
    m = np.abs(dot)
    root = np.sqrt(np.maximum(m, 1e-6))
    g = 1 / (1 + np.exp(-np.copysign(root, dot)))
    ddot = (dout * v).sum(-1, keepdims=True) * g * (1 - g) * np.where(m >= 1e-6, 0.5 / root, 0.0)
    on = mask[:, None, None]
    ddot = np.where(on, ddot, 0.0)
    dx = dout + ddot * (r * w * key - dot / (A * dim) * x)
    dkey = ddot * (r * w * x - dot / (B * dim) * key)
    dv = (np.where(on, g, 0.0) * dout).sum(1, keepdims=True)
    dw = (ddot * r * x * key).sum(0)
    return dx, np.concatenate([dkey, dv], 1).reshape(T, -1), dw * k, dw * q, ddot, dot
