"""Linear attention with one decay per head and layer norm in 64 bits, straight
from the recurrences (numpy), with the sums of absolute values that the error
bounds of the tests are stated in."""
import numpy as np


def bf16(x):
    """Round to bf16 (nearest even), as float64 values."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


def _heads(x, H):
    return np.repeat(x, H // x.shape[2], axis=2)


def scan(q, k, v, log_decay, s0=None, scale=1.0, lengths=None):
    """(o [B, L, H, Dv], s [B, H, Dk, Dv]); rows at and after a length are zero."""
    H = len(log_decay)
    q, k, v = (_heads(np.asarray(x, np.float64), H) for x in (q, k, v))
    B, L, _, Dk = q.shape
    Dv = v.shape[-1]
    g = np.exp(np.asarray(log_decay, np.float64))[:, None, None]
    n = np.full(B, L) if lengths is None else np.clip(lengths, 0, L)
    s = np.zeros((B, H, Dk, Dv)) if s0 is None else np.array(s0, np.float64)
    o = np.zeros((B, L, H, Dv))
    for t in range(L):
        on = t < n
        if not on.any():
            break
        s[on] = g * s[on] + k[on, t][..., :, None] * v[on, t][..., None, :]
        o[on, t] = scale * np.einsum("bhi,bhij->bhj", q[on, t], s[on])
    return o, s


def backward(q, k, v, log_decay, do, s0=None, ds=None, scale=1.0, lengths=None):
    """(dq, dk, dv summed over shared heads, ds0)."""
    H = len(log_decay)
    Hq, Hk, Hv = q.shape[2], k.shape[2], v.shape[2]
    q, k, v = (_heads(np.asarray(x, np.float64), H) for x in (q, k, v))
    do = np.asarray(do, np.float64)
    B, L, _, Dk = q.shape
    Dv = v.shape[-1]
    g = np.exp(np.asarray(log_decay, np.float64))[:, None, None]
    n = np.full(B, L) if lengths is None else np.clip(lengths, 0, L)
    dq, dk, dv = np.zeros((B, L, H, Dk)), np.zeros((B, L, H, Dk)), np.zeros((B, L, H, Dv))
    s = np.zeros((B, H, Dk, Dv)) if s0 is None else np.array(s0, np.float64)
    for t in range(L):
        on = t < n
        s[on] = g * s[on] + k[on, t][..., :, None] * v[on, t][..., None, :]
        dq[on, t] = scale * np.einsum("bhj,bhij->bhi", do[on, t], s[on])
    d = np.zeros((B, H, Dk, Dv)) if ds is None else np.array(ds, np.float64)
    for t in reversed(range(L)):
        on = t < n
        r = d[on] + scale * q[on, t][..., :, None] * do[on, t][..., None, :]
        dk[on, t] = np.einsum("bhj,bhij->bhi", v[on, t], r)
        dv[on, t] = np.einsum("bhi,bhij->bhj", k[on, t], r)
        d[on] = g * r

    def group(x, h):
        return x.reshape(B, L, h, H // h, x.shape[-1]).sum(3)

    return group(dq, Hq), group(dk, Hk), group(dv, Hv), d


def layer_norm(x, w=None, b=None, eps=1e-5):
    x = np.asarray(x, np.float64)
    mean = x.mean(-1)
    rstd = 1 / np.sqrt(((x - mean[..., None]) ** 2).mean(-1) + eps)
    y = (x - mean[..., None]) * rstd[..., None]
    y = y * (1 if w is None else w) + (0 if b is None else b)
    return y, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, w=None):
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    r = np.asarray(rstd, np.float64)[..., None]
    xh = (x - np.asarray(mean, np.float64)[..., None]) * r
    g = dy * (1 if w is None else w)
    dx = r * (g - g.mean(-1, keepdims=True) - xh * (g * xh).mean(-1, keepdims=True))
    lead = tuple(range(x.ndim - 1))
    return dx, (dy * xh).sum(lead), dy.sum(lead)
