"""The operators around the linear layer in a fine-tuning step, on the host in
64 bits (numpy), from their definitions: layer norm, causal attention over packed
sequences, token log-probabilities, AdamW.  AdamW's states are also given in the library's stated IEEE fp32 steps
(8-bit codes and scales are a bit-exact contract)."""
from __future__ import annotations

import numpy as np

F32 = np.float32


def layernorm(x, w=None, b=None, eps=1e-5):
    """(y, mean, rstd) over the rows of x, fp64."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(1)
    dev = x - mean[:, None]
    rstd = 1.0 / np.sqrt((dev * dev).mean(1) + eps)
    y = dev * rstd[:, None]
    if w is not None:
        y = y * np.asarray(w, dtype=np.float64)
    if b is not None:
        y = y + np.asarray(b, dtype=np.float64)
    return y, mean, rstd


def layernorm_backward(x, dy, mean, rstd, w=None):
    """(dx, dw, db), fp64, at the given row statistics."""
    x, dy = np.asarray(x, dtype=np.float64), np.asarray(dy, dtype=np.float64)
    mean, rstd = (np.asarray(t, dtype=np.float64)[:, None] for t in (mean, rstd))
    hat = (x - mean) * rstd
    g = dy if w is None else dy * np.asarray(w, dtype=np.float64)
    dx = rstd * (g - g.mean(1, keepdims=True) - hat * (g * hat).mean(1, keepdims=True))
    return dx, (dy * hat).sum(0), dy.sum(0)


def attention(q, k, v, starts, scale, dout=None):
    """Causal attention over the sequences starts[s] .. starts[s + 1]: (o [T, H, D], lse [H, T]) and,
    with dout, (dq, dk, dv), fp64.  Rows of no sequence: o = 0, lse = -inf, no gradient."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    rows, heads, _ = q.shape
    group = heads // k.shape[1]
    o, lse = np.zeros_like(q), np.full((heads, rows), -np.inf)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for a, b in zip(starts[:-1], starts[1:]):
        if b <= a:
            continue
        later = np.triu(np.ones((b - a, b - a), dtype=bool), 1)
        for h in range(heads):
            g = h // group
            s = np.where(later, -np.inf, scale * q[a:b, h] @ k[a:b, g].T)
            m = s.max(1, keepdims=True)
            e = np.exp(s - m)
            total = e.sum(1, keepdims=True)
            p = e / total
            lse[h, a:b] = (m + np.log(total))[:, 0]
            o[a:b, h] = p @ v[a:b, g]
            if dout is not None:
                do = np.asarray(dout[a:b, h], dtype=np.float64)
                dp = do @ v[a:b, g].T
                ds = scale * p * (dp - (p * dp).sum(1, keepdims=True))
                dq[a:b, h] = ds @ k[a:b, g]
                dk[a:b, g] += ds.T @ q[a:b, h]
                dv[a:b, g] += p.T @ do
    return (o, lse) if dout is None else (o, lse, dq, dk, dv)


def _log_softmax(row):
    """log p of one row by the deviations from its maximum (a row of very large
    logits keeps the digits of log l), and the row's maximum and log l."""
    m = row.max()
    if m == -np.inf:
        return np.full(row.size, -np.inf), m, 0.0
    with np.errstate(over="ignore"):
        d = row - m
    log_l = np.log(np.exp(d).sum())
    return d - log_l, m, log_l


def logprob(x, targets, top=0):
    """(logp, entropy, lse, top_logp, top_ids), fp64: -inf logits are ruled out, equal
    logits ordered by index, targets outside [0, V) give 0."""
    x = np.asarray(x, dtype=np.float64)
    rows, v = x.shape
    lse, entropy, logp = np.zeros(rows), np.zeros(rows), np.zeros(rows)
    top_logp, top_ids = np.zeros((rows, top)), np.zeros((rows, top), dtype=np.int32)
    for i in range(rows):
        lp, m, log_l = _log_softmax(x[i])
        lse[i] = m + log_l
        live = lp[lp > -np.inf]
        entropy[i] = -(np.exp(live) * live).sum()
        if 0 <= targets[i] < v:
            logp[i] = lp[targets[i]]
        order = np.argsort(-x[i], kind="stable")[:top]
        top_ids[i], top_logp[i] = order, lp[order]
    return logp, entropy, lse, top_logp, top_ids


def logprob_backward(x, targets, dlogp, dentropy=None):
    """dlogits, fp64."""
    x = np.asarray(x, dtype=np.float64)
    rows, v = x.shape
    out = np.zeros((rows, v))
    for i in range(rows):
        lp, m, _ = _log_softmax(x[i])
        if m == -np.inf:
            continue
        live = lp > -np.inf
        p, lp = np.exp(lp[live]), lp[live]
        has = 0 <= targets[i] < v
        d = -(float(dlogp[i]) if has else 0.0) * p
        if dentropy is not None:
            d = d - float(dentropy[i]) * p * (lp - (p * lp).sum())
        out[i][live] = d
        if has:
            out[i][targets[i]] += float(dlogp[i])
    return out


BLOCK = 256


def _blocks(x):
    n = x.size
    full = np.zeros(-(-n // BLOCK) * BLOCK, dtype=x.dtype)
    full[:n] = x
    return full.reshape(-1, BLOCK), n


def decode_m(codes, scales):
    c, n = _blocks(codes.astype(F32))
    return (c * np.abs(c) * scales[:, None]).reshape(-1)[:n]


def decode_v(codes, scales):
    c, n = _blocks(codes.astype(F32))
    return ((c * c) * (c * c) * scales[:, None]).reshape(-1)[:n]


def _scaled(x, top):
    """The blocks' scales and |x| over them, each operation rounded to fp32."""
    b, n = _blocks(np.abs(x.astype(F32)))
    with np.errstate(divide="ignore", over="ignore", invalid="ignore", under="ignore"):
        s = (b.max(1) * (F32(1) / F32(top))).astype(F32)
        s = np.where(s >= F32(2.0 ** -126), s, F32(0))
        inv = np.where(s > 0, F32(1) / s, F32(0)).astype(F32)
        return s, (b * inv[:, None]).astype(F32).reshape(-1)[:n]


def encode_m(m):
    s, t = _scaled(m, 127.0 ** 2)
    c = np.minimum(np.rint(np.sqrt(t)), 127)
    return (c * np.sign(m)).astype(np.int8), s


def encode_v(v):
    s, t = _scaled(v, 255.0 ** 4)
    c = np.minimum(np.rint(np.sqrt(np.sqrt(t))), 255)
    some = (v > 0) & (np.repeat(s, BLOCK)[:v.size] > 0)
    return np.where(some, np.maximum(c, 1), c).astype(np.uint8), s


def adamw_states(m, v, g, beta1, beta2, grad_scale=1.0):
    """The new fp32 m and v, each operation rounded to fp32."""
    g = g.astype(F32) * F32(grad_scale)
    m = m * F32(beta1) + g * F32(1.0 - beta1)
    v = v * F32(beta2) + (g * g) * F32(1.0 - beta2)
    return m, v


def adamw_param(p, m, v, lr, beta1, beta2, eps, weight_decay, step):
    """The new weights, fp64, from the new states."""
    p, m, v = (np.asarray(t, dtype=np.float64) for t in (p, m, v))
    mh, vh = m / (1 - beta1 ** step), v / (1 - beta2 ** step)
    return p * (1 - lr * weight_decay) - lr * mh / (np.sqrt(vh) + eps)
