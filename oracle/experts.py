"""The routed experts' products outside FP8 in float64, row by group, from their
definitions: grouped linear and gated linear with their gradients, the 8-bit
integer forms, the router logits' gradient, and the experts' whole pass.

    grouped_linear  y[r] = x[rows[r]] W_g^T
    grouped_gated   [g | u] = x[rows[r]] W13_g^T,  a[r] = s[r] act(g) u
    quant_int8      s = fl32(max |x| / 127) or 1,  q = nearest(fl32(x / s))
    int8            the same products of q times both operands' scales

Rows outside every group are NaN in results per row.  A source index outside the
source reads as zeros.
"""

import numpy as np

from . import dense as od


def _f64(a):
    return None if a is None else np.asarray(a, np.float64)


def take(x, rows):
    """Rows of x by index; outside: zeros."""
    x = _f64(x)
    if rows is None:
        return x
    rows = np.asarray(rows, np.int64)
    out = np.zeros((rows.size, x.shape[1]))
    ok = (rows >= 0) & (rows < x.shape[0])
    out[ok] = x[rows[ok]]
    return out


def spans(offsets, R):
    """(group, first row, end)."""
    if offsets is None:
        return [(0, 0, R)]
    o = [int(v) for v in offsets]
    return [(g, o[g], o[g + 1]) for g in range(len(o) - 1)]


def grouped_linear(x, w, offsets, rows=None):
    x, w = take(x, rows), _f64(w)
    y = np.full((x.shape[0], w.shape[1]), np.nan)
    for g, b, e in spans(offsets, x.shape[0]):
        y[b:e] = x[b:e] @ w[g].T
    return y


def grouped_linear_backward(dy, x, w, offsets, rows=None, dy_rows=None):
    """(dx per row, dw)."""
    dy, x, w = take(dy, dy_rows), take(x, rows), _f64(w)
    dx, dw = np.full(x.shape, np.nan), np.zeros(w.shape)
    for g, b, e in spans(offsets, x.shape[0]):
        dx[b:e] = dy[b:e] @ w[g]
        dw[g] = dy[b:e].T @ x[b:e]
    return dx, dw


def grouped_gated_linear(x, w13, offsets, kind="silu", rows=None, scale=None):
    """(a, h)."""
    h = grouped_linear(x, w13, offsets, rows)
    i = h.shape[1] // 2
    s = 1.0 if scale is None else _f64(scale)[:, None]
    return s * od.act(kind, h[:, :i]) * h[:, i:], h


def grouped_gated_linear_backward(da, x, w13, h, offsets, kind="silu", rows=None, scale=None):
    """(dx per row, dw13, dscale, dh)."""
    da, h = _f64(da), _f64(h)
    i = h.shape[1] // 2
    g, u = h[:, :i], h[:, i:]
    s = 1.0 if scale is None else _f64(scale)[:, None]
    f = od.act(kind, g)
    dh = s * np.concatenate([da * u * od.act_grad(kind, g), da * f], axis=1)
    dx, dw = grouped_linear_backward(dh, x, w13, offsets, rows)
    return dx, dw, (da * f * u).sum(axis=1), dh


def quant_int8(x):
    """(codes as float64, scales float32); a row that is not finite: codes 0,
    scale NaN."""
    x = np.asarray(x, np.float32)
    fine = np.isfinite(x).all(axis=1)
    amax = np.abs(np.where(fine[:, None], x, np.float32(0))).max(axis=1)
    s = (amax / np.float32(127)).astype(np.float32)
    s = np.where(s == 0, np.float32(1), s)
    q = np.clip(np.rint((x[fine] / s[fine, None]).astype(np.float32)), -127, 127)
    codes = np.zeros(x.shape)
    codes[fine] = q
    return codes, np.where(fine, s, np.float32(np.nan))


def int8_linear(q, qs, w, ws, offsets, rows=None):
    """(y, the exact sums)."""
    total = grouped_linear(q, w, offsets, rows)
    s = take(_f64(qs)[:, None], rows)
    y = np.full(total.shape, np.nan)
    for g, b, e in spans(offsets, total.shape[0]):
        y[b:e] = total[b:e] * s[b:e] * _f64(ws)[g][None, :]
    return y, total


def router_backward(dgate, topk, logits):
    """dlogits, the chosen experts held fixed."""
    dgate, logits = _f64(dgate), _f64(logits)
    out = np.zeros(logits.shape)
    for t in range(logits.shape[0]):
        z = logits[t, topk[t]]
        gate = 1.0 / (1.0 + np.exp(-z))
        gate /= gate.sum()
        # dgate_k - sum_j dgate_j gate_j, and 1 - s, without cancellation
        apart = (dgate[t][:, None] - dgate[t][None, :]) @ gate
        np.add.at(out[t], topk[t], apart * gate / (1.0 + np.exp(z)))   # an expert chosen twice: both
    return out


def moe_ffn(x, w13, w2, topk, gates, kind="silu", shared=None):
    """y, token by token; shared: (w13, w2) of an expert with gate 1 or None."""
    x = _f64(x)
    y = np.zeros((x.shape[0], np.asarray(w2[0]).shape[0]))
    for t in range(x.shape[0]):
        choices = [(w13[e], w2[e], gates[t][k]) for k, e in enumerate(topk[t])]
        if shared is not None:
            choices.append((shared[0], shared[1], 1.0))
        for a13, a2, gate in choices:
            a, _ = od.gated_linear(x[t:t + 1], a13, kind)
            y[t] += float(gate) * (a @ _f64(a2).T)[0]
    return y
