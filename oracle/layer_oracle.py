"""Float64 definitions of the operators around the recurrence, written out with plain torch
CPU operations, token by token or row by row, apart from the HIP path.  The `size` values are
sums of the absolute values of the same terms: what a rounding bound is relative to.
"""
from __future__ import annotations

import torch

F64 = torch.float64


def spans(B, T, cu=None):
    """(batch row, first token, token after the last) of each sequence."""
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    c = [int(v) for v in cu]
    return [(0, a, b) for a, b in zip(c, c[1:])]


def f64(t):
    return None if t is None else t.detach().cpu().to(F64)


def short_conv(x, weight, bias=None, silu=False, h0=None, cu=None):
    """y, final state, and the sizes and sums (pre) of the convolution."""
    x, w, bias, h0 = f64(x), f64(weight), f64(bias), f64(h0)
    B, T, D = x.shape
    W = w.shape[1]
    seqs = spans(B, T, cu)
    pre, size = torch.zeros_like(x), torch.zeros_like(x)
    last = torch.zeros(len(seqs), W - 1, D, dtype=F64)
    for n, (r, a, b) in enumerate(seqs):
        window = torch.cat([torch.zeros(W - 1, D, dtype=F64) if h0 is None else h0[n], x[r, a:b]])
        for t in range(b - a):
            terms = window[t:t + W].t() * w
            pre[r, a + t] = terms.sum(1) + (0 if bias is None else bias)
            size[r, a + t] = terms.abs().sum(1) + (0 if bias is None else bias.abs())
        last[n] = window[b - a:]
    return (pre * torch.sigmoid(pre) if silu else pre), last, pre, size


def short_conv_bwd(x, weight, dy, bias=None, silu=False, h0=None, dht=None, cu=None):
    """The gradients of <dy, y> + <dht, final state> by the chain rule, and their sizes."""
    _, _, pre, _ = short_conv(x, weight, bias, silu, h0, cu)
    x, w, dy, h0, dht = f64(x), f64(weight), f64(dy), f64(h0), f64(dht)
    B, T, D = x.shape
    W = w.shape[1]
    s = torch.sigmoid(pre)
    dpre = dy * (s * (1 + pre * (1 - s))) if silu else dy
    seqs = spans(B, T, cu)
    dx, dw, db = torch.zeros_like(x), torch.zeros_like(w), torch.zeros(D, dtype=F64)
    dh0 = torch.zeros(len(seqs), W - 1, D, dtype=F64)
    sizes = dict(dx=torch.zeros_like(x), dweight=torch.zeros_like(w), dh0=torch.zeros_like(dh0), dbias=dpre.abs().sum((0, 1)))
    for n, (r, a, b) in enumerate(seqs):
        window = torch.cat([torch.zeros(W - 1, D, dtype=F64) if h0 is None else h0[n], x[r, a:b]])
        g, m = torch.zeros_like(window), torch.zeros_like(window)
        for t in range(b - a):
            for k in range(W):
                g[t + k] += w[:, k] * dpre[r, a + t]
                m[t + k] += (w[:, k] * dpre[r, a + t]).abs()
                dw[:, k] += window[t + k] * dpre[r, a + t]
                sizes["dweight"][:, k] += (window[t + k] * dpre[r, a + t]).abs()
            db += dpre[r, a + t]
        if dht is not None:
            g[b - a:] += dht[n]
            m[b - a:] += dht[n].abs()
        dh0[n], dx[r, a:b] = g[:W - 1], g[W - 1:]
        sizes["dh0"][n], sizes["dx"][r, a:b] = m[:W - 1], m[W - 1:]
    return dict(dx=dx, dweight=dw, dbias=db, dh0=dh0), sizes


def rms_norm(h, weight, eps):
    """y from the stored sum h."""
    h, w = f64(h), f64(weight)
    return h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * w


def rms_norm_bwd(h, weight, dy, eps, dh=None):
    h, w, dy, dh = f64(h), f64(weight), f64(dy), f64(dh)
    r = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    g = dy * w
    mean, size = (g * h).mean(-1, keepdim=True), (g * h).abs().mean(-1, keepdim=True)
    dx = r * g - h * r ** 3 * mean
    dims = tuple(range(h.dim() - 1))
    sizes = dict(dx=(r * g).abs() + (h * r ** 3).abs() * size + (0 if dh is None else dh.abs()),
                 dweight=(dy * h * r).abs().sum(dims))
    return dict(dx=dx if dh is None else dx + dh, dweight=(dy * h * r).sum(dims)), sizes


def e4m3_values():
    """Every finite value of e4m3, ascending: 2^(e - 7) (1 + m / 8), subnormals m 2^-9."""
    pos = [m * 2.0 ** -9 for m in range(8)] + [2.0 ** (e - 7) * (1 + m / 8) for e in range(1, 16) for m in range(8)]
    pos = pos[:-1]  # the last code is NaN
    return torch.tensor([-v for v in pos[:0:-1]] + pos, dtype=F64)


def ssm_steps(dt, dt_bias=None, softplus=False):
    raw = f64(dt) + (0 if dt_bias is None else f64(dt_bias))
    return torch.nn.functional.softplus(raw, threshold=1e9) if softplus else raw, raw


def _ssm_rows(x, d, A, B, C, h0, cu):
    """Each sequence's tokens, with B and C for every head and its first state."""
    H, G = x.shape[2], B.shape[2]
    Bh, Ch = B.repeat_interleave(H // G, 2), C.repeat_interleave(H // G, 2)
    for n, (r, a, b) in enumerate(spans(x.shape[0], x.shape[1], cu)):
        S = torch.zeros(H, B.shape[3], x.shape[3], dtype=F64) if h0 is None else h0[n].clone()
        yield n, r, a, b, S, Bh, Ch


def ssm(x, dt, A_log, B, C, D=None, dt_bias=None, softplus=False, h0=None, cu=None, D_sign=1.0):
    """y and the final states of S_t = e^{d A} S + d B x^T, y = S^T C + D x, token by token."""
    d, _ = ssm_steps(dt, dt_bias, softplus)
    x, B, C, h0, A = f64(x), f64(B), f64(C), f64(h0), -torch.exp(f64(A_log))
    y = torch.zeros_like(x)
    n_seq = len(spans(x.shape[0], x.shape[1], cu))
    last = torch.zeros(n_seq, x.shape[2], B.shape[3], x.shape[3], dtype=F64)
    for n, r, a, b, S, Bh, Ch in _ssm_rows(x, d, A, B, C, h0, cu):
        for t in range(a, b):
            S = torch.exp(d[r, t] * A)[:, None, None] * S + d[r, t, :, None, None] * Bh[r, t][:, :, None] * x[r, t][:, None, :]
            y[r, t] = (S * Ch[r, t][:, :, None]).sum(1)
        last[n] = S
    return (y if D is None else y + f64(D)[:, None] * x), last


def ssm_bwd(x, dt, A_log, B, C, dy, dht=None, D=None, dt_bias=None, softplus=False, h0=None, cu=None):
    """The gradients of <dy, y> + <dht, final states> by the adjoint recurrence.  `dl` is the
    gradient by each decay's logarithm, `direct` the one by d through d B x^T."""
    d, raw = ssm_steps(dt, dt_bias, softplus)
    x, B, C, dy, h0, dht, A = f64(x), f64(B), f64(C), f64(dy), f64(h0), f64(dht), -torch.exp(f64(A_log))
    H, G = x.shape[2], B.shape[2]
    dx, dl, direct = torch.zeros_like(x), torch.zeros_like(d), torch.zeros_like(d)
    dBh = torch.zeros(*B.shape[:2], H, B.shape[3], dtype=F64)
    dCh = torch.zeros_like(dBh)
    dh0 = torch.zeros(len(spans(x.shape[0], x.shape[1], cu)), H, B.shape[3], x.shape[3], dtype=F64)
    for n, r, a, b, S, Bh, Ch in _ssm_rows(x, d, A, B, C, h0, cu):
        states = [S]
        for t in range(a, b):
            states.append(torch.exp(d[r, t] * A)[:, None, None] * states[-1]
                          + d[r, t, :, None, None] * Bh[r, t][:, :, None] * x[r, t][:, None, :])
        R = torch.zeros_like(S) if dht is None else dht[n].clone()
        for t in range(b - 1, a - 1, -1):
            R = R + Ch[r, t][:, :, None] * dy[r, t][:, None, :]
            dCh[r, t] = (states[t - a + 1] * dy[r, t][:, None, :]).sum(2)
            Rx, RB = (R * x[r, t][:, None, :]).sum(2), (R * Bh[r, t][:, :, None]).sum(1)
            dBh[r, t], dx[r, t] = d[r, t][:, None] * Rx, d[r, t][:, None] * RB
            direct[r, t] = (Rx * Bh[r, t]).sum(1)
            decay = torch.exp(d[r, t] * A)
            dl[r, t] = decay * (R * states[t - a]).sum((1, 2))
            R = decay[:, None, None] * R
        dh0[n] = R
    dd = (direct + dl * A) * (torch.sigmoid(raw) if softplus else 1)
    shape = (*B.shape[:3], H // G, B.shape[3])
    return dict(dx=dx if D is None else dx + f64(D)[:, None] * dy, ddt=dd, dA_log=(dl * d * A).sum((0, 1)),
                dB=dBh.reshape(shape).sum(3), dC=dCh.reshape(shape).sum(3), dD=(dy * x).sum((0, 1, 3)),
                ddt_bias=dd.sum((0, 1)), dh0=dh0, dl=dl, direct=direct)
