"""Plain float64 definitions of the lapmix operators (include/lapmix.h), one token or
row after the other, with running bounds on what float32 evaluation may lose.

``scan`` and ``scan_backward`` work on numpy arrays [B, H, N, d]; ``norm`` and
``norm_backward`` on [rows, C].  The bounds follow the same recurrences on absolute
values: with u = 2^-24, every float32 evaluation order of h_t = f_t h_{t-1} + i_t x_t
(token by token, or tiles joined in a tree) loses at each token at most
k u (f_t M_{t-1} + |i_t x_t|), M the recurrence of |i x| and |h0|, where k u covers a gate's
relative error (the argument of exp is rounded once, |g| u, and a few roundings
follow) and the joins that a token's value passes.
"""

from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24


def gates(g, log_gate):
    """f, 1 - f and df/dg."""
    if log_gate:
        f = np.exp(np.minimum(g, 0.0))
        return f, -np.expm1(np.minimum(g, 0.0)), np.where(g > 0, 0.0, f)
    with np.errstate(over="ignore"):
        f, rest = 1.0 / (1.0 + np.exp(-g)), 1.0 / (1.0 + np.exp(g))
    return f, rest, f * rest


def _k(g):
    """Local roundings at a token in units of u: the gate's, and 64 for products, sums and joins."""
    return 64.0 + np.minimum(np.abs(np.where(np.isfinite(g), g, 0.0)), 104.0)


def _live(lengths, B, N):
    lens = np.full(B, N) if lengths is None else np.clip(np.asarray(lengths), 0, N)
    return (np.arange(N)[None, :] < lens[:, None])[:, None, :, None]


def scan(x, g, h0=None, lengths=None, log_gate=False, coupled=False):
    """dict of h (every token's state), y, hN and bounds e_h (of h) and e_hN."""
    B, H, N, d = x.shape
    live = _live(lengths, B, N)
    x = np.where(live, x, 0.0)
    g = np.where(live, g, 0.0)
    f, rest, _ = gates(g, log_gate)
    i = rest if coupled else np.ones_like(f)
    h = np.zeros((B, H, d)) if h0 is None else np.array(h0, dtype=np.float64)
    M, E, k = np.abs(h), np.zeros_like(h), _k(g)
    hs, es, ms = np.empty(x.shape), np.empty(x.shape), np.empty(x.shape)
    for n in range(N):
        on = live[:, :, n]
        m = f[:, :, n] * M + np.abs(i[:, :, n] * x[:, :, n])
        E = np.where(on, f[:, :, n] * E + k[:, :, n] * U32 * m, E)
        h = np.where(on, f[:, :, n] * h + i[:, :, n] * x[:, :, n], h)
        M = np.where(on, m, M)
        hs[:, :, n], es[:, :, n], ms[:, :, n] = h, E, M
    return {"h": hs, "y": np.where(live, hs, 0.0), "hN": h, "e_y": np.where(live, es, 0.0), "e_hN": E, "e_h": es}


def scan_backward(x, g, dy, h0=None, dhN=None, lengths=None, log_gate=False, coupled=False):
    """dict of dx, dg, dh0 and bounds e_dx, e_dg, e_dh0."""
    B, H, N, d = x.shape
    fwd = scan(x, g, h0, lengths, log_gate, coupled)
    live = _live(lengths, B, N)
    x, g, dy = (np.where(live, t, 0.0) for t in (x, g, dy))
    f, rest, slope = gates(g, log_gate)
    first = np.zeros((B, H, d)) if h0 is None else h0
    before = np.concatenate([first[:, :, None], fwd["h"][:, :, :-1]], axis=2)
    e_before = np.concatenate([np.zeros((B, H, 1, d)), fwd["e_h"][:, :, :-1]], axis=2)
    k = _k(g)
    r = np.zeros((B, H, d)) if dhN is None else np.array(dhN, dtype=np.float64)
    M, E = np.abs(r), np.zeros_like(r)
    out = {n: np.zeros(x.shape) for n in ("dx", "dg", "e_dx", "e_dg")}
    for n in range(N - 1, -1, -1):
        at = (slice(None), slice(None), n)
        on = live[:, :, n]
        dh, mh = dy[at] + r, np.abs(dy[at]) + M
        eh = E + k[at] * U32 * mh
        i = rest[at] if coupled else 1.0
        diff = before[at] - (x[at] if coupled else 0.0)
        size = np.abs(before[at]) + (np.abs(x[at]) if coupled else 0.0)
        dg = dh * diff * slope[at]
        e_dg = slope[at] * (eh * np.abs(diff) + np.abs(dh) * (e_before[at] + 2 * U32 * size)) + k[at] * U32 * np.abs(dg)
        for name, v in (("dx", dh * i), ("e_dx", eh * i + k[at] * U32 * np.abs(dh * i)), ("dg", dg), ("e_dg", e_dg)):
            out[name][at] = np.where(on, v, 0.0)
        r = np.where(on, f[at] * dh, r)
        M = np.where(on, f[at] * mh, M)
        E = np.where(on, f[at] * eh + k[at] * U32 * f[at] * mh, E)
    out["dh0"], out["e_dh0"] = r, E
    return out


def rows_of(x):
    """[B, H, N, d] as token rows [B * N, H * d]."""
    B, H, N, d = x.shape
    return np.ascontiguousarray(x.transpose(0, 2, 1, 3)).reshape(B * N, H * d)


def norm(s, w, eps):
    """y of the stored sum s, and the bound e_y: a row's sum of squares is a sum of C / 64 + 16
    levels at most, whose relative error the root halves, and a handful of roundings follow."""
    C = s.shape[1]
    rstd = 1.0 / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    y = s * rstd * w
    return y, np.abs(y) * U32 * ((C / 64 + 16) / 2 + 8)


def norm_backward(dy, s, w, eps, ds=None):
    """dr, dw and bounds e_dr, e_dw."""
    R, C = s.shape
    rstd = 1.0 / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    u, wdy = s * rstd, w * dy
    dr = rstd * (wdy - u * (wdy * u).mean(1, keepdims=True))
    depth = C / 64 + 16
    e = rstd * U32 * (2 * depth + 16) * (np.abs(wdy) + np.abs(u) * np.abs(wdy * u).mean(1, keepdims=True))
    if ds is not None:
        e = e + U32 * (np.abs(dr) + np.abs(ds))
        dr = dr + ds
    # dw: each slice of rows one after the other, then the slices (at most R terms in a chain)
    return dr, (dy * u).sum(0), e, np.abs(dy * u).sum(0) * U32 * (R + depth + 16)


def e4m3_half_step(v):
    """Half the distance of neighbouring e4m3 values around |v| <= 448."""
    _, e = np.frexp(np.abs(v))
    return np.exp2(np.maximum(e - 1, -6) - 4.0)
