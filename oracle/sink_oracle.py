"""Float64 oracle of sliding-window attention with sinks, its gradient, and the
rotary write into a paged cache.

Mask: the query at position t sees key j iff j <= t and (j > t - window or
j < n_sink).  Everything is dense NumPy over one sequence and one head at a time;
it shares no code with the library.

Next to each result stands a bound on what a kernel with bf16 operands may be
off: U = 2^-8 is half a step of bf16 relative to the value, so a rounded output y
is off by U |y|, and a sum whose weights were rounded to bf16 by U times the sum
of the absolute terms.  W = 2^-13 covers the 32-bit work on a weight p, relative
to p: a score is a sum of hd exact products, off by at most hd 2^-24 sum |q||k|
scale, and e^score is off by as much relatively; the exponential and its argument
add a few 2^-23 of the score.  score_slack() is the larger part, and the tests
hold their inputs to score_slack() <= 0.8 W.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -8   # bf16: eps / 2
W = 2.0 ** -13  # 32-bit work, relative to the sum of absolute terms


def score_slack(q, k, scale: float) -> float:
    """Bound of the 32-bit error of the scores of any row of q and any of k."""
    hd = q.shape[-1]
    a, b = np.abs(q).reshape(-1, hd), np.abs(k).reshape(-1, hd)
    return hd * 2.0 ** -24 * float((a @ b.T).max()) * scale


def mask(t, j, window: int, n_sink: int):
    """[len(t), len(j)] truth values."""
    t, j = np.asarray(t)[:, None], np.asarray(j)[None]
    return (j <= t) & ((j > t - window) | (j < n_sink))


def attend(q, k, v, t, j, window: int, n_sink: int, scale: float):
    """One head: q [m, hd] at positions t, k and v [n, hd] at positions j.
    Returns (o, lse, p, bound of o)."""
    see = mask(t, j, window, n_sink)
    s = np.where(see, q @ k.T * scale, -np.inf)
    top = s.max(-1, keepdims=True)
    e = np.exp(s - top)
    l = e.sum(-1, keepdims=True)
    p = e / l
    v = np.where(see.any(0)[:, None], v, 0.0)  # a row that nobody sees has no part
    o = p @ v
    return o, (top + np.log(l))[:, 0], p, U * np.abs(o) + (U + W) * (p @ np.abs(v))


def sink_window_attention(q, k, v, window: int, n_sink: int, scale: float):
    """q [B, T, Hq, hd], k and v [B, T, Hkv, hd] -> (o, lse [B, Hq, T], bound of o)."""
    B, T, Hq, hd = q.shape
    G = Hq // k.shape[2]
    o, bound = np.empty_like(q), np.empty_like(q)
    lse = np.empty((B, Hq, T))
    t = np.arange(T)
    for b in range(B):
        for h in range(Hq):
            o[b, :, h], lse[b, h], _, bound[b, :, h] = attend(
                q[b, :, h], k[b, :, h // G], v[b, :, h // G], t, t, window, n_sink, scale)
    return o, lse, bound


def sink_window_attention_vjp(q, k, v, d_o, window: int, n_sink: int, scale: float):
    """Gradients {dq, dk, dv} and their bounds {dq, dk, dv} for dL/do = d_o.

    dv = P^T dO with P rounded;  ds = p (dp - delta) scale rounded, where delta
    may come from an o that is off by its own bound."""
    B, T, Hq, hd = q.shape
    G = Hq // k.shape[2]
    g = {"dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v)}
    e = {n: np.zeros_like(x) for n, x in g.items()}
    t = np.arange(T)
    for b in range(B):
        for h in range(Hq):
            qh, kh, vh, do = q[b, :, h], k[b, :, h // G], v[b, :, h // G], d_o[b, :, h]
            o, _, p, eo = attend(qh, kh, vh, t, t, window, n_sink, scale)
            dp = do @ vh.T
            delta = (do * o).sum(-1, keepdims=True)
            ds = p * (dp - delta) * scale
            g["dq"][b, :, h] = ds @ kh
            g["dk"][b, :, h // G] += ds.T @ qh
            g["dv"][b, :, h // G] += p.T @ do
            # |error of ds|: its rounding, that of delta, and 32-bit work on the parts
            e_delta = (np.abs(do) * eo).sum(-1, keepdims=True)
            eds = U * np.abs(ds) + p * e_delta * scale + W * p * scale * (
                np.abs(do) @ np.abs(vh).T + (np.abs(do) * np.abs(o)).sum(-1, keepdims=True))
            e["dq"][b, :, h] = eds @ np.abs(kh)
            e["dk"][b, :, h // G] += eds.T @ np.abs(qh)
            e["dv"][b, :, h // G] += (U + W) * (p.T @ np.abs(do))
    for n in g:
        e[n] = e[n] * (1 + U) + U * np.abs(g[n])
    return g, e


def rotate(x, pos, theta: float):
    """Rotate-half rotary positions of x [n, H, hd] at positions pos [n]."""
    hd = x.shape[-1]
    z = x[..., :hd // 2] + 1j * x[..., hd // 2:]
    i = np.arange(hd // 2)
    z = z * np.exp(1j * np.asarray(pos, np.float64)[:, None] * theta ** (-2.0 * i / hd))[:, None]
    return np.concatenate([z.real, z.imag], -1)
