"""Inputs of a sink-window backward on which the roundings of one sink add up.

All queries are the same, and so are all output gradients.  Key 0, the sink, has the
weight p0 just below the middle between two bf16 numbers for every query from `window`
on; the other keys and their values are 0.  Rounding P to bf16 once puts the same error,
up to U, into every term of dv of the sink; the rounded o is off by as much in every
element, and with it a delta that is formed from it; dS of the sink is the same number
in every row too.  What has none of these errors is off by

  dv_0   U |dv_0| + (U^2 + W) sum_t p_t0 |dO_t|
  dk_0   U |dk_0| + sum_t e_t |q_t|,  e_t = U^2 |ds_t0| + W scale p_t0 (|dO_t| |v_0| + |dO_t| |o_t|)
  dq_t   U |dq_t| + e_t |k_0|

at most: the results' own roundings, P and dS in 16 bits (two bf16 each), and 32-bit
work, with U and W of the oracle.  The keys beside the sink add nothing to dq."""
import numpy as np
import torch

from oracle import sink_oracle as so

WINDOW = 40


def bf16(x):
    return torch.as_tensor(x, dtype=torch.float64).bfloat16()


def inputs(hd, T, Hq, seed):
    """q, k, v, d_o as bf16 tensors of a batch of one."""
    g = np.random.default_rng(seed)
    p0 = 0.5 + 2.0 ** -9 - 2.0 ** -13
    s0 = np.log(p0 / (1 - p0) * WINDOW) * hd ** 0.5  # of q . k_0
    a = float(bf16(s0 / 4))
    q0, k0 = np.zeros(hd), np.zeros(hd)
    q0[:2], k0[:2] = (4.0, 0.25), (a, float(bf16((s0 - 4 * a) / 0.25)))
    q0[2:hd // 2] = g.standard_normal(hd // 2 - 2)
    k0[hd // 2:] = g.standard_normal(hd - hd // 2)
    q = bf16(np.broadcast_to(q0, (1, T, Hq, hd)).copy())
    k, v = (torch.zeros(1, T, 1, hd, dtype=torch.bfloat16) for _ in range(2))
    k[0, 0, 0], v[0, 0, 0] = bf16(k0), 1.0
    # dS of the sink near the middle between two bf16 numbers as well
    for _ in range(1000):
        d = bf16(0.5 + np.abs(g.standard_normal(hd)))
        ds = p0 * (1 - p0) * float(d.double().sum())
        if abs(float(bf16(ds)) / ds - 1) > 0.8 * so.U:
            break
    else:
        raise AssertionError("no such gradient")
    return q, k, v, d[None, None, None].expand(1, T, Hq, hd).contiguous()


def exact(q, k, v, d_o, round_p=False, round_ds=False, round_o=False):
    """dq [T, Hq, hd], dk_0 and dv_0 [hd] in 64 bits, and their bounds; with P or dS
    rounded to one bf16, or delta from the rounded o, where asked for."""
    one = lambda x: bf16(x).double().numpy()  # noqa: E731
    two = lambda x: one(x) + one(x - one(x))  # noqa: E731
    q, k, v, d_o = (x[0].double().numpy() for x in (q, k, v, d_o))
    T, Hq, hd = q.shape
    t, scale = np.arange(T), hd ** -0.5
    out = {"dq": np.zeros_like(q), "dk": np.zeros(hd), "dv": np.zeros(hd)}
    err = {n: np.zeros_like(x) for n, x in out.items()}
    for h in range(Hq):
        o, _, p, _ = so.attend(q[:, h], k[:, 0], v[:, 0], t, t, WINDOW, 1, scale)
        p, do = p[:, :1], d_o[:, h]
        assert np.all(p[WINDOW:] == p[WINDOW:WINDOW + 1]) or np.ptp(p[WINDOW:]) < 1e-12
        delta = (do * (one(o) if round_o else o)).sum(-1, keepdims=True)
        ds = p * (do @ v[:1, 0].T - delta)
        ds = (one(ds) if round_ds else two(ds)) * scale
        out["dq"][:, h] = ds * k[:1, 0]
        out["dk"] += (ds * q[:, h]).sum(0)
        out["dv"] += ((one(p) if round_p else two(p)) * do).sum(0)
        e = so.U ** 2 * np.abs(ds) + so.W * scale * p * (np.abs(do) @ np.abs(v[:1, 0]).T +
                                                         (np.abs(do) * np.abs(o)).sum(-1, keepdims=True))
        err["dq"][:, h] = e * np.abs(k[:1, 0])
        err["dk"] += (e * np.abs(q[:, h])).sum(0)
        err["dv"] += (so.U ** 2 + so.W) * (p * np.abs(do)).sum(0)
    return out, {n: err[n] * (1 + so.U) + so.U * np.abs(out[n]) for n in out}


CASES = [(64, 700, 2, 0), (128, 700, 2, 1), (64, 300, 1, 2), (128, 3000, 3, 3)]  # hd, T, Hq, seed
