"""The state space layers' operators from their definitions, token by token in
fp64 numpy, with the error bounds that the fp32 kernels have to meet.

A kernel's value is compared elementwise with bound = (rounding of the output
dtype) * |value| + (a count of fp32 roundings) * 2^-24 * (the same sums taken
over magnitudes).  The counts: a step of the scan rounds the exponent's
argument, its ex2 (2^-22), one product and one fma, fewer than 8 units in all,
so a state of `len` tokens is within (8 len + 64) units of its sum of
magnitudes, 64 covering the time step's softplus, the argument's rounding over
a contribution's whole decay (it is gone after exp(-20)) and the carried
factors of a split segment.
"""
import numpy as np

U32 = 2.0 ** -24
U_OUT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def silu(v):
    return v / (1.0 + np.exp(-v))


def softplus(v):
    return np.logaddexp(0.0, v)


def conv(x, weight, bias, cu, pool, slots, act, out="f32", commit=None, ckpt=None, every=0,
         start=None):
    """y, its bound, and the pool after; x [N][D], pool [P][W - 1][D] fp64."""
    N, D = x.shape
    W = weight.shape[1]
    y, tol = np.zeros((N, D)), np.zeros((N, D))
    pool = pool.copy()
    new = pool.copy()
    for i in range(len(cu) - 1):
        b, e = int(cu[i]), int(cu[i + 1])
        u = np.concatenate([pool[slots[i]], x[b:e]])
        for t in range(e - b):
            v = (u[t:t + W] * weight.T).sum(0)
            mag = np.abs(u[t:t + W] * weight.T).sum(0)
            if bias is not None:
                v, mag = v + bias, mag + np.abs(bias)
            err = (W + 2) * U32 * mag
            if act:
                err = 1.1 * err + (np.abs(v) + 8) * U32 * np.abs(silu(v))
                v = silu(v)
            y[b + t], tol[b + t] = v, err + U_OUT[out] * np.abs(v)
            if ckpt is not None:
                p0 = 0 if start is None else int(start[i])
                m = (p0 + t + 1) // every - p0 // every - 1
                if (p0 + t + 1) % every == 0 and m < ckpt.shape[1] and ckpt[i, m] >= 0:
                    new[ckpt[i, m]] = u[t + 1:t + W]
        keep = e - b if commit is None else int(commit[i])
        if keep > 0:
            new[slots[i]] = u[keep:keep + W - 1]
    return y, tol, new


def scan(x, dt, A, B, C, D, z, dt_bias, cu, pool, slots, softplus_on=True, out="f32",
         commit=None, ckpt=None, every=0, start=None):
    """y, its bound, the pool after and its bound (all fp64)."""
    N, Dm = x.shape
    G = B.shape[1]
    rep = Dm // G
    y, tol = np.zeros((N, Dm)), np.zeros((N, Dm))
    new, new_tol = pool.copy(), np.zeros_like(pool)
    for i in range(len(cu) - 1):
        b, e = int(cu[i]), int(cu[i + 1])
        h = pool[slots[i]].copy()
        mag = np.abs(h)
        keep = e - b if commit is None else int(commit[i])
        for t in range(e - b):
            r = b + t
            v = dt[r] + (0.0 if dt_bias is None else dt_bias)
            delta = softplus(v) if softplus_on else v
            a = np.exp(delta[:, None] * A)
            Bt, Ct = np.repeat(B[r], rep, 0), np.repeat(C[r], rep, 0)
            h = a * h + (delta * x[r])[:, None] * Bt
            mag = a * mag + np.abs((delta * x[r])[:, None] * Bt)
            units = (8 * (t + 1) + 64) * U32
            o, om = (Ct * h).sum(1), (np.abs(Ct) * mag).sum(1)
            if D is not None:
                o, om = o + D * x[r], om + np.abs(D * x[r])
            err = units * om
            if z is not None:
                g = silu(z[r])
                err = err * np.abs(g) + (np.abs(z[r]) + 8) * U32 * np.abs(o * g)
                o = o * g
            y[r], tol[r] = o, err + U_OUT[out] * np.abs(o)
            if ckpt is not None:
                p0 = 0 if start is None else int(start[i])
                m = (p0 + t + 1) // every - p0 // every - 1
                if (p0 + t + 1) % every == 0 and m < ckpt.shape[1] and ckpt[i, m] >= 0:
                    new[ckpt[i, m]], new_tol[ckpt[i, m]] = h, units * mag
            if t + 1 == keep:
                new[slots[i]], new_tol[slots[i]] = h, units * mag
    return y, tol, new, new_tol


def moves(arrays, src, dst):
    """Every array [P][...] after the moves, all at once."""
    out = []
    for a in arrays:
        new = a.copy()
        for s, d in zip(src, dst):
            if d >= 0:
                new[d] = a[s] if s >= 0 else 0
        out.append(new)
    return out
