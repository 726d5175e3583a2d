"""Linear attention and the head norms from their definitions in fp64 numpy, with
the error bounds that the kernels have to meet.

A value is compared elementwise with bound = (rounding of the output dtype) *
|value| + (a count of fp32 roundings) * 2^-24 * (the same sums taken over
magnitudes).  The counts for linear attention: a token's step rounds its decay,
a product and two fmas, at most 4 units; 64 cover a decay over many tokens taken
as one exponent (an argument of up to 24 rounded, then it has nothing left to
weigh) and the halves of split operands.  An output adds a sum over d_k products
(d_k units).  Where the tensor cores take the state as bf16 the outputs have its
rounding, 2^-8, over the magnitudes of the sum besides.
"""
import numpy as np

U32 = 2.0 ** -24
U_OUT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def linear(q, k, v, g, cu, pool, slots, scale=1.0, out="f32", rounded_state=False, commit=None,
           ckpt=None, every=0, start=None):
    """o, its bound, the pool after and its bound; q, k [N][Hk][dk], v [N][H][dv],
    g [N][H], pool [P][H][dv][dk], all fp64."""
    N, H, dv = v.shape
    rep, dk = H // q.shape[1], q.shape[2]
    q, k = np.repeat(q, rep, 1), np.repeat(k, rep, 1)
    o, tol = np.zeros((N, H, dv)), np.zeros((N, H, dv))
    new, new_tol = pool.copy(), np.zeros_like(pool)
    for i in range(len(cu) - 1):
        b, e = int(cu[i]), int(cu[i + 1])
        S = pool[slots[i]].copy()
        mag = np.abs(S)
        keep = e - b if commit is None else int(commit[i])
        for t in range(e - b):
            r = b + t
            a = np.exp(g[r])[:, None, None]
            kv = v[r][:, :, None] * k[r][:, None, :]
            S = a * S + kv
            mag = a * mag + np.abs(kv)
            units = (4 * (t + 1) + 64) * U32
            o[r] = scale * (S * q[r][:, None, :]).sum(-1)
            om = abs(scale) * (mag * np.abs(q[r])[:, None, :]).sum(-1)
            tol[r] = (units + dk * U32 + (U_OUT["bf16"] if rounded_state else 0)) * om
            tol[r] += U_OUT[out] * np.abs(o[r])
            if ckpt is not None:
                p0 = 0 if start is None else int(start[i])
                m = (p0 + t + 1) // every - p0 // every - 1
                if (p0 + t + 1) % every == 0 and m < ckpt.shape[1] and ckpt[i, m] >= 0:
                    new[ckpt[i, m]], new_tol[ckpt[i, m]] = S, units * mag
            if t + 1 == keep:
                new[slots[i]], new_tol[slots[i]] = S, units * mag
    return o, tol, new, new_tol


def head_norm(x, weight, norm, eps):
    """Norm and weight over the last axis; the roundings: d for the sum, halved by
    the root, one each for the quotient, root, products (8 in all)."""
    d = x.shape[-1]
    y = x
    if norm is not None:
        total = (x * x).sum(-1, keepdims=True)
        y = x / np.sqrt((total / d if norm == "rms" else total) + eps)
    return y if weight is None else y * weight


def rotate(y, table, pos, interleaved):
    """The rotated channels, and the magnitudes of their sums."""
    rot = table.shape[1]
    c, s = table[pos][:, None, :rot // 2], table[pos][:, None, rot // 2:]
    out, mag = y.copy(), np.abs(y)
    a, b = ((slice(0, rot, 2), slice(1, rot, 2)) if interleaved
            else (slice(0, rot // 2), slice(rot // 2, rot)))
    ya, yb = y[..., a], y[..., b]
    out[..., a], out[..., b] = ya * c - yb * s, yb * c + ya * s
    mag[..., a] = np.abs(ya * c) + np.abs(yb * s)
    mag[..., b] = np.abs(yb * c) + np.abs(ya * s)
    return out, mag


def qk_norm(x, weight, norm, eps, table, pos, interleaved, scale, out):
    """One of queries and keys, and its bound: the norm's d / 2 + 8 units and four
    of the rotation and the scale, over the magnitudes of the rotation's sums."""
    y = head_norm(x, weight, norm, eps)
    mag = np.abs(y)
    if table is not None:
        y, mag = rotate(y, table, pos, interleaved)
    y, mag = y * scale, mag * abs(scale)
    return y, (x.shape[-1] / 2 + 12) * U32 * mag + U_OUT[out] * np.abs(y)


def gated_norm(x, gate, weight, silu, eps, out):
    """Outputs and their bound: the norm's d / 2 + 8 units and those of the gate,
    exp of a rounded argument (|gate| units), a sum, a quotient, products (8)."""
    y = head_norm(x, weight, "rms", eps)
    units = x.shape[-1] / 2 + 8
    if gate is not None:
        y = y * (gate if silu else 1.0) / (1.0 + np.exp(-gate))
        units = units + 8 + np.abs(gate)
    return y, units * U32 * np.abs(y) + U_OUT[out] * np.abs(y)
