"""How exact the states of linear attention are, as a norm over a head: the elementwise
bounds of linear_ref have to hold for the worst order of signs and let pass what a
plainer kernel would lose.

Prompts on the tensor cores, per chunk of 64 tokens, in units of 2^-24 of the state.  A
step adds 16 products; its addends are cut two bits behind the last of 24 bits of the
largest, and the sum to 24 bits, always downwards.  The first bf16 of the split operand
comes last: its four steps cut a unit of 2^-23 each off the sum at most (8), and off its
products, which have 16 bits, only where those are small (2 in all); the eight steps
before them hold 2^-7 of the sum and cut as much less (2 at most).  The weights e^x of the
tokens are off by 2 units of 2^-23 at most (4); the state before takes one fused
multiply-add a chunk (1/2); and what earlier chunks were off stays in proportion to what
they added.  16 1/2 in all; the limit is 17 units.

Token by token: a token's two fused multiply-adds and its product round a state of
random sign to 1/2 unit each, 1 in all by their squares, and n of them add up as a
random walk: sqrt(n) units.

Both are far below what one fp32 value of e^g loses where g is small and always the
same: its rounding, up to 2^-25, acts n times in one direction.
"""
import numpy as np
import torch

U32 = 2.0 ** -24
TENSOR = 17 * U32
# log decays whose e^g in fp32 is off by 0.9 of 2^-25 and more, above and below
WEAK = [-1.664e-4, -1.329e-4]


def walked(n):
    return np.sqrt(n) * U32


def state64(k, v, g, first):
    """[dv][dk] after all tokens, of one head: each token with the decays after it."""
    later = np.concatenate([np.cumsum(g[::-1])[::-1][1:], [0.0]])
    return np.exp(g.sum()) * first + (v * np.exp(later)[:, None]).T @ k


def off(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


def one_decay(k, v, g, first):
    """The recurrence in fp32 with one fp32 e^g a token."""
    S = first.astype(np.float32)
    for kt, vt, a in zip(k.astype(np.float32), v.astype(np.float32), np.exp(g).astype(np.float32)):
        S = a * S + vt[:, None] * kt
    return S.astype(np.float64)


def truncated(x, bits):
    m, e = np.frexp(x)
    return np.ldexp(np.trunc(m * 2.0 ** bits) / 2.0 ** bits, e)


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).bfloat16().double().numpy()


def two_parts(k, v, g, first):
    """Exact sums of keys with their decays, split into two bf16."""
    S = first
    for c in range(0, len(k), 64):
        gc = g[c:c + 64]
        w = k[c:c + 64] * np.exp(gc.sum() - np.cumsum(gc))[:, None]
        hi = truncated(w, 8)
        S = np.exp(gc.sum()) * S + v[c:c + 64].T @ (hi + bf16(w - hi))
    return S


def one_sum(k, v, g, first):
    """A part of 15 chunks in one accumulator, cut to 24 bits after each step of 16 tokens
    and part of the keys (in three), from the last chunk to the first."""
    S = first
    for c in range(0, len(k), 960):
        gc = g[c:c + 960]
        w = k[c:c + 960] * np.exp(gc.sum() - np.cumsum(gc))[:, None]
        hi = truncated(w, 8)
        mid = truncated(w - hi, 8)
        U = np.zeros_like(first)
        for t in range((len(gc) - 1) // 64 * 64, -1, -64):
            for part in (hi, mid, w - hi - mid):
                for s in range(t, min(t + 64, len(gc)), 16):
                    U = truncated(U + v[c + s:c + min(s + 16, t + 64)].T @ part[s:min(s + 16, t + 64)], 24)
        S = np.exp(gc.sum()) * S + U
    return S


def numbers(seed, n, dk=64, dv=64):
    rng = np.random.default_rng(seed)
    return bf16(rng.standard_normal((n, dk)) * dk ** -0.5), bf16(rng.standard_normal((n, dv))), np.zeros((dv, dk))


def large_parts_first(k, v, g, first):
    """Chunks whose keys are split into three, the first bf16 summed first: what the later
    ones add is cut at the place of a sum that is already large."""
    S = first
    for c in range(0, len(k), 64):
        gc = g[c:c + 64]
        w = k[c:c + 64] * np.exp(gc.sum() - np.cumsum(gc))[:, None]
        hi = truncated(w, 8)
        mid = truncated(w - hi, 8)
        U = np.zeros_like(first)
        for part in (hi, mid, w - hi - mid):
            for s in range(0, len(gc), 16):
                products = v[c + s:c + min(s + 16, 64)][:, :, None] * part[s:s + 16][:, None, :]
                largest = np.maximum(np.abs(products).max(0), np.abs(U))
                unit = np.ldexp(1.0, np.frexp(largest)[1] - 26)
                U = truncated((np.trunc(products / unit).sum(0) + np.trunc(U / unit)) * unit, 24)
        S = np.exp(gc.sum()) * S + U
    return S
