"""CPU oracle of the 4-bit operands and of the layer for a few tokens, in float64.

TEST INFRASTRUCTURE ONLY, as oracle/moe_oracle.py: the product path never
imports it and it imports nothing from the product path.

  quantize       per 32 values: s - 127 = max(floor(log2 max|x|) - 2, -127); the code is the grid value nearest to
                 x / 2^(s - 127), found by comparing distances, ties to the even code; s = 255 and codes 0 for a block
                 with an infinity or NaN
  values         2^(s - 127) times the grid value; NaN for s = 255
  few_tokens     route, experts and combine, token by token, with a bound on what fp32 arithmetic may be off
"""
from __future__ import annotations

import numpy as np

from . import operators_oracle as Q

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
U2 = 2.0 ** -23  # an fp32 step: what one operation may be off, doubled for units that truncate


def quantize(x):
    """Unpacked codes [..., K] and scale bytes [..., K / 32]."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], -1, 32)
    top = np.abs(b).max(axis=-1)
    bad = ~np.isfinite(b).all(axis=-1)
    top = np.where(bad, 0.0, top)
    e = np.where(top > 0, np.frexp(top)[1] - 1, -10 ** 6)  # top = m 2^(e + 1), m in [1/2, 1)
    s = np.maximum(e - 2, -127)
    y = np.where(bad[..., None], 0.0, b) * np.exp2(-s.astype(np.float64))[..., None]
    d = np.abs(np.abs(y)[..., None] - GRID)
    near = d == d.min(axis=-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(axis=-1), even.argmax(axis=-1), near.argmax(axis=-1))
    code = np.where(np.signbit(b) & ~bad[..., None], code + 8, code)
    return code.reshape(x.shape).astype(np.uint8), np.where(bad, 255, s + 127).astype(np.uint8)


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    packed = np.asarray(packed)
    return np.stack((packed & 15, packed >> 4), axis=-1).reshape(*packed.shape[:-1], -1)


def values(packed, scales):
    c, s = unpack(packed), np.asarray(scales).astype(np.float64)
    scale = np.where(s == 255, np.nan, np.exp2(s - 127.0))
    v = np.where(c >= 8, -1.0, 1.0) * GRID[c % 8]
    return (v.reshape(*v.shape[:-1], -1, 32) * scale[..., None]).reshape(v.shape)


def route(logits, k, renormalize=True):
    """moe_few_tokens's own routing: softmax weights, bars and empty slots as in the grouped routing without a bias."""
    return Q.route_grouped(logits, k, renormalize=renormalize)


def few_tokens(x, idx, w, weights, act, expert_begin, E_loc):
    """(out, bound): weights(e) gives (w0, w0_up | None, w1) of local expert e in float64.

    bound: a product of K terms in fp32 is within K steps of the sum of their absolute values; the activation passes an
    error of z on by at most 1.2 and adds 4 steps (exp2, reciprocal or erf, products); the gate weight, a sum over
    slots, adds k; the second product's terms carry 24 bits each.
    """
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    T, k = idx.shape
    H = x.shape[1]
    out, bound = np.zeros((T, H)), np.zeros((T, H))
    terms = np.zeros((T, H))
    for e in range(E_loc):
        mine = idx == expert_begin + e
        for t in np.nonzero(mine.any(axis=1))[0]:
            w0, w0_up, w1 = weights(e)
            F = w0.shape[0]
            gate, gabs = w[t][mine[t]].sum(), np.abs(w[t][mine[t]]).sum()
            z, dz = w0 @ x[t], H * U2 * (np.abs(w0) @ np.abs(x[t]))
            if act == "swiglu":
                u, du = w0_up @ x[t], H * U2 * (np.abs(w0_up) @ np.abs(x[t]))
                s = Q.act("silu", z)
                a, da = s * u, 1.2 * dz * (np.abs(u) + du) + np.abs(s) * du + 4 * U2 * np.abs(s * u)
            else:
                a = Q.act("gelu", z)
                da = 1.2 * dz + 4 * U2 * np.abs(z)
            a, da = a * gate, da * gabs + np.abs(a) * (k + 1) * U2 * gabs
            out[t] += w1 @ a
            mag = np.abs(w1) @ np.abs(a)
            bound[t] += np.abs(w1) @ da + F * U2 * mag
            terms[t] += mag
    return out, bound + (k + 8) * U2 * terms + 1e-30
