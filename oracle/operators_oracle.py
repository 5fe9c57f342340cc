"""CPU oracle of the operators beside the four-call path, in float64.

TEST INFRASTRUCTURE ONLY, as oracle/moe_oracle.py: the product path never
imports it and it imports nothing from the product path.

Routing is written one token at a time with plain sorts; the products are
written with numpy matrix products.  Definitions:

  route_grouped    s = sigmoid(l) or softmax(l) over the available experts (logit neither NaN nor -inf, bias
                   neither NaN nor -inf; +inf counts as the largest fp32); key = s + bias; a group's key is the sum
                   of its group_top largest; the best topk_group groups stay; the k largest keys, ties lowest id
                   first; weight = scale * s, over the chosen ones' sum when renormalised; empty slots (-1, 0).
  *_backward       the analytic gradients, pinned by central differences in the tests.
  linear           act(x w^T + b) [* (x w_up^T + b_up)] + residual.
"""
from __future__ import annotations

import numpy as np
from scipy.special import erf, expit

FMAX = float(np.finfo(np.float32).max)


def _row_scores(l, b, score):
    l = np.asarray(l, np.float64)
    ok = ~np.isnan(l) & ~np.isneginf(l)
    if b is not None:
        ok &= ~np.isnan(b) & ~np.isneginf(b)
    x = np.minimum(np.where(ok, l, 0.0), FMAX)
    if score == "sigmoid":
        return np.where(ok, expit(x), 0.0), x, ok
    s = np.zeros_like(x)
    if ok.any():
        e = np.exp(x[ok] - x[ok].max())
        s[ok] = e / e.sum()
    return s, x, ok


def _weights(s, x, ids, score, renormalize, scale):
    """Gate weights of the chosen ids; renormalised from logarithms of the scores, which never underflow."""
    if not len(ids):
        return np.zeros(0)
    if not renormalize:
        return scale * s[ids]
    logs = -np.logaddexp(0.0, -x[ids]) if score == "sigmoid" else x[ids]
    e = np.exp(logs - logs.max())
    return scale * e / e.sum()


def route_grouped(logits, k, bias=None, score="softmax", n_group=1, topk_group=1, group_top=1, renormalize=True,
                  scale=1.0):
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    b = None if bias is None else np.asarray(bias, np.float64)
    Eg = E // n_group
    idx = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        s, x, ok = _row_scores(logits[t], b, score)
        key = x if b is None else s + np.minimum(np.where(ok, b, 0.0), FMAX)  # without a bias: the scores' order is the logits'
        groups = []
        for g in range(n_group):
            mine = sorted((e for e in range(g * Eg, (g + 1) * Eg) if ok[e]), key=lambda e: -key[e])[:group_top]
            by_score = b is None and group_top > 1
            groups.append(sum((s if by_score else key)[e] for e in mine) if mine else -np.inf)
        kept = sorted(range(n_group), key=lambda g: (-groups[g], g))[:topk_group]
        cand = [e for e in range(E) if ok[e] and e // Eg in kept]
        ids = sorted(cand, key=lambda e: (-key[e], e))[:k]
        idx[t, :len(ids)] = ids
        w[t, :len(ids)] = _weights(s, x, np.array(ids, int), score, renormalize, scale)
    return idx, w


def gate_weights(logits, idx, score, renormalize, scale, bias=None):
    """topk_w for a fixed choice (slots outside [0, E) are empty); the bias matters where it bars experts."""
    logits = np.asarray(logits, np.float64)
    b = None if bias is None else np.asarray(bias, np.float64)
    w = np.zeros(idx.shape)
    for t in range(len(idx)):
        s, x, ok = _row_scores(logits[t], b, score)
        has = [j for j, e in enumerate(idx[t]) if 0 <= e < logits.shape[1] and ok[e]]
        w[t, has] = _weights(s, x, idx[t][has].astype(int), score, renormalize, scale)
    return w


def route_grouped_backward(logits, idx, d_w, score, renormalize, scale, bias=None):
    """(d_logits, magnitude): the gradient and, for tolerances, the sum of the absolute terms it is made of."""
    logits = np.asarray(logits, np.float64)
    b = None if bias is None else np.asarray(bias, np.float64)
    T, E = logits.shape
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        s, x, ok = _row_scores(logits[t], b, score)
        has = [j for j, e in enumerate(idx[t]) if 0 <= e < E and ok[e]]
        ids, g = idx[t][has].astype(int), scale * np.asarray(d_w[t], np.float64)[has]
        if not len(ids):
            continue
        if renormalize:
            q = _weights(s, x, ids, score, True, 1.0)
            rest = q @ g
            f = expit(-x[ids]) if score == "sigmoid" else 1.0
            np.add.at(out[t], ids, q * (g - rest) * f)
            np.add.at(mag[t], ids, q * (np.abs(g) + q @ np.abs(g)) * f)
        elif score == "sigmoid":
            d = g * s[ids] * expit(-x[ids])
            np.add.at(out[t], ids, d)
            np.add.at(mag[t], ids, np.abs(d))
        else:
            out[t] = -s * (s[ids] @ g)
            mag[t] = s * (s[ids] @ np.abs(g))
            np.add.at(out[t], ids, s[ids] * g)
            np.add.at(mag[t], ids, np.abs(s[ids] * g))
    return out, mag


def combine_backward(d_out, y_perm, inv_perm, topk_w):
    """(d_y_perm with NaN in the rows no slot names, d_topk_w, sum of the absolute terms of d_topk_w)."""
    d_out, y = np.asarray(d_out, np.float64), np.asarray(y_perm, np.float64)
    d_y = np.full(y.shape, np.nan)
    d_w, mag = np.zeros(inv_perm.shape), np.zeros(inv_perm.shape)
    for t, j in np.ndindex(*inv_perm.shape):
        p = inv_perm[t, j]
        if 0 <= p < len(y):
            d_y[p] = float(topk_w[t, j]) * d_out[t]
            d_w[t, j] = d_out[t] @ y[p]
            mag[t, j] = np.abs(d_out[t]) @ np.abs(y[p])
    return d_y, d_w, mag


def act(name, z):
    if name == "none":
        return z
    if name == "gelu":
        return 0.5 * z * (1.0 + erf(z / np.sqrt(2.0)))
    return z * expit(z)


def act_grad(name, z):
    if name == "none":
        return np.ones_like(z)
    if name == "gelu":
        return 0.5 * (1.0 + erf(z / np.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / np.sqrt(2.0 * np.pi)
    s = expit(z)
    return s * (1.0 + z * (1.0 - s))


def linear(x, w, w_up=None, bias=None, bias_up=None, act_name="none", residual=None):
    """(out, z, z_up)."""
    z = x @ w.T + (0.0 if bias is None else bias)
    u = None
    out = act(act_name, z)
    if act_name == "swiglu":
        u = x @ w_up.T + (0.0 if bias_up is None else bias_up)
        out = out * u
    return out + (0.0 if residual is None else residual), z, u


def linear_backward(d_out, x, w, w_up=None, act_name="none", z=None, z_up=None):
    """dict of d_x, d_w, d_w_up, d_bias, d_bias_up, dz, dz_up."""
    if act_name == "swiglu":
        dz, du = d_out * z_up * act_grad("silu", z), d_out * act("silu", z)
        return dict(d_x=dz @ w + du @ w_up, d_w=dz.T @ x, d_w_up=du.T @ x, d_bias=dz.sum(0), d_bias_up=du.sum(0),
                    dz=dz, dz_up=du)
    dz = d_out * (1.0 if act_name == "none" else act_grad(act_name, z))
    return dict(d_x=dz @ w, d_w=dz.T @ x, d_bias=dz.sum(0), dz=dz)
