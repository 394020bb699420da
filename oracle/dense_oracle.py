"""fp64 oracle of the operators beside the expert layer: routing with a bias
for load balance, the gradient of the routing weights, quantisation of
SiLU(gate) * up in groups, and the dense block-scaled FP8 product.  Written
token by token and block by block from the definitions.
"""
from __future__ import annotations

import numpy as np

from .moe_oracle import scores, silu

__all__ = ["route_biased", "route_weights_of", "route_backward", "swiglu_rows", "matmul_blocks"]


def _best(values, candidates, count):
    """The `count` candidates with the largest values, in order, ties to the
    lower index."""
    return sorted(candidates, key=lambda i: (-values[i], i))[:count]


def _softmax_or_sigmoid(l, method):
    """Scores of one row; a row of masked logits alone has scores of 0."""
    if method == "softmax" and np.all(np.isneginf(l)):
        return np.zeros_like(l)
    with np.errstate(invalid="ignore"):
        return scores(l[None], method)[0]


def route_weights_of(l, ids, method, renormalize, scale):
    """Weights of the chosen experts `ids` of one row of logits."""
    p = _softmax_or_sigmoid(l, method)[list(ids)]
    if method == "sigmoid" or renormalize:
        top = max(l[i] for i in ids)
        if np.isneginf(top):
            return np.zeros(len(ids))
        # the ratios p / sum p, from differences of log p (no underflow)
        lp = np.array([-np.logaddexp(0.0, -l[i]) if method == "sigmoid" else l[i] for i in ids])
        r = np.exp(lp - lp.max())
        p = r / r.sum()
    return p * scale


def route_biased(logits, bias, top_k, method="softmax", renormalize=False, k_group=1,
                 group_count=1, group_select_mode=0, routed_scaling_factor=1.0):
    """(weights [M, k], ids [M, k]): choice by c = p + bias, weights from p."""
    logits = np.asarray(logits, dtype=np.float64)
    bias = np.asarray(bias, dtype=np.float64)
    M, E = logits.shape
    gs = E // group_count
    W, I = np.zeros((M, top_k)), np.zeros((M, top_k), dtype=np.int32)
    for t in range(M):
        l = logits[t]
        c = _softmax_or_sigmoid(l, method) + bias
        c = np.where(np.isneginf(l) | np.isnan(c), -np.inf, c)
        allowed = range(E)
        if group_count > 1:
            key = []
            for g in range(group_count):
                part = np.sort(c[g * gs:(g + 1) * gs])
                key.append(part[-1] if group_select_mode == 0 else part[-1] + part[-2])
            kept = _best(key, range(group_count), k_group)
            allowed = [e for e in range(E) if e // gs in kept]
        ids = _best(c, allowed, top_k)
        I[t] = ids
        W[t] = route_weights_of(l, ids, method, renormalize, routed_scaling_factor)
    return W, I


def route_backward(grad_weights, logits, ids, method="softmax", renormalize=False,
                   routed_scaling_factor=1.0):
    """d(sum gw * w) / d logits through p and the quotient rule, by expert."""
    logits = np.asarray(logits, dtype=np.float64)
    gw = np.asarray(grad_weights, dtype=np.float64)
    M, E = logits.shape
    out = np.zeros((M, E))
    renorm = method == "sigmoid" or renormalize
    for t in range(M):
        l = logits[t]
        js = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        chosen = [int(ids[t, j]) for j in js]
        p = _softmax_or_sigmoid(l, method)
        gp = np.zeros(E)
        total = sum(p[e] for e in chosen) if renorm else 1.0
        if total == 0.0:
            continue
        mean = sum(gw[t, j] * p[e] for j, e in zip(js, chosen)) / total if renorm else 0.0
        for j, e in zip(js, chosen):
            gp[e] += routed_scaling_factor * (gw[t, j] - mean) / total
        if method == "sigmoid":
            out[t] = gp * p * (1.0 - p)
        else:
            out[t] = p * (gp - np.dot(gp, p))
    return out


def swiglu_rows(x):
    """SiLU(x[:, :K]) * x[:, K:]."""
    x = np.asarray(x, dtype=np.float64)
    K = x.shape[1] // 2
    return silu(x[:, :K]) * x[:, K:]


def matmul_blocks(a, a_scale, w, w_scale, bias=None):
    """(y, size) of the block-scaled product: a [M, K] and w [K, N] as values,
    a_scale [M, ceil(K/128)], w_scale [ceil(K/128), ceil(N/128)]; size is the
    sum of the terms' magnitudes, for error bounds."""
    a, w = np.asarray(a, dtype=np.float64), np.asarray(w, dtype=np.float64)
    a_scale, w_scale = np.asarray(a_scale, np.float64), np.asarray(w_scale, np.float64)
    M, K = a.shape
    N = w.shape[1]
    y, size = np.zeros((M, N)), np.zeros((M, N))
    for kb in range(-(-K // 128)):
        ks = slice(kb * 128, min(K, kb * 128 + 128))
        for nb in range(-(-N // 128)):
            ns = slice(nb * 128, min(N, nb * 128 + 128))
            s = a_scale[:, kb:kb + 1] * w_scale[kb, nb]
            y[:, ns] += s * (a[:, ks] @ w[ks, ns])
            size[:, ns] += np.abs(s) * (np.abs(a[:, ks]) @ np.abs(w[ks, ns]))
    if bias is not None:
        y += np.asarray(bias, dtype=np.float64)
        size += np.abs(np.asarray(bias, dtype=np.float64))
    return y, size
