"""Plain 64-bit numpy forms of the routed-expert layer's calls (pair by pair, row by row)."""
from __future__ import annotations

import math

import numpy as np

ERR_EXPERT = 2


def plan(ids, E, lora=None, expert_map=None):
    """The plan's arrays and the error bits for ids [T, k]."""
    T, k = ids.shape
    lists, err = [[] for _ in range(E)], 0
    for p, e in enumerate(ids.reshape(-1).tolist()):
        if e == -1:
            continue
        if expert_map is not None:
            if not 0 <= e < len(expert_map):
                err |= ERR_EXPERT
                continue
            e = int(expert_map[e])
            if e < 0:
                continue
        if not 0 <= e < E:
            err |= ERR_EXPERT
            continue
        lists[e].append(p)
    seg = np.concatenate([[0], np.cumsum([len(x) for x in lists])])
    pairs = np.array([p for x in lists for p in x], dtype=np.int64)
    full = {n: np.full(T * k, -1) for n in ("row_pair", "pair_row", "row_expert", "row_lora")}
    full["row_pair"][:len(pairs)] = pairs
    full["pair_row"][pairs] = np.arange(len(pairs))
    full["row_expert"][:len(pairs)] = np.repeat(np.arange(E), np.diff(seg))
    if lora is not None:
        full["row_lora"][:len(pairs)] = np.asarray(lora)[pairs // k]
    return {"seg_start": seg, **full, "pair_row": full["pair_row"].reshape(T, k), "err": err}


def combine(rows, pair_row, weights=None, residual=None):
    """The sums and, for bounds, the sums of magnitudes."""
    T, k = pair_row.shape
    out = np.zeros((T, rows.shape[1])) if residual is None else residual.astype(float).copy()
    size = np.abs(out)
    for t in range(T):
        for j in range(k):
            r = pair_row[t, j]
            if 0 <= r < len(rows):
                y = rows[r] * (1.0 if weights is None else float(weights[t, j]))
                out[t] += y
                size[t] += np.abs(y)
    return out, size


def combine_grad(grad_out, rows, pair_row, weights=None):
    """grad_rows (NaN where no pair leads), grad_weights and the dots' sums of magnitudes."""
    T, k = pair_row.shape
    grad_rows, grad_w, size = np.full(rows.shape, np.nan), np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = pair_row[t, j]
            if 0 <= r < len(rows):
                grad_rows[r] = grad_out[t] * (1.0 if weights is None else float(weights[t, j]))
                grad_w[t, j] = grad_out[t] @ rows[r]
                size[t, j] = np.abs(grad_out[t]) @ np.abs(rows[r])
    return grad_rows, grad_w, size


def activation(z, act):
    if act == "relu":
        return np.maximum(z, 0)
    if act == "silu":
        return z / (1 + np.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + np.vectorize(math.erf)(z / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def linear(x, w, bias=None, delta=None, residual=None, act="none", gated=False):
    """The result, and a bound on what float32 sums and elementary functions may add to the result's own rounding.

    A sum of K products and up to two terms in float32, in any order, with the tensor cores' sums cut rather than rounded
    (2^-22 of the largest partial sum an addition, K / 16 + 2 additions of 16 exact products): relative to the sum of
    magnitudes at most (K / 16 + 4) 2^-22, less 16 terms an instruction; the plain kernels' K 2^-24 is below it too.
    Activations have a slope of at most 1.13, and their float32 values a relative error below 2^-20."""
    z, size = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        z, size = z + bias, size + np.abs(bias)
    if delta is not None:
        z, size = z + delta, size + np.abs(delta)
    err = size * (x.shape[1] / 16 + 4) * 2.0 ** -22
    if gated:
        half = z.shape[1] // 2
        gate, up = activation(z[:, :half], act), z[:, half:]
        y = gate * up
        err = 1.13 * err[:, :half] * np.abs(up) + err[:, half:] * np.abs(gate) + 2.0 ** -20 * (np.abs(y) + np.abs(z[:, :half] * up))
    else:
        y = activation(z, act)
        err = 1.13 * err + 2.0 ** -20 * np.abs(z)
    if residual is not None:
        y = y + residual
    return y, err + 2.0 ** -23 * np.abs(y)
