"""Gated delta rule of the recurrent layers, along chains and trees (oracle; test infrastructure only).

The pages name the need (mlxcel issue #1204: recurrent layers cannot take a mask, and a flattened tree leaks state
between siblings; Splash issue #728: the selected path's recurrent state is the one retained) and leave the
recurrence out.  Reading: the published gated delta rule.  For one value head with state S [DV, DK], log decay g and
write strength beta:

    S <- e^g S;  u = beta (v - S k);  S <- S + u k^T;  o = scale * S q

with q and k divided by sqrt(sum x^2 + norm_eps) when norm_eps > 0, and value head h reading key head
h // (HV / HK).  A tree's node starts from its parent's state (the root from the sequence's).
"""
from __future__ import annotations

import math

import numpy as np


def unit_rows(x, norm_eps: float) -> np.ndarray:
    x = np.asarray(x, dtype=np.float64)
    return x if norm_eps == 0 else x / np.sqrt((x * x).sum(axis=-1, keepdims=True) + norm_eps)


def step(S, q, k, v, g: float, beta: float, scale: float):
    """One token of one head: S [DV, DK] -> (new S, o [DV])."""
    S = math.exp(g) * S if g != -math.inf else np.zeros_like(S)
    u = beta * (v - S @ k)
    S = S + np.outer(u, k)
    return S, scale * (S @ q)


def _scale(scale, DK):
    return 1.0 / math.sqrt(DK) if scale == 0 else scale


def tree_verify(q, k, v, g, beta, state, parents, norm_eps=1e-6, scale=0.0) -> np.ndarray:
    """One (sequence, layer): q/k [T, HK, DK], v [T, HV, DV], g/beta [T, HV], state [HV, DV, DK] -> o [T, HV, DV]."""
    T, HV, DV = v.shape
    q, k = unit_rows(q, norm_eps), unit_rows(k, norm_eps)
    per, sc = HV // k.shape[1], _scale(scale, k.shape[2])
    o = np.zeros((T, HV, DV))
    for h in range(HV):
        forks = []
        for i in range(T):
            S0 = np.asarray(state[h], dtype=np.float64) if parents[i] < 0 else forks[parents[i]]
            S, o[i, h] = step(S0, q[i, h // per], k[i, h // per], v[i, h], float(g[i, h]), float(beta[i, h]), sc)
            forks.append(S)
    return o


def scan(q, k, v, g, beta, state, norm_eps=1e-6, scale=0.0):
    """One (sequence, layer) over its tokens in order -> (o [n, HV, DV], new state [HV, DV, DK])."""
    n, HV, DV = v.shape
    q, k = unit_rows(q, norm_eps), unit_rows(k, norm_eps)
    per, sc = HV // k.shape[1], _scale(scale, k.shape[2])
    o = np.zeros((n, HV, DV))
    new = np.array(state, dtype=np.float64)
    for h in range(HV):
        for t in range(n):
            new[h], o[t, h] = step(new[h], q[t, h // per], k[t, h // per], v[t, h], float(g[t, h]), float(beta[t, h]), sc)
    return o, new


def commit(q, k, v, g, beta, state, path, norm_eps=1e-6) -> np.ndarray:
    """The state after the block's rows ``path``, in order (q only gives the shape of the key heads)."""
    path = [int(p) for p in path]
    return scan(np.asarray(q)[path], np.asarray(k)[path], np.asarray(v)[path], np.asarray(g)[path],
                np.asarray(beta)[path], state, norm_eps)[1]
