"""Oracle of the operators beside the layer, fp64 NumPy: the gated choice of
experts, the block-FP8 product on E4M3 activations, SwiGLU, and the layer with
the gated choice. Written from the formulas in include/moe_fp8.h, one token or
one block at a time.
"""
from __future__ import annotations

from typing import Callable, Optional

import numpy as np

from .moe_oracle import dequantise_activations, e4m3fn_decode, expert_matrices, swiglu_expert

MASKED_LOGIT = -3.3e38
F32_MAX = 3.4028234663852886e38


def expert_scores(logits: np.ndarray, score: str) -> np.ndarray:
    """s_e of each token's row of logits; 0 for masked experts."""
    l = np.asarray(logits, np.float64)
    s = np.zeros(l.shape)
    for t in range(len(l)):
        ok = l[t] > MASKED_LOGIT  # False for NaN
        v = np.minimum(l[t][ok], F32_MAX)
        if not ok.any():
            continue
        if score == "softmax":
            p = np.exp(v - v.max())
            s[t][ok] = p / p.sum()
        elif score == "sigmoid":
            with np.errstate(over="ignore"):
                s[t][ok] = 1.0 / (1.0 + np.exp(-v))
        else:
            raise ValueError(score)
    return s


def gated_choice(logits: np.ndarray, k: int, score: str = "softmax",
                 balance: Optional[np.ndarray] = None, groups: int = 1, top_groups: int = 1,
                 group_rank: int = 1, renormalise: bool = True, scale: float = 1.0):
    """(idx [T][k] int64, gates [T][k] fp64)."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    per = E // groups
    s = expert_scores(l, score)
    b = np.zeros(E) if balance is None else np.asarray(balance, np.float64)
    idx = np.zeros((T, k), np.int64)
    gates = np.zeros((T, k))
    for t in range(T):
        free = [e for e in range(E) if l[t, e] > MASKED_LOGIT]
        c = {e: s[t, e] + b[e] for e in free}
        group_score = []
        for g in range(groups):
            best = sorted((c[e] for e in free if e // per == g), reverse=True)[:group_rank]
            group_score.append(sum(best) if best else -np.inf)
        kept = sorted(range(groups), key=lambda g: (-group_score[g], g))[:top_groups]
        open_ = sorted((e for e in free if e // per in kept), key=lambda e: (-c[e], e))
        shut = [e for e in range(E) if e // per in kept and e not in c]
        idx[t] = (open_ + shut)[:k]
        g = s[t, idx[t]]
        if renormalise:
            g = g / g.sum() if g.sum() > 0 else np.zeros(k)
        gates[t] = g * float(np.float32(scale))
    return idx, gates


def block_weights(w: np.ndarray, scales: np.ndarray, block: int = 128) -> np.ndarray:
    """[N][K] fp64 values of a block-FP8 weight whose last row of blocks may be
    cut short."""
    N, K = w.shape
    s = np.asarray(scales, np.float64)
    rows, cols = np.arange(N) // block, np.arange(K) // block
    return e4m3fn_decode(w) * s[rows][:, cols]


def linear_e4m3(codes: np.ndarray, exps: np.ndarray, w: np.ndarray, scales: np.ndarray,
                bias: Optional[np.ndarray] = None):
    """(y, mag): the product of the quantised activations (exps unbiased) with
    the weights, and the sum of its terms' magnitudes (for error bounds)."""
    a = dequantise_activations(codes, exps, 128)
    wv = block_weights(w, scales)
    y, mag = a @ wv.T, np.abs(a) @ np.abs(wv).T
    if bias is not None:
        y, mag = y + np.asarray(bias, np.float64), mag + np.abs(np.asarray(bias, np.float64))
    return y, mag


def swiglu(gate_up: np.ndarray) -> np.ndarray:
    """silu(g) * u of rows [g | u]."""
    gu = np.asarray(gate_up, np.float64)
    g, u = np.split(gu, 2, axis=1)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def gated_layer(x: np.ndarray, idx: np.ndarray, gates: np.ndarray,
                expert: Callable[[int], dict], inter: int, block: int,
                shared: Optional[dict] = None) -> np.ndarray:
    """The layer's output for a given choice of experts and gates."""
    x = np.asarray(x, np.float64)
    out = np.zeros_like(x)
    for e in np.unique(idx):
        t, j = np.nonzero(idx == e)
        y = swiglu_expert(x[t], *expert_matrices(expert(int(e)), inter, block))
        np.add.at(out, t, gates[t, j][:, None] * y)
    if shared is not None:
        out += swiglu_expert(x, *expert_matrices(shared, inter, block))
    return out
