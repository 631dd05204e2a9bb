"""The routed-expert layer around the grouped GEMM, in float64 loops.

Router, grouped order of the routed slots, dispatch, combine, SwiGLU with its
8-bit checkpoint, and their gradients, written from the definitions: one token
or one slot at a time, no shared code with the HIP path.  Values are float64
arrays (the caller rounds); a checkpoint's codes and scales are those of
``quantize_cache_packed`` for fp8 in blocks of 32.
"""

import numpy as np

from .cache import dequantize_cache_packed, quantize_cache_packed
from .formats import from_dtype_bits

CHECKPOINT_BLOCK = 32


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-np.asarray(x, np.float64)))


def scores(x, score):
    """Scores of one token's logits; experts with a logit of -inf or NaN have none (NaN here)."""
    x = np.asarray(x, np.float64)
    ok = x > -np.inf
    s = np.full(x.shape, np.nan)
    if score == "sigmoid":
        s[ok] = sigmoid(x[ok])
    elif ok.any():
        e = np.exp(x[ok] - x[ok].max())
        s[ok] = e / e.sum()
    return s


def chosen_scores(x, s, chosen, score, renormalize):
    """Scores to renormalize over: a softmax's up to a common factor, so that logits far below the largest of all do
    not vanish beside it."""
    if score == "softmax" and renormalize and len(chosen):
        with np.errstate(over="ignore"):                  # of experts that were not chosen
            s = np.exp(np.asarray(x, np.float64) - max(x[e] for e in chosen))
    return s


def route(logits, top_k, score="softmax", bias=None, groups=1, top_groups=1, group_best=2, renormalize=True, scale=1.0,
          token_mask=None):
    """(weights float64 [T, k], experts int32 [T, k]) of logits [T, E]."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    weights, experts = np.zeros((T, top_k)), np.full((T, top_k), -1, np.int32)
    for t in range(T):
        if token_mask is not None and not token_mask[t]:
            continue
        s = scores(logits[t], score)
        key = s + np.asarray(bias, np.float64) if bias is not None else (logits[t] if groups == 1 else s)
        able = [e for e in range(E) if not np.isnan(s[e]) and key[e] > -np.inf]
        if groups > 1:
            size = E // groups
            value = {}
            for g in range(groups):
                inside = sorted((key[e] for e in able if e // size == g), reverse=True)[:group_best]
                if inside:
                    value[g] = sum(inside)
            kept = sorted(value, key=lambda g: (-value[g], g))[:top_groups]
            able = [e for e in able if e // size in kept]
        chosen = sorted(able, key=lambda e: (-key[e], e))[:top_k]
        s = chosen_scores(logits[t], s, chosen, score, renormalize)
        total = sum(s[e] for e in chosen)
        for j, e in enumerate(chosen):
            experts[t, j] = e
            weights[t, j] = scale * s[e] / total if renormalize and total > 0 else (0.0 if renormalize else scale * s[e])
    return weights, experts


def route_grad(logits, experts, grad_weights, score="softmax", renormalize=True, scale=1.0):
    """Gradient [T, E] of sum(grad_weights * weights) with the choice held."""
    logits = np.asarray(logits, np.float64)
    out = np.zeros(logits.shape)
    for t in range(logits.shape[0]):
        places = [(j, int(e)) for j, e in enumerate(experts[t]) if 0 <= e < logits.shape[1]]
        if not places:
            continue
        s = chosen_scores(logits[t], scores(logits[t], score), [e for _, e in places], score, renormalize)
        total = sum(s[e] for _, e in places)
        u = np.zeros(logits.shape[1])
        if renormalize and total == 0:                    # the weights are 0, whatever the logits do
            continue
        for j, e in places:
            if renormalize:
                mean = sum(grad_weights[t, i] * s[f] for i, f in places) / total
                u[e] = scale * (grad_weights[t, j] - mean) / total
            else:
                u[e] = scale * grad_weights[t, j]
        s0 = np.where(u != 0, np.nan_to_num(s, nan=0.0), 0.0) if renormalize else np.nan_to_num(s, nan=0.0)
        out[t] = u * s0 * (1 - s0) if score == "sigmoid" else s0 * (u - (u * s0).sum())
    return out


def plan(experts, first, local):
    """(offs [local], rows [T, k], slots [T * k]) of experts [T, k]."""
    flat = np.asarray(experts).reshape(-1)
    order = [s for e in range(local) for s in range(flat.size) if flat[s] == first + e] if flat.size < 4096 else \
        [int(s) for e in range(local) for s in np.flatnonzero(flat == first + e)]
    offs = np.cumsum([int((flat == first + e).sum()) for e in range(local)]).astype(np.int32)
    here = set(order)
    order += [s for s in range(flat.size) if s not in here]
    rows = np.zeros(flat.size, np.int32)
    for r, s in enumerate(order):
        rows[s] = r if r < offs[-1] else ~r
    return offs, rows.reshape(np.shape(experts)), np.asarray(order, np.int32)


def dispatch(x, rows):
    """Rows of x [T, H] in the grouped order; zeros where no slot is served."""
    x = np.asarray(x)
    out = np.zeros((rows.size, x.shape[1]), x.dtype)
    for t, j in np.ndindex(rows.shape):
        if 0 <= rows[t, j] < rows.size:
            out[rows[t, j]] = x[t]
    return out


def combine(y, weights, rows):
    y = np.asarray(y, np.float64)
    out = np.zeros((rows.shape[0], y.shape[1]))
    for t, j in np.ndindex(rows.shape):
        if 0 <= rows[t, j] < rows.size:
            out[t] += (1.0 if weights is None else float(weights[t, j])) * y[rows[t, j]]
    return out


def dispatch_grad(grad, rows):
    return combine(grad, None, rows)


def combine_grad(grad_out, y, weights, rows):
    """(grad_y [T * k, H], grad_weights [T, k])."""
    grad_out, y = np.asarray(grad_out, np.float64), np.asarray(y, np.float64)
    gy, gw = np.zeros(y.shape), np.zeros(rows.shape)
    for t, j in np.ndindex(rows.shape):
        if 0 <= rows[t, j] < rows.size:
            gy[rows[t, j]] = float(weights[t, j]) * grad_out[t]
            gw[t, j] = grad_out[t] @ y[rows[t, j]]
    return gy, gw


def swiglu(gate_up):
    g, u = np.split(np.asarray(gate_up, np.float64), 2, axis=1)
    return g * sigmoid(g) * u


def swiglu_grad(gate_up, grad_h):
    """Gradient [R, 2 I] at gate_up (the kept values, where the input was kept in 8 bits)."""
    g, u = np.split(np.asarray(gate_up, np.float64), 2, axis=1)
    s = sigmoid(g)
    return np.concatenate([grad_h * u * s * (1 + g * (1 - s)), grad_h * g * s], axis=1)


def kept(gate_up):
    """The values that gate_up (float32) has after the 8-bit checkpoint."""
    codes, scales = quantize_cache_packed(np.asarray(gate_up, np.float32), "fp8", CHECKPOINT_BLOCK)
    return from_dtype_bits(dequantize_cache_packed(codes, scales, "fp8", CHECKPOINT_BLOCK, "f32"), "f32").astype(
        np.float64)
