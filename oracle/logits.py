"""The logit-side operators, written out plainly: per-request processing of
logits, 4-bit quantisation with group scales, products with 4-bit weights.

TEST INFRASTRUCTURE ONLY (see the package docstring): only the test suite and
``__graft_entry__.smoke()`` call it.

Processing and products are float64 on the exact input values.  Quantisation
is a rule of float32 steps (IEEE division, ties to even), so it is restated in
float32 NumPy and its results are the bits, not an approximation of them.
"""

from __future__ import annotations

import numpy as np

ERR_TOKEN, ERR_PARENT, ERR_MASK = 1, 2, 64


# ---------------------------------------------------------------------------
# processing
# ---------------------------------------------------------------------------

def tokens_before(tokens, parent, i, V):
    """The drafted tokens before row i (chain: 0 .. i-1; tree: the path from
    the root to i, the root excluded), without those outside [0, V)."""
    if tokens is None:
        return []
    if parent is None:
        path = list(tokens[:i])
    else:
        path = []
        while i > 0:
            path.append(tokens[i])
            p = int(parent[i])
            i = p if 0 <= p < i else 0  # malformed: the root's child
    return [int(t) for t in path if 0 <= t < V]


def process_logits(logits, tokens=None, parent=None, history=None, history_len=None, prompt_len=None,
                   repetition=None, frequency=None, presence=None, bias_tokens=None, bias_values=None,
                   bias_len=None, mask=None, mask_index=None):
    """logits float [B, n, V] (exact values); returns (y float64 [B, n, V],
    touched bool [B, n, V]: elements that a penalty, a bias or a mask applied
    to, scale float64 [B, n, V]: the sum of the magnitudes each element's
    float32 steps handle, error bits int [B])."""
    B, n, V = logits.shape
    y = np.asarray(logits, np.float64).copy()
    touched = np.zeros((B, n, V), bool)
    scale = np.zeros((B, n, V))
    err = np.zeros(B, np.int32)
    for b in range(B):
        hist = np.zeros(0, np.int64) if history is None else np.asarray(history[b], np.int64)
        if history is not None and history_len is not None:
            m = int(history_len[b])
            if not 0 <= m <= len(hist):
                err[b] |= ERR_TOKEN
                m = 0 if m < 0 else len(hist)
            hist = hist[:m]
        prompt = min(max(int(prompt_len[b]), 0), len(hist)) if prompt_len is not None else 0
        ok = (hist >= 0) & (hist < V)
        if not ok.all():
            err[b] |= ERR_TOKEN
        made0 = np.bincount(hist[prompt:][ok[prompt:]], minlength=V)
        seen0 = np.bincount(hist[ok], minlength=V)
        rho = 1.0 if repetition is None else float(repetition[b])
        freq = 0.0 if frequency is None else float(frequency[b])
        pres = 0.0 if presence is None else float(presence[b])
        bias, bias_abs, biased = np.zeros(V), np.zeros(V), np.zeros(V, bool)
        if bias_tokens is not None:
            k = bias_tokens.shape[1]
            m = k if bias_len is None else int(bias_len[b])
            if not 0 <= m <= k:
                err[b] |= ERR_TOKEN
                m = 0 if m < 0 else k
            for t, x in zip(bias_tokens[b, :m], bias_values[b, :m]):
                if 0 <= t < V:
                    bias[t] += float(x)
                    bias_abs[t] += abs(float(x))
                    biased[t] = True
                else:
                    err[b] |= ERR_TOKEN
        if tokens is not None:
            used = tokens[b, 1:n] if parent is not None else tokens[b, :n - 1]
            if ((used < 0) | (used >= V)).any():
                err[b] |= ERR_TOKEN
        if parent is not None:
            i = np.arange(1, n)
            if ((parent[b, 1:] < 0) | (parent[b, 1:] >= i)).any():
                err[b] |= ERR_PARENT
        for i in range(n):
            path = tokens_before(None if tokens is None else tokens[b], None if parent is None else parent[b], i, V)
            add = np.bincount(np.asarray(path, np.int64), minlength=V) if path else 0
            seen, made = (seen0 + add) > 0, made0 + add
            with np.errstate(all="ignore"):
                x = y[b, i]
                x1 = np.where(seen, np.where(x > 0, x / rho, x * rho), x)
                pen = np.where(made > 0, freq * made + pres, 0.0)
                x2 = np.where(made > 0, x1 - pen, x1)
                x3 = np.where(np.isneginf(x), x, np.where(biased, x2 + bias, x2))  # -inf stays -inf
                scale[b, i] = (np.abs(x1) + np.abs(freq * made) + abs(pres) + np.abs(pen) + np.abs(x2) + bias_abs
                               + np.abs(x3))
            t = seen | biased
            if mask is not None:
                row = b * n + i if mask_index is None else int(mask_index[b, i])
                if mask_index is not None and not -1 <= row < mask.shape[0]:
                    err[b] |= ERR_MASK
                    row = -1
                if row >= 0:
                    bits = np.unpackbits(np.ascontiguousarray(mask[row]).view(np.uint8), bitorder="little")[:V]
                    x3 = np.where(bits == 1, x3, -np.inf)
                    t = t | (bits == 0)
            y[b, i] = x3
            touched[b, i] = t
    return y, touched, scale, err


# ---------------------------------------------------------------------------
# 4-bit weights
# ---------------------------------------------------------------------------

def to_bf16(x):
    """float32 values -> bfloat16 bit patterns, ties to even (finite values)."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)


def bf16_values(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32)


def quantize_int4(w, group, with_zeros):
    """w float32 [V, d]; returns codes uint8 [V, d / 2], scales (bfloat16
    bits) uint16 [d / group, V], zeros uint8 [d / group, V] or None."""
    V, d = w.shape
    f = np.float32
    x = np.asarray(w, f).reshape(V, d // group, group)
    with np.errstate(all="ignore"):
        if with_zeros:
            lo, hi = np.minimum(x.min(2), f(0)), np.maximum(x.max(2), f(0))
            span = (hi - lo) / f(15)
        else:
            span = np.abs(x).max(2) / f(7)
        finite = np.isfinite(x).all(2) & np.isfinite(span)
        bits = to_bf16(np.where(finite, span, f(0)))
        over = (bits & 0x7F80) == 0x7F80  # the rounding reached infinity
        bits = np.where(finite & ~over, bits, np.uint16(0x7FC0)).astype(np.uint16)
        s = np.where(bits == 0x7FC0, f(0), bf16_values(bits))[..., None]
        q = np.where(s > 0, np.rint(x / s), f(0))
        if with_zeros:
            z = np.where(s[..., 0] > 0, np.clip(np.rint(-lo / s[..., 0]), 0, 15), f(0))
            code = np.clip(q + z[..., None], 0, 15)
        else:
            z = None
            code = np.clip(q, -8, 7) + 8
    code = code.reshape(V, d).astype(np.uint8)
    codes = code[:, 0::2] | (code[:, 1::2] << 4)
    return codes, np.ascontiguousarray(bits.T), None if z is None else np.ascontiguousarray(z.astype(np.uint8).T)


def int4_weights(codes, scales, zeros, group):
    """The values a 4-bit matrix stands for, float64 [V, d]; scales as
    bfloat16 bits."""
    V, half = codes.shape
    q = np.empty((V, 2 * half))
    q[:, 0::2] = codes & 15
    q[:, 1::2] = codes >> 4
    z = 8.0 if zeros is None else np.repeat(zeros.T.astype(np.float64), group, axis=1)
    s = np.repeat(bf16_values(scales).T.astype(np.float64), group, axis=1)
    with np.errstate(all="ignore"):
        return (q - z) * s


def int4_product(x, codes, scales, zeros, group):
    """x float [R, d] (exact values); returns (y float64 [R, V], the sums of
    the terms' magnitudes [R, V], which bound the rounding of any order)."""
    w = int4_weights(codes, scales, zeros, group)
    x = np.asarray(x, np.float64)
    return x @ w.T, np.abs(x) @ np.abs(w).T
