"""CPU oracle of the speculative-decoding operators, in fp64 numpy, from their definitions
(include/nm_decode.h); it shares no code with the GPU path. Loops over tokens and heads are
spelled out where that keeps the definition readable."""
from __future__ import annotations

import numpy as np

LARGEST = {"int8": 127.0, "e4m3": 448.0}


def e4m3_table() -> np.ndarray:
    """The 256 values of the OCP e4m3 codes (fp64; codes 0x7F and 0xFF are NaN)."""
    out = np.empty(256, np.float64)
    for c in range(256):
        exp, frac = (c >> 3) & 15, c & 7
        v = frac * 2.0 ** -9 if exp == 0 else (8 + frac) * 2.0 ** (exp - 10)
        out[c] = np.nan if (c & 0x7F) == 0x7F else (-v if c & 0x80 else v)
    return out


def rope_turns_ref(rot_dim, base=10000.0, scaling="plain", factor=1.0, length=8192.0, low=1.0, high=4.0):
    i = np.arange(rot_dim // 2, dtype=np.float64)
    if scaling == "base":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    t = np.exp(-2.0 * i / rot_dim * np.log(base)) / (2.0 * np.pi)
    if scaling == "linear":
        t = t / factor
    if scaling == "bands":
        w = np.clip((length * t - low) / (high - low), 0.0, 1.0)
        t = t * w + t / factor * (1.0 - w)
    return t


def rope_ref(x, positions, turns, layout="half", scale=1.0):
    """x [tokens, heads, dim] turned in fp64; also the pairs' |a| + |b| per element (for error
    bounds), zero where nothing is turned."""
    x = np.asarray(x, np.float64)
    half = len(turns)
    t = np.asarray(positions, np.float64)[:, None] * np.asarray(turns, np.float64)
    angle = 2.0 * np.pi * (t - np.rint(t))
    c, s = np.cos(angle)[:, None] * scale, np.sin(angle)[:, None] * scale
    first = np.s_[..., :half] if layout == "half" else np.s_[..., 0:2 * half:2]
    second = np.s_[..., half:2 * half] if layout == "half" else np.s_[..., 1:2 * half:2]
    y, size = x.copy(), np.zeros_like(x)
    a, b = x[first], x[second]
    y[first], y[second] = a * c - b * s, b * c + a * s
    size[first] = size[second] = (np.abs(a) + np.abs(b)) * abs(scale)
    return y, size


def rows_of(table, page, b, positions):
    """(block, slot) of a sequence's positions."""
    return table[b, np.asarray(positions) // page], np.asarray(positions) % page


def attention_ref(q, k, v, seen, scale):
    """One sequence: q [n, heads, dim], k and v [keys, kv, dim], seen [n, keys] truth. Returns out
    and sum_j p_j |v_j| (for error bounds), both [n, heads, dim]; zeros where nothing is seen.
    Unseen keys are left out, whatever they hold."""
    q = np.asarray(q, np.float64)
    n, heads, dim = q.shape
    group = heads // k.shape[1]
    out, size = np.zeros_like(q), np.zeros_like(q)
    for t in range(n):
        on = np.nonzero(seen[t])[0]
        if on.size == 0:
            continue
        for g in range(k.shape[1]):
            kk, vv = k[on, g].astype(np.float64), v[on, g].astype(np.float64)
            s = q[t, g * group:(g + 1) * group] @ kk.T * scale
            w = np.exp(s - s.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            out[t, g * group:(g + 1) * group] = w @ vv
            size[t, g * group:(g + 1) * group] = w @ np.abs(vv)
    return out, size


def tree_seen(context, count, masks):
    """[count, context + count] truth from mask words (None: a chain)."""
    seen = np.ones((count, context + count), bool)
    for t in range(count):
        word = (2 << t) - 1 if masks is None else int(masks[t]) & (2 ** 64 - 1)
        for i in range(count):
            seen[t, context + i] = bool((word >> i) & 1)
    return seen


def _weight(x):
    x = np.asarray(x, np.float64)
    return np.where(np.isfinite(x) & (x > 0), x, 0.0)


def draw_ref(weights, uniform) -> int:
    """The first index whose running sum exceeds uniform * total; -1 if no weight is left."""
    running = np.cumsum(weights)
    if not running[-1] > 0:
        return -1
    over = np.nonzero(running > float(uniform) * running[-1])[0]
    return int(over[0]) if over.size else int(np.nonzero(weights)[0][-1])


def verify_chain_ref(target, draft, tokens, uniforms, count):
    """One sequence: (accepted, out_tokens [nodes])."""
    nodes, vocab = target.shape
    out = np.full(nodes, -1, np.int64)
    if count == 0:
        return 0, out
    m = 0
    while m < count - 1:
        x = int(tokens[m + 1])
        if not 0 <= x < vocab or not float(uniforms[m + 1]) * float(draft[m, x]) < float(target[m, x]):
            break
        m += 1
    out[:m] = tokens[1:m + 1]
    token = -1
    if m < count - 1:
        token = draw_ref(_weight(target[m].astype(np.float64) - draft[m].astype(np.float64)), uniforms[0])
    if token < 0:
        token = draw_ref(_weight(target[m]), uniforms[0])
    out[m] = token
    return m, out


def verify_tree_ref(target, tokens, parents, uniforms, count):
    """One sequence: (accepted, out_tokens [nodes], path [nodes])."""
    nodes, vocab = target.shape
    out, path = np.full(nodes, -1, np.int64), np.full(nodes, -1, np.int64)
    if count == 0:
        return 0, out, path
    at, m, reached = 0, 0, [0]
    while True:
        refused, left, nxt = [], 1.0, -1
        for c in range(at + 1, count):
            x = int(tokens[c])
            if parents[c] != at or not 0 <= x < vocab:
                continue
            p = 0.0 if x in refused else float(_weight(target[at, x]))
            if float(uniforms[c]) * left < p:
                nxt = c
                break
            left -= p
            refused.append(x)
        if nxt < 0:
            break
        out[m] = tokens[nxt]
        m, at = m + 1, nxt
        reached.append(nxt)
    rest = _weight(target[at])
    rest[refused] = 0.0
    token = draw_ref(rest, uniforms[0])
    out[m] = token if token >= 0 else draw_ref(_weight(target[at]), uniforms[0])
    path[:m + 1] = reached
    return m, out, path
