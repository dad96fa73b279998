"""How far the attention over a paged cache may be from its definition, from the roundings that
each key goes through. CPU only; the fp64 result is the oracle's."""
import numpy as np

from oracle import decode_oracle as ref

HALF, TINY = 2.0 ** -11, 2.0 ** -25      # fp16: half a step, relative, and below the normal range
LIFT = 7                                 # the largest weight is at least 2^7 in fp16


def attend_exact(q, k, v, seen, scale, z=None, bias=0.0):
    """One sequence: q [n, heads, dim], k and v [keys, kv, dim], seen [n, keys]; z [keys, kv]: v's
    scales (None: an fp16 cache); bias [keys, kv]: what is added to a key's codes and taken off the
    sum, as a value. Returns out and the bound of its error, both [n, heads, dim].

    Per key: the score's fp32 sum of D products, 2^-24 each of the sum of magnitudes; the exponential
    and what is added in its argument, 2^-24 of that argument and 2^-21; the weight's rounding to
    fp16, 2^-11 of it, or half of the smallest step where it is below fp16's normal range (2^-14),
    which a weight is only if it is below 2^-(14 + LIFT) of the row's largest. Those move the
    numerator by their weight in it and, where the sum is of the rounded weights, the result by
    their weight in that. fp32 sums over the keys: 2^-24 a key. The result: half a step."""
    out, size = ref.attention_ref(q, k, v, seen, scale)
    n, heads, dim = q.shape
    kv = k.shape[1]
    group = heads // kv
    bound = np.zeros_like(out)
    zs = np.ones(k.shape[:2]) if z is None else np.maximum(z.astype(np.float64), 2.0 ** -60)
    for t in range(n):
        on = np.nonzero(seen[t])[0]
        if on.size == 0:
            continue
        for h in range(heads):
            g = h // group
            kk, vv, zz = k[on, g].astype(np.float64), np.abs(v[on, g].astype(np.float64)), zs[on, g]
            a = np.abs(q[t, h].astype(np.float64))
            s = kk @ q[t, h].astype(np.float64) * scale
            reach = (np.abs(kk) + (0.0 if np.isscalar(bias) else 2 * bias[on, g, None])) @ a * abs(scale)
            p = np.exp(s - s.max())
            argument = np.abs(s).max() * 1.5 + np.abs(np.log2(zz)).max() + 2 * LIFT
            eps = (dim + 4) * 2.0 ** -24 * reach.max() + argument * 2.0 ** -24 * 2 + 2.0 ** -21
            total = p.sum()
            y = p * zz
            top = y.max()
            tail = (y < top * 2.0 ** -(14 + LIFT)) * (TINY * 2.0 ** -LIFT * top)
            codes = vv / zz[:, None]
            lost = (tail @ codes + (tail / zz).sum() * np.abs(out[t, h])) / total
            sums = (on.size + 64) * 2.0 ** -24
            bound[t, h] = ((size[t, h] + np.abs(out[t, h])) * (HALF + 2 * eps + sums) + lost +
                           HALF * np.abs(out[t, h]) + TINY)
    return out, bound


def markers(keys, kv, dim, first=0):
    """Values that count tiles: key j holds 1 at dim (j // 32) % dim of every head, else 0. With equal
    scores the result is each dim's share of the keys, so that a tile left out or taken twice moves
    its dim by one over the number of tiles that share it."""
    v = np.zeros((keys, kv, dim))
    at = first + np.arange(keys)
    v[np.arange(keys), :, at // 32 % dim] = 1.0
    return v
