"""CPU tests of the attention's error bound: it holds for results rounded as the kernels round
them, and rejects a tile of keys left out or taken twice."""
import numpy as np
import pytest

from tests.attend_bounds import LIFT, attend_exact, markers


def rounded(q, k, v, seen, scale, z=None, drop=(), twice=()):
    """The definition with weights in fp16 (lifted by 2^LIFT, v's scale in them) and the result in
    fp16; keys in `drop` left out, in `twice` taken twice."""
    out = np.zeros(q.shape)
    group = q.shape[1] // k.shape[1]
    times = np.ones(len(k))
    times[list(drop)], times[list(twice)] = 0.0, 2.0
    for t in range(q.shape[0]):
        for h in range(q.shape[1]):
            s = k[:, h // group] @ q[t, h].astype(np.float64) * scale
            zz = np.ones(len(k)) if z is None else z[:, h // group].astype(np.float64)
            y = np.where(seen[t], np.exp(s) * zz, 0.0)
            y *= 2.0 ** LIFT / y.max()
            w = y.astype(np.float16).astype(np.float64)
            total = (times * (w if z is None else y / zz)).sum()
            out[t, h] = (times * w / zz) @ v[:, h // group] / total
    return out.astype(np.float16).astype(np.float64)


@pytest.mark.parametrize("coded", [False, True])
@pytest.mark.parametrize("keys", [20011, 40001])
def test_the_bound_sees_one_tile(keys, coded):
    rng = np.random.default_rng(keys)
    dim, kv = 128, 1
    q = (0.125 * rng.standard_normal((1, 2, dim))).astype(np.float16)
    k = rng.standard_normal((keys, kv, dim)).astype(np.float16).astype(np.float64)
    z = np.full((keys, kv), 1 / 64, np.float32) if coded else None
    v, seen = markers(keys, kv, dim), np.ones((1, keys), bool)
    want, bound = attend_exact(q, k, v, seen, dim ** -0.5, z)
    good = rounded(q, k, v, seen, dim ** -0.5, z)
    assert np.all(np.abs(good - want) <= bound)
    for tile in (0, 1, keys // 64, keys // 32 - 1):
        span = range(32 * tile, 32 * tile + 32)
        for kw in (dict(drop=span), dict(twice=span)):
            bad = rounded(q, k, v, seen, dim ** -0.5, z, **kw)
            assert np.any(np.abs(bad - want) > bound), f"tile {tile} {list(kw)}"


def test_the_bound_holds_for_long_tails():
    """Weights below fp16's normal range: the bound covers them, and not their loss."""
    keys, dim = 4096, 16
    k, v = np.zeros((keys, 1, dim)), np.random.default_rng(1).uniform(0.5, 1.0, (keys, 1, dim))
    k[0, 0, 0], v[0] = 1.0, 0.0
    q = np.zeros((1, 1, dim), np.float16)
    q[..., 0] = 1.0
    seen = np.ones((1, keys), bool)
    for bits in (14.5, 20.5, 23.5):
        want, bound = attend_exact(q, k, v, seen, bits * np.log(2.0))
        assert np.all(np.abs(rounded(q, k, v, seen, bits * np.log(2.0)) - want) <= bound)
        assert np.all(want > bound)


def test_the_bound_of_rows_without_keys_is_zero():
    want, bound = attend_exact(np.ones((2, 1, 4)), np.ones((3, 1, 4)), np.ones((3, 1, 4)),
                               np.array([[True, False, True], [False] * 3]), 1.0)
    assert np.all(want[0] == 1) and np.all(want[1] == 0) and np.all(bound[1] == 0)
