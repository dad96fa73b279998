"""The block products' gelu, followed step by step in fp32 on the CPU. v_rcp_f32 and v_exp_f32 are good to
1 ulp, so each takes a step either way.

How far it may be from x Phi(x), in U = 2^-24 of the result: the fit 1.6; t = 1 / (1 + k |x|) 3 (a rounding and
1 ulp), which the product t P(t), whose relative slope is below 2, takes as 6; the polynomial's roundings 3 (its
terms are at most twice their sum); three products 3, exp 2, the subtraction 1 (Q is at most as large as the
result): 18 with its last digit; and the exponent x^2 / 2 has 2.5 roundings of its own size, 1.25 x^2."""
import itertools
import math
import os
import re

import numpy as np
import pytest
import torch

F = np.float32
U = 2.0 ** -24
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def fma(a, b, c):
    # products of two fp32 values are exact in 64 bits; the sum's second rounding is 2^-29 of fp32's
    return (np.asarray(a, np.float64) * np.asarray(b, np.float64) + np.asarray(c, np.float64)).astype(F)


def moved(x, ulps):
    return x if ulps == 0 else np.nextafter(x, F(np.inf if ulps > 0 else -np.inf))


def source():
    """The factor k of t = 1 / (1 + k |x|) and the polynomial's coefficients, as the header has them."""
    with open(os.path.join(ROOT, "semi_structured_sparse_amd", "csrc", "nm_epilogue.h")) as f:
        body = re.search(r"float gelu\(float x\) \{(.*?)\n\}", f.read(), re.S).group(1)
    k = re.search(r"fmaf\(w, ([0-9.e+-]+)f, 1\.0f\)", body).group(1)
    first = re.search(r"float p = ([0-9.e+-]+)f;", body).group(1)
    return F(k), [F(c) for c in [first, *re.findall(r"p = fmaf\(p, t, ([0-9.e+-]+)f\);", body)]]


@pytest.mark.parametrize("rcp,exp", itertools.product((-1, 0, 1), repeat=2))
def test_gelu_is_within_its_roundings(rcp, exp):
    k, coefficients = source()
    assert len(coefficients) == 8
    x = np.concatenate([np.linspace(-7.7, 7.7, 400001), np.geomspace(1e-6, 1, 2001), -np.geomspace(1e-6, 1, 2001)]).astype(F)
    w = np.abs(x)
    t = moved((1.0 / fma(w, k, 1.0).astype(np.float64)).astype(F), rcp)
    p = np.full_like(x, coefficients[0])
    for c in coefficients[1:]:
        p = fma(p, t, c)
    power = (w * w) * F(-0.72134752044448170)
    e = moved(np.exp2(power.astype(np.float64)).astype(F), exp)
    y = np.where(x < 0, F(0), x) - w * t * p * e
    x = x.astype(np.float64)
    want = 0.5 * x * torch.special.erfc(torch.from_numpy(-x * math.sqrt(0.5))).numpy()
    off = np.abs(y - want)
    allowed = (18.0 + 1.25 * x * x) * U * np.abs(want)
    assert (off <= allowed).all(), f"{(off / np.maximum(allowed, 1e-300)).max():.3g} of the allowed distance"
