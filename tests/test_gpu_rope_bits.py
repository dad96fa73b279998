"""GPU tests of the rotation's precision where fp16's last rounding does not hide it: pairs that
turn onto an axis, so that one result nearly cancels, and rows quantised after the rotation.

Before its rounding to fp16 (or to a code) a result is off by at most 2^-22 (|a| + |b|) |scale|:
2^-24 each for the angle's cosine or sine (their own half step, the angle's and the polynomial's
part), its product with the scale, the products with a and b, and their sum."""
import numpy as np
import pytest
import torch

import semi_structured_sparse_amd as nm
from oracle import decode_oracle as ref
from tests.gpu_helpers import device, say
from tests.test_gpu_decode import HALF, TINY, close, i32, up

pytestmark = pytest.mark.gpu
FINE = 2.0 ** -22


def onto_an_axis(positions, turns, heads, dim, layout, first):
    """fp16 [tokens, heads, dim] whose pairs, turned by their angle, leave their first (or second)
    element near zero; the pairs' lengths differ by head."""
    t = positions[:, None].astype(np.float64) * turns
    angle = 2.0 * np.pi * (t - np.rint(t))
    a, b = (np.sin(angle), np.cos(angle)) if first else (np.cos(angle), -np.sin(angle))
    half = len(turns)
    x = np.zeros((len(positions), heads, dim))
    size = (0.5 + np.arange(heads) / heads)[:, None]
    at = (np.s_[..., :half], np.s_[..., half:2 * half]) if layout == "half" else (np.s_[..., 0:2 * half:2], np.s_[..., 1:2 * half:2])
    x[at[0]], x[at[1]] = a[:, None] * size, b[:, None] * size
    x[..., 2 * half:] = 1.0
    return x.astype(np.float16)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("dim,rot,odd", [(128, 128, False), (64, 32, False), (128, 128, True), (80, 20, False)])
@pytest.mark.parametrize("far", [300, 1000000])
def test_results_that_nearly_cancel(layout, first, dim, rot, odd, far):
    say(f"rope bits {layout} {dim}/{rot} {far}")
    rng = np.random.default_rng(dim + rot + far)
    pos = rng.integers(-far, far, 200).astype(np.int32)
    turns = ref.rope_turns_ref(rot, base=500000.0)
    x = onto_an_axis(pos, turns, 3, dim, layout, first)
    want, size = ref.rope_ref(x, pos, turns, layout)
    given = up(x)
    if odd:                                            # the form that takes any stride
        room = torch.zeros(200, 3 * dim + 1, dtype=torch.float16, device=device())
        room[:, :3 * dim] = given.view(200, -1)
        given = room[:, :3 * dim].unflatten(1, (3, dim))
    got = nm.nm_rope(given, i32(pos), up(turns), layout=layout)
    close(got, want, HALF * np.abs(want) + FINE * size + TINY * (size > 0), f"{layout} {dim}/{rot}")


@pytest.mark.parametrize("far", [300, 1000000])
def test_as_many_results_are_the_nearest_as_in_plain_fp32(far):
    """Results that nearly cancel, against the fp16 nearest to the exact one: how many miss it says
    how large the error before the rounding is on average. Cosines and sines rounded once to fp32,
    with rounded products and difference, miss 6% and 12%; a quarter more is allowed."""
    pos = np.random.default_rng(far).integers(-far, far + 1, 20000).astype(np.int32)
    turns = ref.rope_turns_ref(128, base=500000.0)
    x = onto_an_axis(pos, turns, 1, 128, "half", True)
    nearest = ref.rope_ref(x, pos, turns)[0][..., :64].astype(np.float16)
    t = pos[:, None].astype(np.float64) * turns
    angle = 2.0 * np.pi * (t - np.rint(t))[:, None]
    c, s = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
    a, b = x[..., :64].astype(np.float32), x[..., 64:].astype(np.float32)
    plain = ((a * c - b * s).astype(np.float16) != nearest).mean()
    got = nm.nm_rope(up(x), i32(pos), up(turns)).cpu().numpy()[..., :64]
    missed = (got != nearest).mean()
    assert missed <= 1.25 * plain, f"{missed:.4f}, plain {plain:.4f}"


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("far", [300, 1000000])
def test_appended_rows_that_nearly_cancel(layout, far):
    """The same through nm_rope_kv_append: q, and k in an fp16 cache."""
    rng = np.random.default_rng(far)
    batch, tokens, heads, kv, dim = 2, 100, 4, 2, 128
    pos = rng.integers(0, far, (batch, tokens)).astype(np.int32)
    turns = ref.rope_turns_ref(dim, base=500000.0)
    x = onto_an_axis(pos.reshape(-1), turns, heads + kv, dim, layout, True).reshape(batch, tokens, heads + kv, dim)
    want, size = ref.rope_ref(x.reshape(-1, heads + kv, dim), pos.reshape(-1), turns, layout, 0.75)
    bound = (HALF * np.abs(want) + FINE * size + TINY).reshape(x.shape)
    want = want.reshape(x.shape)
    cache = nm.kv_cache(2 * 7, 16, kv, dim, device=device())
    table, fused = i32(np.arange(14).reshape(2, 7)), up(x)
    k = fused[:, :, heads:]
    q = nm.nm_rope_kv_append(cache, fused[:, :, :heads], k, k.contiguous(), i32(pos), up(turns), table, i32([0, 5]),
                             layout=layout, scale=0.75)
    close(q, want[:, :, :heads], bound[:, :, :heads], "q")
    close(nm.nm_kv_read(cache, table, i32([0, 5]), tokens)[0], want[:, :, heads:], bound[:, :, heads:], "k")


@pytest.mark.parametrize("form", ["int8", "e4m3"])
def test_codes_of_rotated_rows(form):
    """A code is the rounding of the exact row, unless that lies within the rotation's error of a
    border (then one of the two): 2^-22 (|a| + |b|) and the product's and quotient's 2^-23."""
    rng = np.random.default_rng(11)
    tokens, kv, dim = 500, 2, 128
    most = 127.0 if form == "int8" else 448.0
    pos = rng.integers(0, 100000, (1, tokens)).astype(np.int32)
    turns = ref.rope_turns_ref(dim, base=500000.0)
    k = rng.standard_normal((1, tokens, kv, dim)).astype(np.float16)
    cache = nm.kv_cache(32, 16, kv, dim, torch.int8 if form == "int8" else torch.float8_e4m3fn, device())
    nm.nm_rope_kv_append(cache, None, up(k), up(k), i32(pos), up(turns), i32(np.arange(32)[None]), i32([0]))
    torch.cuda.synchronize()
    at = np.arange(tokens)
    codes = (cache.k.cpu().numpy().astype(np.float64) if form == "int8" else
             ref.e4m3_table()[cache.k.view(torch.uint8).cpu().numpy()])[at // 16, :, at % 16]
    want, size = ref.rope_ref(k[0], pos[0], turns)
    amax = np.abs(want).max(-1, keepdims=True)
    exact = want / amax * most
    slack = (FINE * size / amax * most + np.abs(exact) * (FINE * size.max(-1, keepdims=True) / amax + 2.0 ** -22))

    def rounded(y):
        if form == "int8":
            return np.rint(y)
        return torch.from_numpy(np.clip(y, -448, 448)).to(torch.float32).to(torch.float8_e4m3fn).double().numpy()

    low, high = rounded(exact - slack), rounded(exact + slack)
    assert np.all((codes >= low) & (codes <= high))
    assert (low != high).mean() < 2e-3            # nearly all codes are pinned
