"""GPU tests of the speculative-decoding operators against the fp64 oracle.

Tolerances, derived from the roundings each operator makes (fp16 half step: 2^-11 relative,
2^-25 absolute below the normal range):
  rope    one rounding to fp16; sine and cosine in fp32 to within 2^-19 of a unit, products in
          fp32: 2^-11 |y| + 2^-18 (|a| + |b|) + 2^-25
  cache   8-bit rows without rotation hold exactly the codes and scales the definition gives in
          fp32; reading rounds code * scale once. With the rotation the row is off by the above
          (without the fp16 step), then by half a code step.
  attend  each weight is rounded to fp16 (2^-11 relative; 2^-25 of v's largest scale for the
          smallest weights), the score's fp32 sum is off by at most (D + 4) 2^-24 of the sum of
          magnitudes, exponentials and the running rescales by 2^-20 together
  verify  whole numbers, equal
"""
import numpy as np
import pytest
import torch

import semi_structured_sparse_amd as nm
from oracle import decode_oracle as ref
from tests.gpu_helpers import device, say

pytestmark = pytest.mark.gpu
HALF, TINY = 2.0 ** -11, 2.0 ** -25
FORMATS = {"fp16": torch.float16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(device())


def i32(a):
    return up(np.asarray(a, np.int32))


def halves(rng, *shape):
    return rng.standard_normal(shape).astype(np.float16)


def close(got, want, bound, tag):
    got = got.cpu().numpy().astype(np.float64) if torch.is_tensor(got) else got
    err = np.abs(got - want)
    worst = np.max(err / bound) if err.size else 0.0
    assert np.all(err <= bound), f"{tag}: worst {worst:.3g} of the bound"
    return worst


# ------------------------------------------------------------------------------------ rope
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,heads,dim,rot", [
    (1, 1, 128, 128), (3, 5, 64, 64), (7, 3, 128, 64), (2, 9, 256, 32), (5, 2, 80, 20), (4, 3, 33, 32), (3, 2, 6, 2),
    (2, 1, 1024, 1024), (1, 2, 96, 96), (65, 40, 128, 128), (3, 1, 112, 112), (2, 3, 48, 16)])
def test_rope(layout, tokens, heads, dim, rot):
    say(f"rope {layout} {tokens}x{heads}x{dim}/{rot}")
    rng = np.random.default_rng(tokens * 1000 + dim + rot)
    x = halves(rng, tokens, heads, dim)
    pos = rng.integers(0, 1000000, tokens).astype(np.int32)
    pos[0] = -7
    pos[-1] = 131071
    turns = ref.rope_turns_ref(rot, base=500000.0)
    want, size = ref.rope_ref(x, pos, turns, layout, 1.25)
    got = nm.nm_rope(up(x), i32(pos), up(turns), layout=layout, scale=1.25)
    torch.cuda.synchronize()
    close(got, want, HALF * np.abs(want) + 2.0 ** -18 * size + TINY * (size > 0), f"{layout} {dim}/{rot}")
    assert np.array_equal(got.cpu().numpy()[..., rot:], x[..., rot:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_slices_and_in_place(layout):
    """q and k as one slice of a fused projection's rows, out of place and in place; the rest of
    the rows untouched."""
    rng = np.random.default_rng(5)
    fused = halves(rng, 9, 12, 128)
    pos, turns = np.arange(100, 109, dtype=np.int32), ref.rope_turns_ref(128)
    want, size = ref.rope_ref(fused[:, 1:9], pos, turns, layout)
    bound = HALF * np.abs(want) + 2.0 ** -18 * size + TINY
    f = up(fused)
    close(nm.nm_rope(f[:, 1:9], i32(pos), up(turns), layout=layout), want, bound, "slice")
    back = nm.nm_rope(f[:, 1:9], i32(pos), up(turns), layout=layout, out=f[:, 1:9])
    assert back.data_ptr() == f[:, 1:9].data_ptr()
    torch.cuda.synchronize()
    close(f[:, 1:9], want, bound, "in place")
    assert np.array_equal(f.cpu().numpy()[:, :1], fused[:, :1]) and np.array_equal(f.cpu().numpy()[:, 9:], fused[:, 9:])
    # an odd element offset and an odd stride take the narrow path
    flat = torch.zeros(9 * 1025 + 1, dtype=torch.float16, device=device())
    odd = flat[1:].as_strided((9, 8, 128), (1025, 128, 1))
    odd.copy_(up(fused[:, 1:9]))
    close(nm.nm_rope(odd, i32(pos), up(turns), layout=layout), want, bound, "odd")


def test_rope_turns_back():
    """Negative positions undo positive ones (the transposed map), up to two roundings."""
    rng = np.random.default_rng(6)
    x = halves(rng, 16, 4, 128)
    pos = rng.integers(1, 100000, 16).astype(np.int32)
    turns = nm.rope_turns(128, device=device())
    y = nm.nm_rope(nm.nm_rope(up(x), i32(pos), turns), i32(-pos), turns)
    size = ref.rope_ref(x, pos, turns.cpu().numpy())[1]
    close(y, x.astype(np.float64), 4 * HALF * size + TINY * 4, "back")


def test_rope_far_positions():
    """2^31 - 1 positions at one turn in 2 pi keep their fraction."""
    x = np.ones((2, 1, 64), np.float16)
    pos = np.array([2 ** 31 - 1, -2 ** 31], np.int32)
    turns = ref.rope_turns_ref(64)
    want, size = ref.rope_ref(x, pos, turns)
    close(nm.nm_rope(up(x), i32(pos), up(turns)), want, HALF * np.abs(want) + 2.0 ** -18 * size + TINY, "far")


# ----------------------------------------------------------------------------------- cache
class Paged:
    """A cache of random contents with a shuffled page table; its host copy decodes to fp64."""

    def __init__(self, rng, batch, pages, page, kv, dim, form, spare=3):
        self.page, self.form, self.dim = page, form, dim
        self.blocks = batch * pages + spare
        self.table = rng.permutation(self.blocks)[:batch * pages].reshape(batch, pages).astype(np.int32)
        shape = (self.blocks, kv, page, dim)
        if form == "fp16":
            k, v = (up(halves(rng, *shape)) for _ in range(2))
            self.cache = nm.KVCache(k, v)
        else:
            raw = [rng.integers(-127, 128, shape).astype(np.int8) if form == "int8" else
                   rng.integers(0, 127, shape).astype(np.uint8) | (rng.integers(0, 2, shape) << 7).astype(np.uint8)
                   for _ in range(2)]
            scales = [(0.5 + rng.random(shape[:3])).astype(np.float32) * (2.0 ** -6 if form == "int8" else 2.0 ** -8)
                      for _ in range(2)]
            self.cache = nm.KVCache(*(up(r).view(FORMATS[form]) for r in raw), *(up(s) for s in scales))

    def values(self):
        out = []
        for codes, scale in ((self.cache.k, self.cache.k_scale), (self.cache.v, self.cache.v_scale)):
            if self.form == "e4m3":
                x = ref.e4m3_table()[codes.view(torch.uint8).cpu().numpy()]
            else:
                x = codes.cpu().numpy().astype(np.float64)
            out.append(x if scale is None else x * scale.cpu().numpy().astype(np.float64)[..., None])
        return out

    def rows(self, values, b, positions):
        block, slot = ref.rows_of(self.table, self.page, b, positions)
        return values[block, :, slot]


def expected_codes(x, form):
    """Codes and scales of fp32 rows, by the definition in fp32 (torch on the CPU)."""
    x = torch.from_numpy(np.ascontiguousarray(x)).float()
    if form == "fp16":
        return x.half(), None
    most = 127.0 if form == "int8" else 448.0
    amax = x.abs().amax(-1, keepdim=True)
    held = amax >= 1e-30
    y = torch.where(held, x * (torch.tensor(most) / amax.clamp(min=1e-30)), torch.zeros_like(x)).clamp(-most, most)
    codes = y.round().to(torch.int8) if form == "int8" else y.to(torch.float8_e4m3fn)
    return codes, torch.where(held, amax / most, torch.zeros_like(amax))[..., 0]


@pytest.mark.parametrize("form", list(FORMATS))
@pytest.mark.parametrize("batch,tokens,kv,dim,page", [(1, 1, 1, 128, 16), (3, 5, 2, 64, 16), (2, 37, 3, 128, 32),
                                                       (4, 1, 8, 128, 64), (2, 19, 1, 256, 16), (1, 300, 2, 64, 128)])
def test_append_and_read(form, batch, tokens, kv, dim, page):
    say(f"append {form} {batch}x{tokens}x{kv}x{dim} page {page}")
    rng = np.random.default_rng(batch * 100 + tokens)
    pages = -(-(tokens + 40) // page)
    p = Paged(rng, batch, pages, page, kv, dim, form)
    start = rng.integers(0, 40, batch).astype(np.int32)
    count = rng.integers(0, tokens + 1, batch).astype(np.int32)
    count[0] = tokens
    k, v = halves(rng, batch, tokens, kv, dim), halves(rng, batch, tokens, kv, dim)
    k[0, 0, 0] = 0.0                                     # a row of zeros
    v[0, 0, 0, 1:] *= 2.0 ** -12                         # subnormal halves next to a normal one
    before = [c.view(torch.uint8 if form != "fp16" else torch.int16).cpu().numpy().copy() for c in p.cache[:2]]
    nm.nm_kv_append(p.cache, up(k), up(v), up(p.table), i32(start), i32(count))
    torch.cuda.synchronize()
    after = [c.view(torch.uint8 if form != "fp16" else torch.int16).cpu().numpy() for c in p.cache[:2]]
    touched = np.zeros((p.blocks, page), bool)
    for side, x, scale in ((0, k, p.cache.k_scale), (1, v, p.cache.v_scale)):
        codes, scales = expected_codes(x, form)
        codes = codes.view(torch.uint8 if form != "fp16" else torch.int16).numpy()
        for b in range(batch):
            at = start[b] + np.arange(count[b])
            block, slot = ref.rows_of(p.table, page, b, at)
            touched[block, slot] = True
            assert np.array_equal(after[side][block, :, slot], codes[b, :count[b]])
            if scales is not None:
                assert np.array_equal(scale.cpu().numpy()[block, :, slot], scales.numpy()[b, :count[b]])
    for side in range(2):                                # nothing else was written
        keep = ~np.broadcast_to(touched[:, None, :], after[side].shape[:3])
        assert np.array_equal(after[side][keep], before[side][keep])
    got_k, got_v = nm.nm_kv_read(p.cache, up(p.table), i32(start), tokens, i32(count))
    values = p.values()
    for got, val in ((got_k, values[0]), (got_v, values[1])):
        got = got.cpu().numpy().astype(np.float64)
        for b in range(batch):
            want = p.rows(val, b, start[b] + np.arange(count[b]))
            close(got[b, :count[b]], want, HALF * np.abs(want) + TINY, f"read {form}")
            assert np.all(got[b, count[b]:] == 0)


@pytest.mark.parametrize("form", list(FORMATS))
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim,rot,heads,kv,tokens", [(128, 128, 8, 2, 3), (64, 32, 4, 4, 1), (256, 256, 2, 1, 17),
                                                       (128, 16, 0, 3, 2), (64, 64, 5, 5, 70), (256, 48, 3, 1, 2)])
def test_rope_append(form, layout, dim, rot, heads, kv, tokens):
    say(f"rope append {form} {layout} {dim}/{rot}")
    rng = np.random.default_rng(dim + rot + tokens)
    batch, page = 3, 16
    p = Paged(rng, batch, -(-(tokens + 20) // page), page, kv, dim, form)
    fused = halves(rng, batch, tokens, heads + 2 * kv, dim)
    start = np.array([0, 13, 20], np.int32)
    count = np.array([tokens, max(0, tokens - 1), tokens], np.int32)
    pos = (start[:, None] + rng.integers(0, 5000, (batch, tokens))).astype(np.int32)
    turns = ref.rope_turns_ref(rot)
    f = up(fused)
    q = f[:, :, :heads] if heads else None
    out = nm.nm_rope_kv_append(p.cache, q, f[:, :, heads:heads + kv], f[:, :, heads + kv:], i32(pos), up(turns),
                               up(p.table), i32(start), i32(count), layout=layout, scale=0.75)
    got_k, got_v = nm.nm_kv_read(p.cache, up(p.table), i32(start), tokens, i32(count))
    torch.cuda.synchronize()
    flat = fused.reshape(batch * tokens, -1, dim)
    turned, size = ref.rope_ref(flat[:, :heads + kv], pos.reshape(-1), turns, layout, 0.75)
    turned, size = (a.reshape(batch, tokens, heads + kv, dim) for a in (turned, size))
    live = np.arange(tokens)[None, :] < count[:, None]
    if heads:
        want = turned[:, :, :heads] * live[..., None, None]
        close(out, want, HALF * np.abs(want) + 2.0 ** -18 * size[:, :, :heads] + TINY, "q")
    else:
        assert out is None
    for got, x, extra in ((got_k, turned[:, :, heads:], 2.0 ** -18 * size[:, :, heads:]),
                          (got_v, fused[:, :, heads + kv:].astype(np.float64), 0.0)):
        amax = np.abs(x).max(-1, keepdims=True)
        # half a step of the code, widened for the row's own error and fp32 steps
        step = {"fp16": 0.0 * amax + TINY, "int8": amax / 254, "e4m3": 2.0 ** -4 * np.abs(x) + amax * 2.0 ** -10 / 448}[form]
        bound = (1 + 2.0 ** -10) * (step + extra) + 2 * HALF * (np.abs(x) + step) + TINY
        x = x * live[..., None, None]
        close(got, x, bound, f"k or v {form}")


def test_rope_append_in_place():
    rng = np.random.default_rng(8)
    p = Paged(rng, 2, 2, 16, 2, 128, "int8")
    fused = up(halves(rng, 2, 4, 8, 128))
    q, k, v = fused[:, :, :4], fused[:, :, 4:6], fused[:, :, 6:]
    args = (i32(np.arange(8).reshape(2, 4)), nm.rope_turns(128, device=device()), up(p.table), i32([0, 3]))
    want = nm.nm_rope_kv_append(p.cache, q, k, v, *args)
    got = nm.nm_rope_kv_append(p.cache, q, k, v, *args, out=q)
    assert got.data_ptr() == q.data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("form", list(FORMATS))
def test_cache_bad_pages_and_positions(form):
    """Table entries and positions out of range are skipped by writes and read as zeros."""
    rng = np.random.default_rng(9)
    p = Paged(rng, 2, 3, 16, 2, 64, form)
    table = p.table.copy()
    table[0, 1], table[1, 0], table[1, 2] = -1, p.blocks, 2 ** 31 - 1
    k = up(halves(rng, 2, 48, 2, 64))
    before = [c.view(torch.uint8 if form != "fp16" else torch.int16).cpu().numpy().copy() for c in p.cache[:2]]
    nm.nm_kv_append(p.cache, k, k, up(table), i32([0, -8]), None)
    torch.cuda.synchronize()
    after = [c.view(torch.uint8 if form != "fp16" else torch.int16).cpu().numpy() for c in p.cache[:2]]
    written = {p.table[0, 0], p.table[0, 2], p.table[1, 1]}
    for side in range(2):
        for block in range(p.blocks):
            same = np.array_equal(after[side][block], before[side][block])
            assert same != (block in written), f"block {block}"
    got, _ = nm.nm_kv_read(p.cache, up(table), i32([0, -8]), 48)
    got = got.cpu().numpy()
    assert np.all(got[0, 16:32] == 0) and np.all(got[1, :24] == 0) and np.all(got[1, 40:] == 0)
    assert np.any(got[0, :16] != 0) and np.any(got[0, 32:] != 0) and np.any(got[1, 24:40] != 0)
    got, _ = nm.nm_kv_read(p.cache, up(p.table), i32([40, 2 ** 31 - 20]), 48)
    assert np.all(got.cpu().numpy()[0, 8:] == 0) and np.all(got.cpu().numpy()[1] == 0)


@pytest.mark.parametrize("form", ["int8", "e4m3"])
def test_cache_holds_non_finite_rows_as_nan(form):
    rng = np.random.default_rng(10)
    p = Paged(rng, 1, 1, 16, 2, 64, form)
    k = halves(rng, 1, 3, 2, 64)
    k[0, 0, 0, 5], k[0, 1, 1, 63] = np.inf, np.nan
    nm.nm_kv_append(p.cache, up(k), up(k), up(p.table), i32([0]))
    got = nm.nm_kv_read(p.cache, up(p.table), i32([0]), 3)[0].cpu().numpy()
    bad = np.zeros((3, 2), bool)
    bad[0, 0] = bad[1, 1] = True
    assert np.array_equal(np.isnan(got[0]).all(-1), bad) and np.array_equal(np.isnan(got[0]).any(-1), bad)


@pytest.mark.parametrize("form", list(FORMATS))
@pytest.mark.parametrize("dim,nodes,page", [(128, 24, 16), (64, 64, 32), (256, 64, 16), (128, 1, 16)])
def test_compact(form, dim, nodes, page):
    rng = np.random.default_rng(nodes + dim)
    batch, kv = 4, 3
    p = Paged(rng, batch, -(-(nodes + 50) // page), page, kv, dim, form)
    start = np.array([0, 15, 50, 7], np.int32)
    path = np.full((batch, nodes), -1, np.int32)
    accepted = np.zeros(batch, np.int32)
    for b in range(batch):
        nodes_on = np.sort(rng.choice(np.arange(1, nodes), size=rng.integers(0, nodes), replace=False)) if nodes > 1 else []
        path[b, 0] = 0
        path[b, 1:1 + len(nodes_on)] = nodes_on
        accepted[b] = len(nodes_on)
    path[3], accepted[3] = np.concatenate([[0], rng.permutation(np.arange(1, nodes))]), nodes - 1   # any order
    before = p.values()
    nm.nm_kv_compact(p.cache, up(p.table), i32(start), i32(path), i32(accepted))
    torch.cuda.synchronize()
    after = p.values()
    for old, new in zip(before, after):
        want = old.copy()
        for b in range(batch):
            d = np.arange(1, accepted[b] + 1)
            block, slot = ref.rows_of(p.table, page, b, start[b] + d)
            want[block, :, slot] = p.rows(old, b, start[b] + path[b, d])
        assert np.array_equal(new, want)


def test_compact_leaves_bad_entries_alone():
    rng = np.random.default_rng(12)
    p = Paged(rng, 1, 1, 16, 1, 64, "int8")
    before = p.values()
    nm.nm_kv_compact(p.cache, up(p.table), i32([12]), i32([[0, 7, -1, 9, 3, 3]]), i32([99]))
    torch.cuda.synchronize()
    after = p.values()
    for old, new in zip(before, after):       # 12+1 <- 19 (past the table), 14 <- bad, 15 <- 21, 16 ...: nothing
        assert np.array_equal(old, new)


# --------------------------------------------------------------------------------- attend
def attend_case(rng, p, context, tokens, heads, count=None, masks=None, scale=None, workspace=True, q=None, tag=""):
    """Runs the attention on the paged cache p and checks it against the oracle."""
    batch = len(context)
    kv, dim = p.cache.k.shape[1], p.dim
    if q is None:
        q = halves(rng, batch, tokens, heads, dim)
    counts = np.full(batch, tokens) if count is None else np.asarray(count)
    qd, table = up(q), up(p.table)
    ws = nm.tree_attention_workspace(qd, p.cache, table) if workspace else None
    got = nm.nm_tree_attention(qd, p.cache, table, i32(context),
                               mask=None if masks is None else up(np.asarray(masks, np.uint64).view(np.int64)),
                               count=None if count is None else i32(count), scale=scale, workspace=ws)
    torch.cuda.synchronize()
    if ws is not None:
        assert not ws[:65536].any(), "counters are left at zero"
    out = got.cpu().numpy().astype(np.float64)
    k, v = p.values()
    s = 1.0 / np.sqrt(dim) if scale is None else scale
    for b in range(batch):
        n = counts[b]
        keys = context[b] + n
        kk, vv = p.rows(k, b, np.arange(keys)), p.rows(v, b, np.arange(keys))
        seen = ref.tree_seen(context[b], n, None if masks is None else masks[b])
        want, size = ref.attention_ref(q[b, :n], kk, vv, seen, s)
        bound = attend_bound(q[b, :n], kk, vv, s, want, size)
        close(out[b, :n], want, bound, f"{tag} sequence {b}")
        assert np.all(out[b, n:] == 0)
    return got


def attend_bound(q, k, v, scale, want, size):
    group = q.shape[1] // k.shape[1]
    dim = q.shape[-1]
    kk = np.nan_to_num(np.abs(k).max(0), posinf=0.0) if k.shape[0] else np.zeros(k.shape[1:])
    reach = np.einsum("nhd,hd->nh", np.abs(q.astype(np.float64)), np.repeat(kk, group, 0)) * abs(scale)
    scores = (dim + 4) * 2.0 ** -24 * reach
    vmax = np.repeat(np.nan_to_num(np.abs(v), posinf=0.0).max((0, 2)) if v.shape[0] else np.zeros(k.shape[1]), group)
    return (HALF * np.abs(want) + size * (HALF + 2.0 ** -20 + 2 * scores[..., None]) +
            max(1, k.shape[0]) * TINY * vmax[None, :, None] + TINY)


def tree_masks(rng, batch, tokens):
    """Random trees as mask words (a node sees itself and the nodes above it)."""
    masks = np.zeros((batch, tokens), object)
    for b in range(batch):
        for t in range(tokens):
            above = masks[b, rng.integers(max(0, t - 4), t)] if t else 0
            masks[b, t] = int(above) | (1 << t)
    return masks.astype(np.uint64)


@pytest.mark.parametrize("form", list(FORMATS))
@pytest.mark.parametrize("heads,kv,dim,page", [(32, 8, 128, 16), (4, 4, 64, 32), (10, 2, 128, 64), (8, 1, 256, 16),
                                                (16, 1, 64, 16), (3, 1, 128, 1024)])
@pytest.mark.parametrize("context", [[0], [1, 31, 32, 33], [777], [1000, 5, 127, 128, 129]])
def test_attend_single_token(form, heads, kv, dim, page, context):
    say(f"attend 1 {form} {heads}/{kv} {dim} page {page} context {context}")
    rng = np.random.default_rng(sum(context) + heads)
    p = Paged(rng, len(context), -(-(max(context) + 1) // page), page, kv, dim, form)
    attend_case(rng, p, context, 1, heads, tag=f"{form} {heads}/{kv} {dim}")


@pytest.mark.parametrize("form", list(FORMATS))
@pytest.mark.parametrize("heads,kv,dim,page,tokens", [(8, 2, 128, 16, 2), (8, 2, 64, 32, 5), (64, 8, 128, 32, 24),
                                                        (5, 1, 256, 16, 9), (8, 1, 128, 64, 64), (2, 2, 64, 16, 33),
                                                        (16, 1, 64, 16, 64), (10, 2, 128, 128, 13)])
@pytest.mark.parametrize("masked", [False, True])
def test_attend_nodes(form, heads, kv, dim, page, tokens, masked):
    say(f"attend {tokens} {form} {heads}/{kv} {dim} page {page} tree {masked}")
    rng = np.random.default_rng(tokens + heads + dim)
    context = [0, 1, 40, 333]
    p = Paged(rng, 4, -(-(max(context) + tokens) // page), page, kv, dim, form)
    masks = tree_masks(rng, 4, tokens) if masked else None
    attend_case(rng, p, context, tokens, heads, masks=masks, tag=f"{form} tree {masked}")
    attend_case(rng, p, context, tokens, heads, masks=masks, workspace=False, tag="no workspace")
    attend_case(rng, p, context, tokens, heads, count=[tokens, 0, max(1, tokens - 3), 1], masks=masks, tag="counts")


@pytest.mark.parametrize("form", list(FORMATS))
def test_attend_long_contexts(form):
    say(f"attend long {form}")
    rng = np.random.default_rng(77)
    context = [20011, 64, 9999]
    p = Paged(rng, 3, -(-(max(context) + 7) // 64), 64, 2, 128, form)
    attend_case(rng, p, context, 7, 8, tag=f"long {form}")
    attend_case(rng, p, context, 7, 8, workspace=False, tag=f"long, no workspace {form}")
    attend_case(rng, p, context, 1, 2, tag=f"long single {form}")


def test_attend_many_sequences():
    rng = np.random.default_rng(78)
    context = rng.integers(0, 200, 130).tolist()
    p = Paged(rng, 130, 14, 16, 2, 64, "int8")
    attend_case(rng, p, context, 3, 4, tag="130 sequences")


@pytest.mark.parametrize("form", list(FORMATS))
def test_attend_rows_without_keys(form):
    """Nodes whose mask leaves nothing over an empty context give zeros."""
    rng = np.random.default_rng(79)
    p = Paged(rng, 2, 2, 16, 2, 128, form)
    masks = np.array([[1, 0, 5, 0], [0, 0, 0, 0]], np.uint64)
    got = attend_case(rng, p, [0, 0], 4, 4, masks=masks, tag="empty rows")
    assert not got[1].any() and not got[0, 1].any() and got[0, 0].any()


@pytest.mark.parametrize("form", list(FORMATS))
def test_attend_ignores_what_is_not_seen(form):
    """NaN and infinities in slots past the end, in drafts that a node does not see, and in their
    scales do not reach a result; the nodes that see a poisoned draft get NaN."""
    rng = np.random.default_rng(80)
    context, tokens = [37, 0, 20], 6
    p = Paged(rng, 3, 4, 16, 2, 128, form)
    masks = np.tile(np.array([1, 3, 5, 9, 17, 33], np.uint64), (3, 1))    # node 0 and itself
    q = halves(rng, 3, tokens, 4, 128)
    clean = attend_case(rng, p, context, tokens, 4, masks=masks, q=q, tag="clean").cpu().numpy()
    for b in range(3):
        for j in list(range(context[b] + tokens, 64)) + [context[b] + 3]:
            block, slot = p.table[b, j // 16], j % 16
            for codes, scale in ((p.cache.k, p.cache.k_scale), (p.cache.v, p.cache.v_scale)):
                if form == "fp16":
                    codes[block, :, slot] = float("inf") if j % 2 else float("nan")
                else:
                    if form == "e4m3" and j >= context[b] + tokens:
                        codes.view(torch.uint8)[block, :, slot] = 0x7F
                    scale[block, :, slot] = float("inf") if j >= context[b] + tokens and j % 2 else float("nan")
    ws = nm.tree_attention_workspace(up(q), p.cache, up(p.table))
    for w in (ws, None):
        got = nm.nm_tree_attention(up(q), p.cache, up(p.table), i32(context), mask=up(masks.view(np.int64)), workspace=w)
        got = got.cpu().numpy()
        assert np.isnan(got[:, 3]).all()
        keep = [0, 1, 2, 4, 5]
        assert np.array_equal(got[:, keep].view(np.uint16), clean[:, keep].view(np.uint16))


def test_attend_extreme_scores():
    """Scores in the thousands: the largest wins, nothing overflows; and keys of equal score
    share evenly."""
    rng = np.random.default_rng(81)
    p = Paged(rng, 1, 8, 16, 1, 64, "fp16")
    p.cache.k.mul_(60.0)
    attend_case(rng, p, [100], 3, 2, scale=4.0, q=(halves(rng, 1, 3, 2, 64) * np.float16(8)), tag="large scores")
    attend_case(rng, p, [100], 3, 2, q=np.zeros((1, 3, 2, 64), np.float16), tag="equal scores")
    attend_case(rng, p, [100], 3, 2, scale=0.0, tag="scale 0")
    attend_case(rng, p, [100], 3, 2, scale=-0.3, tag="negative scale")


@pytest.mark.parametrize("form", ["int8", "e4m3"])
@pytest.mark.parametrize("factor", [2.0 ** -40, 2.0 ** -24, 2.0 ** 8])
def test_attend_small_and_uneven_value_scales(form, factor):
    """Values far below and above one keep their relative precision, also where the scales of
    one sequence's tokens differ by orders of magnitude."""
    rng = np.random.default_rng(82)
    p = Paged(rng, 2, 20, 16, 2, 64, form)
    p.cache.v_scale.mul_(factor)
    p.cache.v_scale[::2].mul_(2.0 ** -6)
    p.cache.v_scale[3] = 0.0
    kv = p.cache
    q = halves(rng, 2, 2, 4, 64)
    got = nm.nm_tree_attention(up(q), kv, up(p.table), i32([300, 17]),
                               workspace=nm.tree_attention_workspace(up(q), kv, up(p.table)))
    torch.cuda.synchronize()
    k, v = p.values()
    for b, ctx in enumerate([300, 17]):
        kk, vv = p.rows(k, b, np.arange(ctx + 2)), p.rows(v, b, np.arange(ctx + 2))
        want, size = ref.attention_ref(q[b], kk, vv, ref.tree_seen(ctx, 2, None), 1 / 8)
        close(got[b], want, attend_bound(q[b], kk, vv, 1 / 8, want, size) + TINY, f"{form} {factor}")


def test_attend_slices_strides_and_alignment():
    rng = np.random.default_rng(83)
    p = Paged(rng, 2, 3, 16, 2, 128, "int8")
    fused = up(halves(rng, 2, 3, 12, 128))
    args = (p.cache, up(p.table), i32([40, 3]))
    a = nm.nm_tree_attention(fused[:, :, 2:10], *args)
    b = nm.nm_tree_attention(fused[:, :, 2:10].contiguous(), *args)
    assert torch.equal(a, b)
    out = torch.full_like(b, float("nan"))
    assert nm.nm_tree_attention(fused[:, :, 2:10], *args, out=out) is out and torch.equal(out, b)


def test_attend_bad_tables_stay_in_bounds():
    """Contexts past the table and entries out of range: any values, no fault, zeros stay zeros."""
    rng = np.random.default_rng(84)
    p = Paged(rng, 3, 4, 16, 2, 128, "e4m3")
    table = p.table.copy()
    table[0, 1], table[1, 0], table[2, 3] = -1, 2 ** 31 - 1, p.blocks
    q = up(halves(rng, 3, 5, 4, 128))
    ws = nm.tree_attention_workspace(q, p.cache, up(table))
    for w in (ws, None):
        out = nm.nm_tree_attention(q, p.cache, up(table), i32([2 ** 31 - 1, -9, 62]), count=i32([5, 0, 99]), workspace=w)
        torch.cuda.synchronize()
        assert not out[1].any()


def test_attend_is_deterministic_and_workspace_reusable():
    rng = np.random.default_rng(85)
    p = Paged(rng, 4, 40, 64, 4, 128, "int8")
    q = up(halves(rng, 4, 4, 16, 128))
    table, ctx = up(p.table), i32([2500, 100, 1999, 7])
    ws = nm.tree_attention_workspace(q, p.cache, table)
    first = nm.nm_tree_attention(q, p.cache, table, ctx, workspace=ws)
    for _ in range(20):
        small = nm.nm_tree_attention(q[:1, :1].contiguous(), p.cache, table[:1], ctx[:1], workspace=ws)
        assert torch.equal(nm.nm_tree_attention(q, p.cache, table, ctx, workspace=ws), first)
    assert small.shape == (1, 1, 16, 128)


# --------------------------------------------------------------------------------- verify
def probabilities(rng, *shape, spread=4.0):
    x = np.exp(rng.standard_normal(shape) * spread / 2)
    return (x / x.sum(-1, keepdims=True)).astype(np.float32)


def chain_case(rng, batch, nodes, vocab, spread=4.0):
    target = probabilities(rng, batch, nodes, vocab, spread=spread)
    draft = (target[:, :nodes - 1] * np.exp(rng.standard_normal((batch, nodes - 1, vocab)) * 0.5)).astype(np.float32)
    draft /= draft.sum(-1, keepdims=True)
    tokens = np.zeros((batch, nodes), np.int32)
    for b in range(batch):
        for i in range(1, nodes):
            tokens[b, i] = rng.choice(vocab, p=draft[b, i - 1].astype(np.float64) / draft[b, i - 1].astype(np.float64).sum())
    return target, draft, tokens, rng.random((batch, nodes)).astype(np.float32)


def check_chain(target, draft, tokens, uniforms, count=None, workspace=True):
    batch, nodes, vocab = target.shape
    ws = nm.verify_workspace(batch, vocab) if workspace else None
    acc, out = nm.nm_verify_chain(up(target), up(draft), i32(tokens), up(uniforms),
                                  None if count is None else i32(count), workspace=ws)
    acc, out = acc.cpu().numpy(), out.cpu().numpy()
    if ws is not None:
        assert not ws[:65536].any()
    for b in range(batch):
        n = nodes if count is None else min(max(int(count[b]), 0), nodes)
        m, want = ref.verify_chain_ref(target[b], draft[b], tokens[b], uniforms[b], n)
        assert acc[b] == m and np.array_equal(out[b], want), f"sequence {b}: {acc[b]} {out[b]} want {m} {want}"
    return acc


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("batch,nodes,vocab", [(1, 1, 1), (1, 2, 7), (5, 4, 100), (8, 5, 32000), (3, 9, 4097), (2, 64, 333),
                                                (70, 3, 1025), (1, 3, 151936)])
def test_verify_chain(batch, nodes, vocab, workspace):
    say(f"verify chain {batch}x{nodes}x{vocab}")
    rng = np.random.default_rng(batch * nodes + vocab)
    case = chain_case(rng, batch, nodes, vocab)
    check_chain(*case, workspace=workspace)
    check_chain(*case, count=rng.integers(-1, nodes + 2, batch), workspace=workspace)


def test_verify_chain_all_and_none_accepted():
    rng = np.random.default_rng(3)
    target, draft, tokens, u = chain_case(rng, 4, 6, 500)
    u[:, 1:] = 0.0
    assert np.all(check_chain(target, draft, tokens, u) == 5)
    u[:, 1:] = np.float32(1 - 2.0 ** -24)
    target[:, :, :] = 1e-9
    target[:, :, 7] = 1.0
    tokens[:, 1:] = 8
    assert np.all(check_chain(target, draft, tokens, u) == 0)


def test_verify_chain_ends_of_the_draw():
    """Uniforms of 0 and just below 1, weights at the row's two ends only, ties, an empty
    remainder (target equal to draft), rows of zeros, NaN and infinities, tokens out of range."""
    rng = np.random.default_rng(4)
    vocab = 3001
    target, draft, tokens, u = chain_case(rng, 8, 3, vocab)
    top = np.float32(1 - 2.0 ** -24)
    target[0, 0], draft[0, 0] = 0.0, 0.0
    target[0, 0, [0, -1]] = 0.5
    tokens[0, 1], u[0] = 5, (0.0, 0.5, 0.5)
    target[1, 0], draft[1, 0] = target[0, 0], 0.0
    tokens[1, 1], u[1] = 5, (top, 0.5, 0.5)
    target[2, 0], draft[2, 0] = 1.0 / vocab, 1.0 / vocab     # equal: nothing left, the target itself
    u[2] = (0.5, top, 0.0)
    tokens[2, 1] = -3                                          # out of range: refused
    target[3, 0] = 0.0                                         # no weight at all: -1
    tokens[3, 1] = 17
    target[4, 0], u[4, 1] = np.nan, 0.0
    target[4, 0, 40] = 0.25
    draft[4, 0] = 0.0
    target[5, 0, 3], target[5, 0, 9] = np.inf, -1.0
    tokens[5, 1] = vocab                                       # out of range
    draft[6, 0] = np.nan                                       # nothing comparable: refused, drawn from the target
    check_chain(target, draft, tokens, u)
    check_chain(target, draft, tokens, u, workspace=False)


def tree_case(rng, batch, nodes, vocab, spread=4.0):
    target = probabilities(rng, batch, nodes, vocab, spread=spread)
    parents = np.full((batch, nodes), -1, np.int32)
    tokens = np.zeros((batch, nodes), np.int32)
    for b in range(batch):
        for i in range(1, nodes):
            parents[b, i] = rng.integers(max(0, i - 6), i)
            likely = np.argsort(-target[b, parents[b, i]])[:4]
            tokens[b, i] = rng.choice(likely)                  # siblings repeat now and then
    return target, tokens, parents, rng.random((batch, nodes)).astype(np.float32)


def check_tree(target, tokens, parents, uniforms, count=None, workspace=True):
    batch, nodes, vocab = target.shape
    ws = nm.verify_workspace(batch, vocab) if workspace else None
    acc, out, path = nm.nm_verify_tree(up(target), i32(tokens), i32(parents), up(uniforms),
                                       None if count is None else i32(count), workspace=ws)
    acc, out, path = acc.cpu().numpy(), out.cpu().numpy(), path.cpu().numpy()
    for b in range(batch):
        n = nodes if count is None else min(max(int(count[b]), 0), nodes)
        m, want, walked = ref.verify_tree_ref(target[b], tokens[b], parents[b], uniforms[b], n)
        assert acc[b] == m and np.array_equal(out[b], want) and np.array_equal(path[b], walked), f"sequence {b}"
    return acc


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("batch,nodes,vocab", [(1, 1, 5), (4, 8, 50), (6, 64, 700), (3, 24, 32000), (40, 16, 1000),
                                                (2, 33, 4099)])
def test_verify_tree(batch, nodes, vocab, workspace):
    say(f"verify tree {batch}x{nodes}x{vocab}")
    rng = np.random.default_rng(batch + nodes * vocab)
    case = tree_case(rng, batch, nodes, vocab)
    check_tree(*case, workspace=workspace)
    check_tree(*case, count=rng.integers(-1, nodes + 2, batch), workspace=workspace)


def test_verify_tree_deep_paths_and_refusals():
    rng = np.random.default_rng(21)
    target, tokens, parents, u = tree_case(rng, 6, 32, 300)
    u[:3] = 0.0                                                # everything that can stands
    acc = check_tree(target, tokens, parents, u)
    assert np.all(acc[:3] >= 2)
    u[:] = np.float32(1 - 2.0 ** -24)
    check_tree(target, tokens, parents, u)
    target[:] = 0.0                                            # the refused tokens held all the mass
    target[:, :, 11] = 1.0
    tokens[:, 1:] = 12
    assert np.all(check_tree(target, tokens, parents, u) == 0)
    tokens[0, 1:], parents[0, 1:] = 11, 0
    u[0, 1:] = 1.0
    check_tree(target, tokens, parents, u)


def test_verify_tree_bad_parents_and_tokens():
    rng = np.random.default_rng(22)
    target, tokens, parents, u = tree_case(rng, 4, 20, 200)
    parents[0, 3], parents[0, 5], parents[1, 2], parents[2, 7] = 3, 90, -5, 2 ** 31 - 1
    tokens[1, 1], tokens[3, 2] = -1, 200
    target[2, 0, :50] = np.nan
    u[:, 1:] *= 0.2
    check_tree(target, tokens, parents, u)
    check_tree(target, tokens, parents, u, workspace=False)


# ------------------------------------------------------------------------ graphs, streams
def test_step_under_graph_capture():
    """The step's calls captured once and replayed over changing inputs, against eager calls."""
    rng = np.random.default_rng(90)
    p = Paged(rng, 2, 20, 16, 2, 128, "int8")
    table, turns = up(p.table), nm.rope_turns(128, device=device())
    fused = up(halves(rng, 2, 6, 12, 128))
    pos, ctx = i32(np.arange(12).reshape(2, 6) + 200), i32([200, 150])
    masks = up(tree_masks(rng, 2, 6).view(np.int64))
    target, tokens, parents, u = tree_case(rng, 2, 6, 3000)
    t, tk, pr, un = up(target), i32(tokens), i32(parents), up(u)
    ws = nm.tree_attention_workspace(fused[:, :, :8], p.cache, table)
    vs = nm.verify_workspace(2, 3000)
    out = torch.empty(2, 6, 8, 128, dtype=torch.float16, device=device())

    def step():
        q = nm.nm_rope_kv_append(p.cache, fused[:, :, :8], fused[:, :, 8:10], fused[:, :, 10:], pos, turns, table, ctx)
        nm.nm_tree_attention(q, p.cache, table, ctx, mask=masks, workspace=ws, out=out)
        acc, toks, path = nm.nm_verify_tree(t, tk, pr, un, workspace=vs)
        nm.nm_kv_compact(p.cache, table, ctx, path, acc)
        return (acc, toks, path, *nm.nm_kv_read(p.cache, table, ctx, 6))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        made = step()
    for i in range(4):
        fused.copy_(up(halves(rng, 2, 6, 12, 128)))
        un.copy_(up(rng.random((2, 6)).astype(np.float32)))
        ctx.copy_(i32([200 - 3 * i, 150 + i]))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (out, *made)]
        want_rest = step()
        torch.cuda.synchronize()
        for a, b in zip(got, (out, *want_rest)):
            assert torch.equal(a, b), f"replay {i}"


def test_calls_run_on_the_current_stream():
    rng = np.random.default_rng(91)
    p = Paged(rng, 2, 10, 16, 2, 64, "e4m3")
    q, table, ctx = up(halves(rng, 2, 3, 4, 64)), up(p.table), i32([100, 60])
    want = nm.nm_tree_attention(q, p.cache, table, ctx)
    s = torch.cuda.Stream()
    q2 = torch.zeros_like(q)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(10_000_000)
        q2.copy_(q)                                            # the call must come after this
        got = nm.nm_tree_attention(q2, p.cache, table, ctx)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


# ------------------------------------------------------------------------------ more ranges
@pytest.mark.parametrize("form", list(FORMATS))
def test_attend_uneven_batches(form):
    """One long sequence among short and empty ones, an odd number of key heads, and one key head
    alone over a long context (more chunks than a join takes): the chunks' search and caps."""
    rng = np.random.default_rng(86)
    context = [0, 9000] + rng.integers(0, 70, 40).tolist()
    p = Paged(rng, 42, -(-9004 // 64), 64, 3, 64, form)
    attend_case(rng, p, context, 2, 6, tag="one long")
    p = Paged(rng, 1, -(-40009 // 128), 128, 1, 128, form)
    attend_case(rng, p, [40000], 1, 1, tag="one head")
    attend_case(rng, p, [39990], 9, 16, tag="one head, 144 rows")


@pytest.mark.parametrize("form", ["int8", "fp16"])
def test_cache_beyond_four_gigabytes(form):
    """Offsets past 32 bits: the same tokens in the last blocks of a cache of more than 4 GiB a
    side and in the first blocks give the same bits."""
    rng = np.random.default_rng(87)
    kv, page, dim = 8, 64, 128
    blocks = 2 ** 32 // (kv * page * dim * (1 if form == "int8" else 2)) + 40
    c = nm.kv_cache(blocks, page, kv, dim, FORMATS[form], device=device())
    k, v = up(halves(rng, 2, 300, kv, dim)), up(halves(rng, 2, 300, kv, dim))
    q = up(halves(rng, 2, 4, 32, dim))
    results = []
    for first in (0, blocks - 12):
        table = i32(first + rng.permutation(12).reshape(2, 6))
        nm.nm_kv_append(c, k, v, table, i32([7, 0]))
        read = nm.nm_kv_read(c, table, i32([7, 0]), 300)
        out = nm.nm_tree_attention(q, c, table, i32([300, 296]), workspace=nm.tree_attention_workspace(q, c, table))
        results.append((*read, out[1:]))
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert results[0][0].float().abs().sum() > 0


def test_verify_with_a_small_workspace_runs_unsplit():
    rng = np.random.default_rng(88)
    target, draft, tokens, u = chain_case(rng, 3, 4, 20000)
    want = nm.nm_verify_chain(up(target), up(draft), i32(tokens), up(u))
    got = nm.nm_verify_chain(up(target), up(draft), i32(tokens), up(u),
                             workspace=torch.zeros(70000, dtype=torch.uint8, device=device()))
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_verify_rows_of_large_vocabularies_end_anywhere():
    """Thresholds in the first and last elements of every workgroup's run."""
    rng = np.random.default_rng(89)
    vocab = 50021
    target = np.zeros((64, 1, vocab), np.float32)
    at = np.unique(np.concatenate([[0, vocab - 1], rng.integers(0, vocab, 61), [1024]]))[:64]
    for b in range(64):
        target[b, 0, at[b % len(at)]] = 0.25 + b
    check_chain(target, np.zeros((64, 0, vocab), np.float32), np.zeros((64, 1), np.int32),
                rng.random((64, 1)).astype(np.float32))


@pytest.mark.parametrize("form", list(FORMATS))
def test_example_gives_the_same_text(form):
    """Decoding with draft trees gives the text of plain decoding, in fewer steps."""
    from examples import speculative_decode as ex
    plain, tree, steps = ex.main(["--tokens", "64", "--format", form])
    assert plain == tree
    assert steps < 64


class _Refuses:
    """Stands for the quick way and takes nothing, so that decode.py's own checks make the call."""

    def __getattr__(self, name):
        return lambda *args: NotImplemented


class _Counts:
    """The quick way, counting the calls that it took."""

    def __init__(self, inner):
        self.inner, self.took, self.left = inner, [], []

    def __getattr__(self, name):
        def call(*args):
            done = getattr(self.inner, name)(*args)
            (self.left if done is NotImplemented else self.took).append(name)
            return done
        return call


@pytest.mark.gpu
@pytest.mark.parametrize("form", [torch.float16, torch.int8, torch.float8_e4m3fn])
def test_both_ways_to_the_library(form, monkeypatch):
    from semi_structured_sparse_amd import decode

    def calls():
        g = torch.Generator().manual_seed(7)
        dev = torch.device("cuda")
        batch, nodes, heads, kv, dim, vocab = 2, 5, 4, 2, 64, 1001
        cache = nm.kv_cache(12, 16, kv, dim, dtype=form)
        table = torch.arange(12, dtype=torch.int32, device=dev).view(batch, 6).contiguous()
        start = torch.tensor([30, 7], dtype=torch.int32, device=dev)
        count = torch.tensor([5, 3], dtype=torch.int32, device=dev)
        fused = torch.randn(batch, nodes, (heads + 2 * kv) * dim, generator=g).half().to(dev)
        q = fused[..., : heads * dim].unflatten(-1, (heads, dim))
        k = fused[..., heads * dim: (heads + kv) * dim].unflatten(-1, (kv, dim))
        v = fused[..., (heads + kv) * dim:].unflatten(-1, (kv, dim))
        turns = nm.rope_turns(dim, device=dev)
        pos = start[:, None] + torch.arange(nodes, dtype=torch.int32, device=dev)
        made = [nm.nm_rope(q.reshape(-1, heads, dim), pos.reshape(-1).contiguous(), turns)]
        past = torch.randn(batch, 30, kv, dim, generator=g).half().to(dev)
        nm.nm_kv_append(cache, past, past, table, torch.zeros_like(start))
        turned = nm.nm_rope_kv_append(cache, q, k, v, pos, turns, table, start, count, layout="interleaved")
        assert nm.nm_rope_kv_append(cache, None, k, v, pos, turns, table, start, count, layout="interleaved") is None
        mask = torch.tensor([[1, 3, 5, 11, 21]] * batch, dtype=torch.int64, device=dev)
        work = nm.tree_attention_workspace(turned, cache, table)
        made += [turned, nm.nm_tree_attention(turned, cache, table, start, mask, count, workspace=work)]
        p = torch.rand(batch, nodes, vocab, generator=g).to(dev)
        p /= p.sum(-1, keepdim=True)
        tokens = torch.randint(0, vocab, (batch, nodes), generator=g).int().to(dev)
        u = torch.rand(batch, nodes, generator=g).to(dev)
        parents = torch.tensor([[-1, 0, 0, 1, 2]] * batch, dtype=torch.int32, device=dev)
        ws = nm.verify_workspace(batch, vocab)
        made += nm.nm_verify_chain(p, p[:, 1:].contiguous(), tokens, u, count, ws)
        made += nm.nm_verify_tree(p, tokens, parents, u, count, ws)
        path = torch.tensor([[0, 2, 4, -1, -1]] * batch, dtype=torch.int32, device=dev)
        nm.nm_kv_compact(cache, table, start, path, torch.tensor([2, 1], dtype=torch.int32, device=dev))
        made += nm.nm_kv_read(cache, table, torch.zeros_like(start), 40, start + 5)
        return made

    counts = _Counts(decode._bound())
    monkeypatch.setattr(decode, "_quick", counts)
    quick = calls()
    assert not counts.left and set(counts.took) == set(decode._QUICK)
    monkeypatch.setattr(decode, "_quick", _Refuses())
    for a, b in zip(quick, calls(), strict=True):
        assert a.dtype == b.dtype and a.shape == b.shape and a.stride() == b.stride()
        assert torch.equal(a, b)


@pytest.mark.parametrize("dim", [16, 2])
def test_rope_of_more_tokens_than_a_grid(dim):
    """2^23 tokens and more in wide rows take a second grid (the narrow form's limit is further
    off); tokens around the border and at both ends are checked."""
    tokens = 2 ** 23 + 5
    x = torch.arange(tokens * dim, dtype=torch.int32, device=device()).remainder_(1013).half().view(tokens, 1, dim)
    pos = torch.arange(tokens, dtype=torch.int32, device=device())
    turns = ref.rope_turns_ref(dim)
    got = nm.nm_rope(x, pos, up(turns))
    for at in (0, 2 ** 23 - 4, tokens - 4):
        part = slice(at, at + 4)
        want, size = ref.rope_ref(x[part].cpu().numpy(), pos[part].cpu().numpy(), turns)
        close(got[part], want, HALF * np.abs(want) + 2.0 ** -18 * size + TINY, f"from {at}")


@pytest.mark.parametrize("context", [0, 5, 700, 9000])
def test_attend_equal_values_are_exact(context):
    """In an fp16 cache the weights' sum is of the weights as they multiply v: where all v are
    3, so is the result, but for fp32 sums ((keys + 8) 2^-24 each) and the last rounding."""
    rng = np.random.default_rng(context)
    cache = nm.kv_cache(160, 64, 2, 128)
    cache.k.copy_(up(halves(rng, 160, 2, 64, 128)))
    cache.v.fill_(3.0)
    table = i32(np.arange(160)[None])
    q = up(halves(rng, 1, 3, 8, 128))
    for work in (None, nm.tree_attention_workspace(q, cache, table)):
        got = nm.nm_tree_attention(q, cache, table, i32([context]), workspace=work)
        want = np.full(got.shape, 3.0)
        close(got, want, 3.0 * (HALF + 2 * (context + 8) * 2.0 ** -24) + 0 * want, f"{context}")


@pytest.mark.parametrize("workspace", [True, False])
def test_verify_rows_with_nothing_left(workspace):
    """A wide vocabulary whose rest is empty (drawn from the target after all), with infinities
    and NaN in some runs of the row, and with refused tokens in the first and the last."""
    rng = np.random.default_rng(91)
    vocab = 150001
    target, draft, tokens, u = chain_case(rng, 4, 2, vocab)
    draft[0, 0] = target[0, 0]                       # equal, refused by its token
    tokens[:, 1] = -1
    draft[1, 0] = 1.0                                # more than the target has anywhere
    target[2, 0, [5, 70000, 149999]] = np.inf, np.nan, -np.inf
    draft[2, 0, [6, 70001]] = -np.inf, np.nan
    target[3, 0], draft[3, 0] = 0.0, 0.0
    check_chain(target, draft, tokens, u, workspace=workspace)
    target, tokens, parents, u = tree_case(rng, 3, 5, vocab)
    parents[:, 1:] = 0
    target[0, 0] = 0.0                               # the first child's token holds it all, and is refused
    target[0, 0, vocab - 1] = 0.25
    tokens[:, 1:] = np.array([vocab - 1, 0, 1, 2])
    u[0, 1:] = 0.5
    target[1, 0, [3, 149998]] = np.inf
    u[1:, 1:] = 0.999
    check_tree(target, tokens, parents, u, workspace=workspace)
