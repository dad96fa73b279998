"""GPU tests of the attention where its range ends: tables, weights, scales, sums and workspaces.
Bounds are those of tests/attend_bounds.py, derived there."""
import numpy as np
import pytest
import torch

import semi_structured_sparse_amd as nm
from oracle import decode_oracle as ref
from tests.attend_bounds import HALF, TINY, attend_exact, markers
from tests.gpu_helpers import device, say
from tests.test_gpu_decode import FORMATS, Paged, close, halves, i32, tree_masks, up

pytestmark = pytest.mark.gpu
LARGEST = {"int8": 127.0, "e4m3": 448.0}


def cache_of(k, v, form, page=16, k_scale=None, v_scale=None):
    """A cache of one sequence whose tokens are k, v [keys, kv, dim] (codes where a scale [keys, kv]
    is given), in consecutive pages; its table."""
    keys, kv, dim = k.shape
    pages = -(-keys // page)

    def paged(x, dtype):
        full = np.zeros((pages * page,) + x.shape[1:], np.float32)
        full[:keys] = x
        full = full.reshape((pages, page) + x.shape[1:])
        return torch.from_numpy(np.ascontiguousarray(full.swapaxes(1, 2))).to(dtype).to(device())

    scales = [None if s is None else paged(s, torch.float32) for s in (k_scale, v_scale)]
    return nm.KVCache(paged(k, FORMATS[form]), paged(v, FORMATS[form]), *scales), i32(np.arange(pages)[None])


def attend(q, cache, table, context, workspace, **kw):
    ws = nm.tree_attention_workspace(q, cache, table) if workspace else None
    out = nm.nm_tree_attention(q, cache, table, i32(context), workspace=ws, **kw)
    torch.cuda.synchronize()
    return out.cpu().numpy().astype(np.float64)


# --------------------------------------------------------------------- the end of the page table
@pytest.mark.parametrize("form", list(FORMATS))
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("width", [1, 2, 3, 4, 129])
def test_nodes_past_the_page_table_are_not_there(form, masked, width):
    """context + count is clamped to the table's positions, which end inside a tile of 32 where
    pages of 16 are odd in number: nodes past them see what fits, and are seen by none."""
    say(f"table end {form} {width} {masked}")
    rng = np.random.default_rng(width)
    tokens, cap = 5, 16 * width
    context = [cap - 3, cap, cap + 7, cap - 5, 2 ** 31 - 1]
    p = Paged(rng, len(context), width, 16, 2, 128, form)
    masks = tree_masks(rng, len(context), tokens) if masked else None
    q = halves(rng, len(context), tokens, 4, 128)
    counts = [5, 5, 5, 4, 5]
    k, v = p.values()
    for workspace in (True, False):
        got = attend(up(q), p.cache, up(p.table), context, workspace, count=i32(counts),
                     mask=None if masks is None else up(masks.view(np.int64)))
        for b in range(len(context)):
            held = min(context[b], cap)
            keys = min(held + counts[b], cap)
            seen = ref.tree_seen(held, counts[b], None if masks is None else masks[b])[:, :keys]
            at = np.arange(keys)
            z = None
            if form != "fp16":
                z = p.cache.v_scale.cpu().numpy()[p.table[b, at // 16], :, at % 16]
            bias = 0.0
            if form == "int8":
                bias = 128.0 * p.cache.k_scale.cpu().numpy()[p.table[b, at // 16], :, at % 16].astype(np.float64)
            want, bound = attend_exact(q[b, :counts[b]], p.rows(k, b, at), p.rows(v, b, at), seen, 128 ** -0.5, z, bias)
            close(got[b, :counts[b]], want, bound, f"width {width} sequence {b}")
            assert np.all(got[b, counts[b]:] == 0)


@pytest.mark.parametrize("form", list(FORMATS))
def test_a_context_below_zero_shortens_the_nodes(form):
    """context and context + count are both clamped to 0: of 5 nodes from -3 on, positions 0 and 1."""
    rng = np.random.default_rng(7)
    p = Paged(rng, 3, 2, 16, 2, 64, form)
    q = up(halves(rng, 3, 5, 4, 64))
    got = attend(q, p.cache, up(p.table), [-3, -5, -2 ** 31], False)
    want = attend(q, p.cache, up(p.table), [0, 0, 0], False, mask=up(np.tile(np.array([1, 3, 3, 3, 3]), (3, 1))))
    assert np.array_equal(got[0], want[0]) and not got[1:].any()


# ------------------------------------------------------------------------------- small weights
@pytest.mark.parametrize("form", list(FORMATS))
@pytest.mark.parametrize("bits", [14.5, 18.5, 20.5, 22.5, 23.5])
def test_long_tails_below_a_dominant_key_keep_their_share(form, bits):
    """Four keys, one for each wave, lead and hold nothing; all that is left of the result is the
    tail, 2^-bits of them each."""
    say(f"tail {form} {bits}")
    rng = np.random.default_rng(int(2 * bits))
    keys, kv, dim = 4096, 1, 64
    k, v = np.zeros((keys, kv, dim)), np.zeros((keys, kv, dim))
    k[0:128:32, 0, 0] = 64.0
    v[:, 0] = rng.integers(64, 128, (keys, dim)) if form != "e4m3" else rng.choice([64.0, 80.0, 96.0, 112.0], (keys, dim))
    v[0:128:32] = 0.0
    q = np.zeros((1, 1, 1, dim), np.float16)
    q[..., 0] = 1.0
    ks = vs = None
    if form != "fp16":
        ks, vs = np.full((keys, kv), 1 / 64, np.float32), np.full((keys, kv), 8.0 if form == "int8" else 2.0, np.float32)
    cache, table = cache_of(k, v, form, 64, ks, vs)
    scale = bits * np.log(2.0) / (64.0 if form == "fp16" else 1.0)
    values = v * (1.0 if vs is None else vs[..., None].astype(np.float64))
    keyed = k * (1.0 if ks is None else ks[..., None].astype(np.float64))
    want, bound = attend_exact(q[0], keyed, values, np.ones((1, keys), bool), np.float64(np.float32(scale)), vs,
                               0.0 if form != "int8" else 128.0 * ks)
    assert np.abs(want).min() > 2.0 ** -14
    for workspace in (False, True):
        got = attend(up(q), cache, table, [keys - 1], workspace, scale=scale)
        close(got[0], want, bound, f"{form} {bits} bits, workspace {workspace}")


@pytest.mark.parametrize("form", ["int8", "e4m3"])
@pytest.mark.parametrize("bits", [18.5, 24.5])
def test_rows_of_zeros_keep_their_weight_in_the_sum(form, bits):
    """One key of large values over a long tail whose values are zeros (scale 0): they shrink the
    result by their share, whatever lies between the scales."""
    keys, kv, dim = 65536, 1, 64
    k, v = np.zeros((keys, kv, dim)), np.zeros((keys, kv, dim))
    k[5, 0, 0], v[5, 0] = 1.0, np.arange(64, 128) // 8 * 8
    q = np.zeros((1, 1, 1, dim), np.float16)
    q[..., 0] = 1.0
    ks, vs = np.ones((keys, kv), np.float32), np.zeros((keys, kv), np.float32)
    vs[5] = 512.0 if form == "int8" else 128.0
    cache, table = cache_of(k, v, form, 128, ks, vs)
    scale = float(np.float32(bits * np.log(2.0)))
    share = 1.0 / (1.0 + (keys - 1) * np.exp(-scale))
    want = v[5] * np.float64(vs[5, 0]) * share
    # the exponentials 2^-20 together, the sum in fp32 over 65536 keys, both weights' rounding
    bound = np.abs(want) * (2 * HALF + 2.0 ** -19 + keys * 2.0 ** -24 * (1.0 - share)) + HALF * np.abs(want)
    for workspace in (False, True):
        got = attend(up(q), cache, table, [keys - 1], workspace, scale=scale)
        close(got[0, 0], want, bound, f"{form} workspace {workspace}")


# ---------------------------------------------------------------------------------- odd values
def test_codes_that_are_not_numbers_stay_with_the_nodes_that_see_them():
    """e4m3 codes of NaN in a draft's value row, whose scale is a number: the nodes that see the
    draft get NaN, the others what they had."""
    rng = np.random.default_rng(80)
    context, tokens = [37, 0, 20, 95], 6
    p = Paged(rng, 4, 8, 16, 2, 128, "e4m3")
    masks = np.tile(np.array([1, 3, 5, 9, 17, 33], np.uint64), (4, 1))
    args = (up(halves(rng, 4, tokens, 4, 128)), p.cache, up(p.table), context)
    mask = up(masks.view(np.int64))
    clean = attend(*args, False, mask=mask)
    for b in range(4):
        j = context[b] + 3
        p.cache.v.view(torch.uint8)[p.table[b, j // 16], :, j % 16, 5 + b] = 0x7F if b % 2 else 0xFF
    got = attend(*args, False, mask=mask)
    keep = [0, 1, 2, 4, 5]
    assert np.array_equal(got[:, keep], clean[:, keep])
    assert np.isnan(got[:, 3]).all()


# ---------------------------------------------------------------------------------- long sums
@pytest.mark.parametrize("form", list(FORMATS))
@pytest.mark.parametrize("workspace", [False, True])
def test_long_sums_of_values_that_cancel(form, workspace):
    """131072 keys whose weights are fp16 numbers (scores log2 of 1 + r/1024, so that the rounding to
    fp16 takes the exponential's error off) and whose weighted values, multiples of 2^-6, nearly
    cancel in pairs: every partial sum of a wave stays below 2^18, exact in fp32. What is left are
    the sum of the weights (8192 positive terms a lane, 2^-24 of the sum so far each, which is half
    of the whole on average: 2^-12; 2^-20 for exponentials and joins) and the last rounding."""
    say(f"cancel {form} {workspace}")
    rng = np.random.default_rng(5)
    keys, kv, dim = 131072, 1, 64
    w = 1.0 + rng.integers(0, 1024, keys) / 1024.0
    w[::32] = 2.0                                # the largest comes first in every tile
    if form == "fp16":                           # the score is the key's own: held equal
        w[:] = 2.0
    k = np.zeros((keys, kv, dim))
    k[:, 0, 0] = 1.0
    codes = rng.integers(1, 8, (keys // 2, 1, dim)) * 16.0 * rng.choice([-1.0, 1.0], (keys // 2, 1, dim))
    v = np.repeat(codes, 2, 0)
    v[1::2] *= -1.0
    ks = vs = None
    if form == "fp16":
        v[::2] += 0.5                            # what is left of each pair
    else:
        ks, vs = np.log2(w)[:, None].astype(np.float32), np.ones((keys, kv), np.float32)
    parts = (w[:, None] * v[:, 0]).reshape(-1, 4, 32, dim)
    assert np.abs(np.cumsum(parts.sum(2), 0)).max() + np.abs(parts).sum(2).max() < 2 ** 18
    want = (parts.sum((0, 1, 2)) / w.sum())[None, None]
    q = np.zeros((1, 1, 1, dim), np.float16)
    q[..., 0] = 1.0
    cache, table = cache_of(k, v, form, 128, ks, vs)
    got = attend(up(q), cache, table, [keys - 1], workspace, scale=np.log(2.0))
    close(got[0], want, np.abs(want) * (HALF + 2.0 ** -12 + 2.0 ** -20) + TINY, f"{form} {workspace}")


@pytest.mark.parametrize("form", list(FORMATS))
@pytest.mark.parametrize("keys,rows", [(20011, 1), (40001, 9), (131071, 16)])
def test_every_tile_counts_once(form, keys, rows):
    """Values that mark their tile: a tile of 32 keys left out, or taken twice, moves a result by one
    over the number of tiles that share its dim, 10% where the bound is 0.4% at most."""
    say(f"markers {form} {keys} {rows}")
    rng = np.random.default_rng(keys)
    kv, dim = 1, 128 if keys < 100000 else 256
    k = rng.standard_normal((keys, kv, dim)).astype(np.float16).astype(np.float64)
    v, ks, vs = markers(keys, kv, dim), None, None
    if form != "fp16":
        ks, vs = np.full((keys, kv), 2.0 ** -6, np.float32), np.full((keys, kv), 1 / 64, np.float32)
        k, v = np.round(k * 16) * 4 % 64, v * 64.0     # whole numbers that e4m3 holds: multiples of 4 below 64
    q = (halves(rng, 1, 1, rows, dim) * np.float16(0.125)).astype(np.float16)
    values = v * (1.0 if vs is None else vs[..., None].astype(np.float64))
    keyed = k * (1.0 if ks is None else ks[..., None].astype(np.float64))
    want, bound = attend_exact(q[0], keyed, values, np.ones((1, keys), bool), dim ** -0.5, vs,
                               0.0 if form != "int8" else 128.0 * ks)
    cache, table = cache_of(k, v, form, 64, ks, vs)
    for workspace in (False, True):
        got = attend(up(q), cache, table, [keys - 1], workspace)
        close(got[0], want, bound, f"{form} {keys} workspace {workspace}")


@pytest.mark.parametrize("form", ["int8", "e4m3"])
@pytest.mark.parametrize("factor", [2.0 ** -5, 1.0, 2.0 ** 6])
def test_small_and_uneven_value_scales_keep_their_bits(form, factor):
    """Results that fp16 holds in full, of values whose scales differ by 2^6 from page to page."""
    rng = np.random.default_rng(82)
    p = Paged(rng, 2, 20, 16, 2, 64, form)
    p.cache.v.view(torch.uint8).bitwise_and_(0x7F)             # positive: nothing cancels
    p.cache.v_scale.mul_(factor)
    p.cache.v_scale[::2].mul_(2.0 ** -6)
    p.cache.v_scale[3] = 0.0
    q = halves(rng, 2, 2, 4, 64)
    context = [300, 17]
    k, v = p.values()
    for workspace in (True, False):
        got = attend(up(q), p.cache, up(p.table), context, workspace)
        for b, ctx in enumerate(context):
            at = np.arange(ctx + 2)
            pick = (p.table[b, at // 16], slice(None), at % 16)
            z, ks = p.cache.v_scale.cpu().numpy()[pick], p.cache.k_scale.cpu().numpy()[pick]
            want, bound = attend_exact(q[b], p.rows(k, b, at), p.rows(v, b, at), ref.tree_seen(ctx, 2, None), 1 / 8, z,
                                       0.0 if form != "int8" else 128.0 * ks.astype(np.float64))
            assert np.abs(want).min() > 2.0 ** -14
            close(got[b], want, bound, f"{form} {factor} sequence {b}")


# --------------------------------------------------------------------------------- workspaces
def steps(rng, kv, heads, dim, form, width, page=64, batch=1):
    cache = nm.kv_cache(batch * width, page, kv, dim, FORMATS[form], device=device())
    rows = up(halves(rng, batch, page * width, kv, dim))
    table = i32(np.arange(batch * width).reshape(batch, width))
    nm.nm_kv_append(cache, rows, rows.flip(1).contiguous(), table, i32([0] * batch))
    return cache, table


@pytest.mark.parametrize("form", list(FORMATS))
@pytest.mark.parametrize("heads,kv,dim", [(64, 8, 128), (32, 8, 64), (16, 1, 256), (5, 5, 128)])
def test_a_workspace_serves_every_smaller_step(form, heads, kv, dim):
    """What a step of 64 nodes over the widest table asks for is enough for steps of fewer nodes,
    sequences or pages."""
    wide = nm.kv_cache(4, 64, kv, dim, FORMATS[form], device=device())

    def need(tokens, width, batch):
        q = torch.empty(batch, tokens, heads, dim, dtype=torch.float16, device=device())
        ws = nm.tree_attention_workspace(q, wide, torch.zeros(batch, width, dtype=torch.int32, device=device()))
        return 0 if ws is None else ws.numel()

    for batch, width in ((1, 256), (3, 64), (8, 2048)):
        most = 0
        for tokens in range(1, 65):
            now = need(tokens, width, batch)
            assert now >= most, f"{tokens} nodes need {now}, fewer {most}"
            most = now
        assert need(64, width // 2, batch) <= most and need(64, width, max(1, batch // 2)) <= most


@pytest.mark.parametrize("form", list(FORMATS))
@pytest.mark.parametrize("share", [0.9, 0.5, 0.2, 0.02])
def test_a_small_workspace_splits_as_far_as_it_goes(form, share):
    """Less than the query's bytes split over fewer workgroups, with the result of the whole to the
    order of its sums; the partial results stay within what was given."""
    rng = np.random.default_rng(4)
    heads, kv, dim, width = 64, 8, 128, 128
    cache, table = steps(rng, kv, heads, dim, form, width)
    q = up(halves(rng, 1, 6, heads, dim))
    full = nm.tree_attention_workspace(q, cache, table)
    want = nm.nm_tree_attention(q, cache, table, i32([8000]), workspace=full)
    room = 65536 + int((full.numel() - 65536) * share) // 16 * 16
    guarded = torch.full((full.numel() + 4096,), 0xA5, dtype=torch.uint8, device=device())
    guarded[:65536] = 0
    small = guarded[:room]
    got = nm.nm_tree_attention(q, cache, table, i32([8000]), workspace=small)
    torch.cuda.synchronize()
    assert not guarded[:65536].any() and bool((guarded[room:] == 0xA5).all())
    assert bool((small[65536:] != 0xA5).any()) == (share > 0.1)
    alone = nm.nm_tree_attention(q, cache, table, i32([8000]))
    # both within the roundings of the definition: twice the weights' and the result's half steps,
    # where values of about one in magnitude cancel
    worst = 4 * HALF * cache_size(cache)
    for other in (got, alone):
        assert (other.float() - want.float()).abs().max().item() <= worst


def cache_size(cache):
    top = cache.v.float().abs().amax((1, 2, 3)) if cache.v_scale is None else \
        (cache.v.float().abs().amax(-1) * cache.v_scale).amax((1, 2))
    return float(top.max())


def test_a_verification_workspace_serves_fewer_sequences():
    def need(batch):
        ws = nm.verify_workspace(batch, 32000)
        return 0 if ws is None else ws.numel()

    sizes = [need(b) for b in (1, 7, 64, 500, 512, 513, 4000)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    assert nm.verify_workspace(4, 100) is None


def test_a_step_takes_the_workspace_of_a_larger_one():
    """6 nodes with the workspace of 8 and of 64: the same bits as with their own."""
    rng = np.random.default_rng(6)
    cache, table = steps(rng, 8, 64, 128, "int8", 256)
    q = up(halves(rng, 1, 64, 64, 128))
    few = q[:, :6].contiguous()
    want = nm.nm_tree_attention(few, cache, table, i32([16000]), workspace=nm.tree_attention_workspace(few, cache, table))
    for nodes in (8, 64):
        ws = nm.tree_attention_workspace(q[:, :nodes].contiguous(), cache, table)
        assert torch.equal(nm.nm_tree_attention(few, cache, table, i32([16000]), workspace=ws), want)


def test_the_example_makes_its_workspaces_for_its_trees():
    """What the example hands to the calls is what its largest step asks for."""
    from examples import speculative_decode as ex
    nodes = 12
    model = ex.Model(nodes, "int8")
    q = torch.empty(1, nodes, model.heads, model.dim, dtype=torch.float16, device=device())
    need = nm.tree_attention_workspace(q, model.caches[0], model.table)
    text, _ = ex.generate(model, [1, 5, 9, 1, 5], 8, nodes)
    assert len(text) == 13 and model.workspace.numel() >= need.numel()
    few = nm.verify_workspace(1, model.vocab)
    assert few is None or model.verify_workspace.numel() >= few.numel()
