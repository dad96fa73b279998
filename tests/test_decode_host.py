"""CPU tests of the speculative-decoding operators: refusals (no HIP call is made before the
arguments pass), the host table of rotary frequencies, the binding's checks, and the oracle
against closed forms."""
import ctypes
import math

import numpy as np
import pytest
import torch

import semi_structured_sparse_amd as nm
from oracle import decode_oracle as ref
from semi_structured_sparse_amd import decode

A = 0x10000   # an aligned fake device address: checks never dereference it


def _cache(**kw):
    c = decode._CacheStruct()
    given = dict(k=A, v=A, k_scale=A, v_scale=A, blocks=8, kv_heads=2, page=16, head_dim=128, format=1)
    given.update(kw)
    for name, v in given.items():
        setattr(c, name, v)
    return c


def _call(name, defaults, kw):
    a = dict(defaults)
    cache = {k[6:]: v for k, v in kw.items() if k.startswith("cache_")}
    a.update({k: v for k, v in kw.items() if not k.startswith("cache_")})
    if "cache" in a and a["cache"] is not None:
        a["cache"] = _cache(**cache)
    return getattr(nm.lib(), name)(*a.values())


PAGES = [
    (dict(cache=None), nm.NM_ERR_NULL), (dict(cache_k=None), nm.NM_ERR_NULL), (dict(cache_v=None), nm.NM_ERR_NULL),
    (dict(table=None), nm.NM_ERR_NULL), (dict(cache_k_scale=None), nm.NM_ERR_NULL),
    (dict(cache_v_scale=None), nm.NM_ERR_NULL),
    (dict(cache_format=3), nm.NM_ERR_FORMAT), (dict(cache_format=-1), nm.NM_ERR_FORMAT),
    (dict(cache_head_dim=96), nm.NM_ERR_FORMAT), (dict(cache_head_dim=0), nm.NM_ERR_FORMAT),
    (dict(cache_page=8), nm.NM_ERR_FORMAT), (dict(cache_page=48), nm.NM_ERR_FORMAT),
    (dict(cache_page=2048), nm.NM_ERR_FORMAT), (dict(cache_page=-16), nm.NM_ERR_FORMAT),
    (dict(cache_blocks=0), nm.NM_ERR_SHAPE), (dict(cache_blocks=1 << 31), nm.NM_ERR_SHAPE),
    (dict(cache_kv_heads=0), nm.NM_ERR_SHAPE), (dict(table_width=0), nm.NM_ERR_SHAPE),
    (dict(table_width=1 << 27), nm.NM_ERR_SHAPE), (dict(batch=0), nm.NM_ERR_SHAPE), (dict(batch=1 << 17), nm.NM_ERR_SHAPE),
    (dict(cache_k=A + 8), nm.NM_ERR_ALIGN), (dict(cache_v=A + 2), nm.NM_ERR_ALIGN), (dict(table=A + 2), nm.NM_ERR_ALIGN),
    (dict(cache_k_scale=A + 4), nm.NM_ERR_ALIGN), (dict(cache_v_scale=A + 8), nm.NM_ERR_ALIGN),
]

ROPE = dict(x=A, y=A, positions=A, turns=A, tokens=4, heads=3, head_dim=128, rot_dim=64, layout=0, scale=1.0,
            x_stride=384, y_stride=384, stream=None)
APPEND = dict(cache=True, k=A, v=A, k_stride=256, v_stride=256, table=A, table_width=4, start=A, count=A, batch=2,
              tokens=3, stream=None)
ROPE_APPEND = dict(cache=True, q=A, q_out=A, q_heads=4, q_stride=512, q_out_stride=512, k=A, v=A, k_stride=256,
                   v_stride=256, positions=A, turns=A, rot_dim=128, layout=1, scale=1.0, table=A, table_width=4,
                   start=A, count=A, batch=2, tokens=3, stream=None)
READ = dict(cache=True, k_out=A, v_out=A, table=A, table_width=4, start=A, count=A, batch=2, tokens=3, stream=None)
COMPACT = dict(cache=True, table=A, table_width=4, start=A, path=A, accepted=A, batch=2, nodes=5, stream=None)
ATTEND = dict(cache=True, q=A, out=A, heads=8, q_stride=1024, table=A, table_width=4, context=A, mask=A, count=A,
              batch=2, tokens=3, scale=0.1, workspace=None, workspace_bytes=0, stream=None)
CHAIN = dict(target=A, draft=A, tokens=A, uniforms=A, count=A, accepted=A, out_tokens=A, batch=2, nodes=4, vocab=100,
             workspace=None, workspace_bytes=0, stream=None)
TREE = dict(target=A, tokens=A, parents=A, uniforms=A, count=A, accepted=A, out_tokens=A, path=A, batch=2, nodes=4,
            vocab=100, workspace=None, workspace_bytes=0, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), nm.NM_ERR_NULL), (dict(y=None), nm.NM_ERR_NULL), (dict(positions=None), nm.NM_ERR_NULL),
    (dict(turns=None), nm.NM_ERR_NULL), (dict(tokens=0), nm.NM_ERR_SHAPE), (dict(tokens=(1 << 30) + 1), nm.NM_ERR_SHAPE),
    (dict(heads=0), nm.NM_ERR_SHAPE), (dict(heads=65537), nm.NM_ERR_SHAPE), (dict(head_dim=1), nm.NM_ERR_SHAPE),
    (dict(head_dim=1025), nm.NM_ERR_SHAPE), (dict(rot_dim=0), nm.NM_ERR_SHAPE), (dict(rot_dim=63), nm.NM_ERR_SHAPE),
    (dict(rot_dim=130), nm.NM_ERR_SHAPE), (dict(layout=2), nm.NM_ERR_FORMAT), (dict(layout=-1), nm.NM_ERR_FORMAT),
    (dict(x_stride=383), nm.NM_ERR_SHAPE), (dict(y_stride=383), nm.NM_ERR_SHAPE), (dict(x_stride=1 << 41), nm.NM_ERR_SHAPE),
    (dict(x=A + 1), nm.NM_ERR_ALIGN), (dict(y=A + 1), nm.NM_ERR_ALIGN), (dict(positions=A + 2), nm.NM_ERR_ALIGN),
    (dict(turns=A + 4), nm.NM_ERR_ALIGN),
])
def test_rope_refusals(kw, want):
    assert _call("nm_rope", ROPE, kw) == want


@pytest.mark.parametrize("kw,want", PAGES + [
    (dict(k=None), nm.NM_ERR_NULL), (dict(v=None), nm.NM_ERR_NULL), (dict(start=None), nm.NM_ERR_NULL),
    (dict(tokens=0), nm.NM_ERR_SHAPE), (dict(tokens=(1 << 24) + 1), nm.NM_ERR_SHAPE),
    (dict(batch=65536, tokens=1 << 24), nm.NM_ERR_SHAPE),
    (dict(k_stride=255), nm.NM_ERR_SHAPE), (dict(v_stride=248), nm.NM_ERR_SHAPE), (dict(k_stride=260), nm.NM_ERR_ALIGN),
    (dict(v_stride=257), nm.NM_ERR_ALIGN), (dict(k=A + 8), nm.NM_ERR_ALIGN), (dict(v=A + 2), nm.NM_ERR_ALIGN),
    (dict(start=A + 1), nm.NM_ERR_ALIGN), (dict(count=A + 2), nm.NM_ERR_ALIGN),
])
def test_append_refusals(kw, want):
    assert _call("nm_kv_append", APPEND, kw) == want


@pytest.mark.parametrize("kw,want", PAGES + [
    (dict(q=None), nm.NM_ERR_NULL), (dict(q_out=None), nm.NM_ERR_NULL), (dict(k=None), nm.NM_ERR_NULL),
    (dict(positions=None), nm.NM_ERR_NULL), (dict(turns=None), nm.NM_ERR_NULL),
    (dict(q_heads=-1), nm.NM_ERR_SHAPE), (dict(q_stride=511), nm.NM_ERR_SHAPE), (dict(q_out_stride=504), nm.NM_ERR_SHAPE),
    (dict(rot_dim=24), nm.NM_ERR_SHAPE), (dict(rot_dim=144), nm.NM_ERR_SHAPE), (dict(layout=5), nm.NM_ERR_FORMAT),
    (dict(q=A + 8), nm.NM_ERR_ALIGN), (dict(q_out_stride=516), nm.NM_ERR_ALIGN), (dict(turns=A + 4), nm.NM_ERR_ALIGN),
])
def test_rope_append_refusals(kw, want):
    assert _call("nm_rope_kv_append", ROPE_APPEND, kw) == want


@pytest.mark.parametrize("kw,want", PAGES + [
    (dict(k_out=None), nm.NM_ERR_NULL), (dict(v_out=None), nm.NM_ERR_NULL), (dict(start=None), nm.NM_ERR_NULL),
    (dict(tokens=0), nm.NM_ERR_SHAPE), (dict(k_out=A + 8), nm.NM_ERR_ALIGN), (dict(count=A + 1), nm.NM_ERR_ALIGN),
])
def test_read_refusals(kw, want):
    assert _call("nm_kv_read", READ, kw) == want


@pytest.mark.parametrize("kw,want", PAGES + [
    (dict(start=None), nm.NM_ERR_NULL), (dict(path=None), nm.NM_ERR_NULL), (dict(accepted=None), nm.NM_ERR_NULL),
    (dict(nodes=0), nm.NM_ERR_SHAPE), (dict(nodes=65), nm.NM_ERR_SHAPE), (dict(path=A + 2), nm.NM_ERR_ALIGN),
])
def test_compact_refusals(kw, want):
    assert _call("nm_kv_compact", COMPACT, kw) == want


@pytest.mark.parametrize("kw,want", PAGES + [
    (dict(q=None), nm.NM_ERR_NULL), (dict(out=None), nm.NM_ERR_NULL), (dict(context=None), nm.NM_ERR_NULL),
    (dict(tokens=0), nm.NM_ERR_SHAPE), (dict(tokens=65), nm.NM_ERR_SHAPE), (dict(heads=0), nm.NM_ERR_SHAPE),
    (dict(heads=7), nm.NM_ERR_SHAPE), (dict(heads=34, q_stride=34 * 128), nm.NM_ERR_SHAPE),
    (dict(q_stride=1016), nm.NM_ERR_SHAPE), (dict(scale=math.inf), nm.NM_ERR_SHAPE), (dict(scale=math.nan), nm.NM_ERR_SHAPE),
    (dict(q=A + 8), nm.NM_ERR_ALIGN), (dict(q_stride=1028), nm.NM_ERR_ALIGN), (dict(out=A + 4), nm.NM_ERR_ALIGN),
    (dict(mask=A + 4), nm.NM_ERR_ALIGN), (dict(context=A + 2), nm.NM_ERR_ALIGN), (dict(workspace=A + 8), nm.NM_ERR_ALIGN),
])
def test_attention_refusals(kw, want):
    assert _call("nm_tree_attention", ATTEND, kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(target=None), nm.NM_ERR_NULL), (dict(draft=None), nm.NM_ERR_NULL), (dict(tokens=None), nm.NM_ERR_NULL),
    (dict(uniforms=None), nm.NM_ERR_NULL), (dict(accepted=None), nm.NM_ERR_NULL), (dict(out_tokens=None), nm.NM_ERR_NULL),
    (dict(batch=0), nm.NM_ERR_SHAPE), (dict(nodes=0), nm.NM_ERR_SHAPE), (dict(nodes=65), nm.NM_ERR_SHAPE),
    (dict(vocab=0), nm.NM_ERR_SHAPE), (dict(vocab=(1 << 24) + 1), nm.NM_ERR_SHAPE), (dict(target=A + 2), nm.NM_ERR_ALIGN),
    (dict(count=A + 1), nm.NM_ERR_ALIGN), (dict(workspace=A + 4), nm.NM_ERR_ALIGN),
])
def test_verify_refusals(kw, want):
    assert _call("nm_verify_chain", CHAIN, kw) == want
    if "draft" not in kw:
        assert _call("nm_verify_tree", TREE, kw) == want


def test_verify_tree_needs_its_arrays():
    assert _call("nm_verify_tree", TREE, dict(parents=None)) == nm.NM_ERR_NULL
    assert _call("nm_verify_tree", TREE, dict(path=None)) == nm.NM_ERR_NULL


def test_workspace_queries_refuse_quietly():
    """Bad arguments, or no device, give 0 and no error."""
    lib = nm.lib()
    assert lib.nm_tree_attention_workspace_bytes(_cache(head_dim=80), 8, 4, 2, 3) == 0
    assert lib.nm_tree_attention_workspace_bytes(_cache(), 7, 4, 2, 3) == 0
    assert lib.nm_verify_workspace_bytes(0, 100) == 0
    assert lib.nm_verify_workspace_bytes(1, -5) == 0


def test_format_status():
    assert nm.NM_ERR_FORMAT == 8
    assert "format" in nm.status_string(nm.NM_ERR_FORMAT)


# --------------------------------------------------------------------- rotary frequencies
# The table and the oracle round each power, quotient and product in 64 bits a few times:
# relative 2^-48 holds with room.
@pytest.mark.parametrize("rot", [2, 4, 20, 64, 128, 1024])
@pytest.mark.parametrize("kw", [dict(), dict(base=500000.0), dict(scaling="linear", factor=4.0),
                                dict(scaling="base", factor=8.0),
                                dict(scaling="bands", factor=8.0, length=8192.0, low=1.0, high=4.0, base=500000.0),
                                dict(scaling="bands", factor=32.0, length=4096.0, low=0.0, high=32.0)])
def test_rope_turns(rot, kw):
    if kw.get("scaling") == "base" and rot < 4:
        with pytest.raises(nm.NMArgumentError):
            nm.rope_turns(rot, **kw)
        return
    got = nm.rope_turns(rot, **kw).numpy()
    want = ref.rope_turns_ref(rot, **kw)
    assert got.shape == (rot // 2,)
    assert np.all(np.abs(got - want) <= 2.0 ** -46 * want)


def test_rope_turns_base_slows_the_last_pair_by_the_factor():
    plain, slowed = nm.rope_turns(64), nm.rope_turns(64, scaling="base", factor=8.0)
    assert float(slowed[0]) == float(plain[0])
    assert abs(float(plain[-1] / slowed[-1]) - 8.0) < 1e-9


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=1026), dict(rot_dim=8, base=0.0),
                                dict(rot_dim=8, base=math.nan), dict(rot_dim=8, scaling="linear", factor=0.0),
                                dict(rot_dim=8, scaling="bands", factor=2.0, low=4.0, high=4.0),
                                dict(rot_dim=8, scaling="bands", factor=2.0, length=-1.0)])
def test_rope_turns_refusals(kw):
    with pytest.raises(nm.NMArgumentError):
        nm.rope_turns(**kw)


def test_rope_turns_null_and_unknown():
    room = (ctypes.c_double * 4)()
    assert nm.lib().nm_rope_turns(None, 8, 0, 1e4, 1, 1, 0, 1) == nm.NM_ERR_NULL
    assert nm.lib().nm_rope_turns(room, 8, 4, 1e4, 1, 1, 0, 1) == nm.NM_ERR_FORMAT
    with pytest.raises(ValueError):
        nm.rope_turns(8, scaling="other")


# ------------------------------------------------------------------------ binding's checks
def test_binding_needs_gpu_tensors():
    x = torch.zeros(2, 3, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="GPU"):
        nm.nm_rope(x, torch.zeros(2, dtype=torch.int32), torch.zeros(32, dtype=torch.float64))
    with pytest.raises(TypeError):
        nm.nm_rope([1.0], None, None)
    with pytest.raises(ValueError, match="GPU"):
        nm.nm_verify_chain(torch.zeros(1, 2, 5), torch.zeros(1, 1, 5), None, None)
    with pytest.raises(ValueError):
        nm.kv_cache(2, 16, 1, 64, dtype=torch.bfloat16, device="cpu")


def test_rows_checks():
    d = torch.device("cpu")
    fused = torch.zeros(2, 3, 10, 64, dtype=torch.float16)
    p, step = decode._rows(fused[:, :, 2:6], "q", 4, d)
    assert p == fused.data_ptr() + 2 * 2 * 64 and step == 640
    assert decode._rows(fused[:, :1, 2:6], "q", 4, d)[1] == 3 * 640         # one token a sequence
    assert decode._rows(fused[:1, :1], "q", 4, d)[1] == 640
    for bad in (fused[:, :2, 2:6], fused.transpose(2, 3), fused[..., ::2], fused[:, :, ::2]):
        with pytest.raises(ValueError):
            decode._rows(bad, "q", 4, d)
    with pytest.raises(ValueError):
        decode._rows(fused.float(), "q", 4, d)
    with pytest.raises(ValueError):
        decode._rows(fused, "q", 3, d)


def test_cache_checks():
    d = torch.device("cpu")
    c = nm.kv_cache(3, 16, 2, 64, dtype=torch.float8_e4m3fn, device="cpu")
    s = decode._cache_arg(c, d)
    assert (s.blocks, s.kv_heads, s.page, s.head_dim, s.format) == (3, 2, 16, 64, 2)
    with pytest.raises(ValueError):
        decode._cache_arg(c._replace(k_scale=None), d)
    with pytest.raises(ValueError):
        decode._cache_arg(c._replace(v=c.v[:2]), d)
    with pytest.raises(ValueError):
        decode._cache_arg(c._replace(v_scale=c.v_scale.double()), d)
    with pytest.raises(ValueError):
        decode._cache_arg(nm.KVCache(torch.zeros(3, 2, 16, 64), torch.zeros(3, 2, 16, 64)), d)


# ----------------------------------------------------------------------------- the oracle
def test_oracle_e4m3_table():
    t = ref.e4m3_table()
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, want, equal_nan=True)


def test_oracle_rope_turns_a_quarter():
    x = np.arange(1, 9, dtype=np.float64).reshape(1, 1, 8)
    y, _ = ref.rope_ref(x, [1], [0.25, 0.5], "half")
    assert np.allclose(y, [[[-3, -2, 1, -4, 5, 6, 7, 8]]])
    y, _ = ref.rope_ref(x, [1], [0.25, 0.5], "interleaved")
    assert np.allclose(y, [[[-2, 1, -3, -4, 5, 6, 7, 8]]])


def test_oracle_attention_closed_forms():
    v = np.random.default_rng(0).standard_normal((5, 1, 4))
    out, _ = ref.attention_ref(np.zeros((1, 2, 4)), np.ones((5, 1, 4)), v, np.ones((1, 5), bool), 1.0)
    assert np.allclose(out[0], v.mean(0))
    seen = np.zeros((1, 5), bool)
    assert np.all(ref.attention_ref(np.ones((1, 2, 4)), v, v, seen, 1.0)[0] == 0)
    seen[0, 3] = True
    assert np.allclose(ref.attention_ref(np.ones((1, 2, 4)), v, v, seen, 1.0)[0], v[3])


def test_oracle_chain_keeps_the_target_distribution():
    """Over a fine grid of uniforms the first output token's frequencies are the target's."""
    target, draft = np.array([[0.5, 0.2, 0.3], [1.0, 0.0, 0.0]]), np.array([[0.2, 0.7, 0.1]])
    got = np.zeros(3)
    grid = (np.arange(200) + 0.5) / 200
    for x in range(3):
        for u in grid:
            for r in grid[::10]:
                _, out = ref.verify_chain_ref(target, draft, [0, x], [r, u], 2)
                got[out[0]] += draft[0, x] / (grid.size * grid[::10].size)
    assert np.allclose(got, target[0], atol=0.03)


def test_oracle_tree_keeps_the_target_distribution():
    target = np.tile(np.array([0.4, 0.3, 0.2, 0.1]), (4, 1))
    got = np.zeros(4)
    rng = np.random.default_rng(1)
    for u in rng.random((20000, 4)):
        _, out, _ = ref.verify_tree_ref(target, [0, 1, 1, 3], [-1, 0, 0, 0], u, 4)
        got[out[0]] += 1 / 20000
    assert np.allclose(got, target[0], atol=0.02)


@pytest.mark.parametrize("name,base,kw", [
    ("nm_kv_append", "APPEND", dict(batch=1 << 6, tokens=1 << 24, cache_kv_heads=32, k_stride=32 * 128, v_stride=32 * 128)),
    ("nm_rope_kv_append", "ROPE_APPEND", dict(batch=1 << 6, tokens=1 << 22, q_heads=1024, q_stride=1 << 17, q_out_stride=1 << 17)),
    ("nm_kv_read", "READ", dict(batch=1 << 6, tokens=1 << 24, cache_kv_heads=32)),
    ("nm_tree_attention", "ATTEND", dict(batch=4096, cache_kv_heads=4096, heads=4096, q_stride=4096 * 128)),
])
def test_calls_past_a_grid_are_refused(name, base, kw):
    """One grid has fewer than 2^32 threads across; nm_rope takes several, these calls refuse."""
    assert _call(name, globals()[base], kw) == nm.NM_ERR_SHAPE
