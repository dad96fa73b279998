"""Python binding of include/nm_decode.h: what stands between the sparse products of a
speculative decoding step. Rotary positions, a paged key/value cache in fp16, int8 or e4m3,
the attention of drafted trees, chains or single tokens over it, and the verification of the
drafts. Argument marshalling only, as in the rest of the package; every step runs in the HIP
kernels of libnmsparse.so. A call goes through _nmtorch.so (csrc/nm_torch.cpp), which does the
same in a third to half of the host's time; what that does not take (a refusal, tensors of a
device that is not the current one, all calls where the extension is not built) goes through the
checks here, which raise or make the call.
"""
from __future__ import annotations

import ctypes
import functools
import math
import warnings
from typing import NamedTuple, Optional

_c = ctypes
NM_ERR_FORMAT = 8
MAX_NODES = 64                       # nodes of one sequence's step (attention, verification)
LAYOUTS = {"half": 0, "interleaved": 1}
SCALINGS = {"plain": 0, "linear": 1, "base": 2, "bands": 3}


class _CacheStruct(_c.Structure):
    _fields_ = [("k", _c.c_void_p), ("v", _c.c_void_p), ("k_scale", _c.c_void_p), ("v_scale", _c.c_void_p),
                ("blocks", _c.c_int64), ("kv_heads", _c.c_int32), ("page", _c.c_int32),
                ("head_dim", _c.c_int32), ("format", _c.c_int32)]


_P, _I, _L, _F, _D, _Z = _c.c_void_p, _c.c_int, _c.c_int64, _c.c_float, _c.c_double, _c.c_size_t
_C = _c.POINTER(_CacheStruct)
SIGNATURES = {
    "nm_rope_turns": (_I, [_P, _I, _I, _D, _D, _D, _D, _D]),
    "nm_rope": (_I, [_P, _P, _P, _P, _L, _L, _I, _I, _I, _F, _L, _L, _P]),
    "nm_kv_append": (_I, [_C, _P, _P, _L, _L, _P, _L, _P, _P, _L, _L, _P]),
    "nm_rope_kv_append": (_I, [_C, _P, _P, _L, _L, _L, _P, _P, _L, _L, _P, _P, _I, _I, _F, _P, _L, _P, _P, _L, _L, _P]),
    "nm_kv_read": (_I, [_C, _P, _P, _P, _L, _P, _P, _L, _L, _P]),
    "nm_kv_compact": (_I, [_C, _P, _L, _P, _P, _P, _L, _L, _P]),
    "nm_tree_attention": (_I, [_C, _P, _P, _L, _L, _P, _L, _P, _P, _P, _L, _L, _F, _P, _Z, _P]),
    "nm_tree_attention_workspace_bytes": (_Z, [_C, _L, _L, _L, _L]),
    "nm_verify_chain": (_I, [_P, _P, _P, _P, _P, _P, _P, _L, _L, _L, _P, _Z, _P]),
    "nm_verify_tree": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _L, _L, _L, _P, _Z, _P]),
    "nm_verify_workspace_bytes": (_Z, [_L, _L]),
}


def _nm():
    import semi_structured_sparse_amd as nm
    return nm


@functools.lru_cache(None)
def _formats():
    import torch
    return {torch.float16: 0, torch.int8: 1, torch.float8_e4m3fn: 2}


class KVCache(NamedTuple):
    """A paged cache: k and v [blocks, kv_heads, page, head_dim] in fp16, int8 or e4m3, and
    for the 8-bit formats their fp32 scales [blocks, kv_heads, page]. Made by kv_cache(), or
    from tensors of these shapes."""
    k: "torch.Tensor"
    v: "torch.Tensor"
    k_scale: Optional["torch.Tensor"] = None
    v_scale: Optional["torch.Tensor"] = None


def kv_cache(blocks: int, page: int, kv_heads: int, head_dim: int, dtype=None, device=None) -> KVCache:
    """A cache of zeros. dtype: torch.float16 (default), torch.int8 or torch.float8_e4m3fn."""
    import torch
    dtype = torch.float16 if dtype is None else dtype
    if dtype not in _formats():
        raise ValueError(f"a cache is fp16, int8 or float8_e4m3fn, not {dtype}")
    device = torch.device("cuda" if device is None else device)
    shape = (blocks, kv_heads, page, head_dim)
    k, v = (torch.zeros(shape, dtype=torch.uint8 if dtype == torch.float8_e4m3fn else dtype, device=device).view(dtype)
            for _ in range(2))
    if dtype == torch.float16:
        return KVCache(k, v)
    return KVCache(k, v, *(torch.zeros(shape[:3], dtype=torch.float32, device=device) for _ in range(2)))


def _tensor(t, name, dtype, shape, device):
    """Checks a contiguous tensor argument and returns its address (None for None)."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if t.device != device:
            raise ValueError(f"{name} must be on {device}, got {t.device}")
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _device_of(t, name):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device (no CPU path)")
    return t.device


def _rows(t, name, ndim, device):
    """Checks fp16 [..., heads, head_dim] whose heads are contiguous and whose leading dims are
    evenly spaced tokens; returns (address, token stride in elements)."""
    import torch
    if t.dtype != torch.float16:
        raise ValueError(f"{name} must be {torch.float16}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    size, step = t.shape, t.stride()
    row = size[-1] * size[-2]
    if (step[-1] != 1 and size[-1] > 1) or (step[-2] != size[-1] and size[-2] > 1):
        raise ValueError(f"{name}'s heads must be contiguous")
    if ndim == 3:
        return t.data_ptr(), step[0] if size[0] > 1 else row
    if size[1] == 1:
        return t.data_ptr(), step[0] if size[0] > 1 else row
    if size[0] > 1 and step[0] != size[1] * step[1]:
        raise ValueError(f"{name}'s tokens must be evenly spaced over the batch")
    return t.data_ptr(), step[1]


def _cache_arg(cache, device):
    """The C structure of a cache, with its tensors checked."""
    import torch
    k, v, k_scale, v_scale = cache
    form = _formats().get(k.dtype)
    if not form:
        k_scale = v_scale = None
    if form is None:
        raise ValueError(f"a cache is fp16, int8 or float8_e4m3fn, not {k.dtype}")
    if k.dim() != 4:
        raise ValueError("a cache's k and v must be [blocks, kv_heads, page, head_dim]")
    shape = k.shape
    if form:
        if k_scale is None or v_scale is None:
            raise ValueError("an 8-bit cache needs k_scale and v_scale")
        k_scale = _tensor(k_scale, "cache.k_scale", torch.float32, shape[:3], device)
        v_scale = _tensor(v_scale, "cache.v_scale", torch.float32, shape[:3], device)
    return _CacheStruct(_tensor(k, "cache.k", k.dtype, shape, device), _tensor(v, "cache.v", k.dtype, shape, device),
                        k_scale, v_scale, *shape, form)


def _paging(table, first, first_name, count, batch, device):
    """Checks a page table and its per-sequence lengths; returns their addresses."""
    import torch
    if table.dim() != 2:
        raise ValueError("block_table must be [batch, pages]")
    return (_tensor(table, "block_table", torch.int32, (batch, table.shape[1]), device),
            _tensor(first, first_name, torch.int32, (batch,), device),
            _tensor(count, "count", torch.int32, (batch,), device))


_functions = {}   # of the loaded library, by name
_quick = None     # _nmtorch, bound to that library on the first call
_QUICK = ("nm_rope", "nm_kv_append", "nm_rope_kv_append", "nm_kv_read", "nm_kv_compact", "nm_tree_attention",
          "nm_verify_chain", "nm_verify_tree")


class _Absent:
    """Stands for the extension where it does not load, and takes no call."""

    def __getattr__(self, name):
        return lambda *args: NotImplemented


def _bound():
    global _quick
    if _quick is None:
        lib = _nm().lib()
        try:
            from . import _nmtorch
        except ImportError as e:
            warnings.warn(f"_nmtorch.so does not load ({e}): the decoding calls take longer on the host; build it with "
                          "python -m semi_structured_sparse_amd.build", RuntimeWarning, stacklevel=3)
            _quick = _Absent()
            return _quick
        _nmtorch.bind(*(_c.cast(getattr(lib, name), _c.c_void_p).value for name in _QUICK))
        _quick = _nmtorch
    return _quick


def _run(name, device, *args):
    """Calls the library on the tensors' device and its current stream."""
    import torch
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(_nm().lib(), name)
    index = device.index
    # the stream's handle without a Stream object: 0.1 us in place of 1.9
    if torch.cuda.current_device() == index:
        st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if st:
        _nm()._check(name, st)


def _layout(layout):
    if layout not in LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(LAYOUTS)}")
    return LAYOUTS[layout]


def _turns(turns, device):
    import torch
    if turns.dim() != 1:
        raise ValueError("turns must be [rot_dim / 2]")
    return _tensor(turns, "turns", torch.float64, turns.shape, device), 2 * turns.shape[0]


def rope_turns(rot_dim: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
               length: float = 8192.0, low: float = 1.0, high: float = 4.0, device=None):
    """fp64 [rot_dim/2]: the turns each pair makes per position (an inverse frequency in radians
    divided by 2 pi). scaling: "plain", "linear", "base" or "bands", as nm_decode.h defines."""
    import torch
    if scaling not in SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(SCALINGS)}")
    nm = _nm()
    turns = torch.empty(max(1, rot_dim // 2), dtype=torch.float64)
    room = turns.data_ptr()
    nm._check("nm_rope_turns", nm.lib().nm_rope_turns(room, rot_dim, SCALINGS[scaling], base, factor, length, low, high))
    return turns if device is None else turns.to(device)


def nm_rope(x, positions, turns, layout: str = "half", scale: float = 1.0, out=None):
    """Rotary positions on x fp16 [tokens, heads, head_dim] (a slice of a fused projection's
    output will do): the first 2 * len(turns) elements of each head turned by positions int32
    [tokens], the rest copied. out: fp16 of x's shape, x itself included; made if not given."""
    done = (_quick or _bound()).nm_rope(x, positions, turns, LAYOUTS.get(layout, -1), scale, out)
    if done is not NotImplemented:
        return done
    import torch
    device = _device_of(x, "x")
    xp, xs = _rows(x, "x", 3, device)
    tokens, heads, dim = x.shape
    if out is None:
        out = x.new_empty((tokens, heads, dim))
    elif out.shape != x.shape:
        raise ValueError("out must have x's shape")
    yp, ys = _rows(out, "out", 3, device)
    tp, rot = _turns(turns, device)
    _run("nm_rope", device, xp, yp, _tensor(positions, "positions", torch.int32, (tokens,), device), tp, tokens, heads,
         dim, rot, _layout(layout), scale, xs, ys)
    return out


def nm_kv_append(cache: KVCache, k, v, block_table, start, count=None) -> None:
    """Writes k, v fp16 [batch, tokens, kv_heads, head_dim] into the cache at positions
    start[b] + t of sequences whose pages block_table int32 [batch, pages] lists, for t below
    count[b] (int32, None: all)."""
    done = (_quick or _bound()).nm_kv_append(*cache, k, v, block_table, start, count)
    if done is not NotImplemented:
        return done
    device = _device_of(k, "k")
    c = _cache_arg(cache, device)
    kp, ks = _rows(k, "k", 4, device)
    vp, vs = _rows(v, "v", 4, device)
    batch, tokens = k.shape[:2]
    if k.shape != v.shape or k.shape[2] != c.kv_heads or k.shape[3] != c.head_dim:
        raise ValueError(f"k and v must be [batch, tokens, {c.kv_heads}, {c.head_dim}]")
    tp, sp, np_ = _paging(block_table, start, "start", count, batch, device)
    _run("nm_kv_append", device, c, kp, vp, ks, vs, tp, block_table.shape[1], sp, np_, batch, tokens)


def nm_rope_kv_append(cache: KVCache, q, k, v, positions, turns, block_table, start, count=None,
                      layout: str = "half", scale: float = 1.0, out=None):
    """nm_rope on q and k and nm_kv_append in one launch: returns q turned, fp16 [batch, tokens,
    heads, head_dim] (zeros for tokens at or past count; out may be q). positions int32 [batch,
    tokens]. q None: k and v only, returns None."""
    done = (_quick or _bound()).nm_rope_kv_append(*cache, q, k, v, positions, turns, block_table, start, count,
                                                  LAYOUTS.get(layout, -1), scale, out)
    if done is not NotImplemented:
        return done
    import torch
    device = _device_of(k, "k")
    c = _cache_arg(cache, device)
    kp, ks = _rows(k, "k", 4, device)
    vp, vs = _rows(v, "v", 4, device)
    batch, tokens = k.shape[:2]
    if k.shape != v.shape or k.shape[2] != c.kv_heads or k.shape[3] != c.head_dim:
        raise ValueError(f"k and v must be [batch, tokens, {c.kv_heads}, {c.head_dim}]")
    qp, qs, op, os_, heads = None, 0, None, 0, 0
    if q is not None:
        qp, qs = _rows(q, "q", 4, device)
        heads = q.shape[2]
        if q.shape[:2] != k.shape[:2] or q.shape[3] != c.head_dim:
            raise ValueError(f"q must be [{batch}, {tokens}, heads, {c.head_dim}]")
        if out is None:
            out = q.new_empty((batch, tokens, heads, c.head_dim))
        elif out.shape != q.shape:
            raise ValueError("out must have q's shape")
        op, os_ = _rows(out, "out", 4, device)
    rp, rot = _turns(turns, device)
    tp, sp, np_ = _paging(block_table, start, "start", count, batch, device)
    _run("nm_rope_kv_append", device, c, qp, op, heads, qs, os_, kp, vp, ks, vs,
         _tensor(positions, "positions", torch.int32, (batch, tokens), device), rp, rot, _layout(layout), scale,
         tp, block_table.shape[1], sp, np_, batch, tokens)
    return out


def nm_kv_read(cache: KVCache, block_table, start, tokens: int, count=None, out=None):
    """(k, v) fp16 [batch, tokens, kv_heads, head_dim]: the values at positions start[b] + t, zeros
    for t at or past count[b]. out: a pair of such tensors."""
    done = (_quick or _bound()).nm_kv_read(*cache, block_table, start, tokens, count, *((None, None) if out is None else out))
    if done is not NotImplemented:
        return done
    import torch
    device = _device_of(block_table, "block_table")
    c = _cache_arg(cache, device)
    batch = block_table.shape[0]
    shape = (batch, tokens, c.kv_heads, c.head_dim)
    if out is None:
        out = (torch.empty(shape, dtype=torch.float16, device=device), torch.empty(shape, dtype=torch.float16, device=device))
    kp, vp = (_tensor(t, name, torch.float16, shape, device) for t, name in zip(out, ("out[0]", "out[1]")))
    tp, sp, np_ = _paging(block_table, start, "start", count, batch, device)
    _run("nm_kv_read", device, c, kp, vp, tp, block_table.shape[1], sp, np_, batch, tokens)
    return out


def nm_kv_compact(cache: KVCache, block_table, start, path, accepted) -> None:
    """Moves the rows at start[b] + path[b, d] to start[b] + d for 1 <= d <= accepted[b]: path
    int32 [batch, nodes] and accepted int32 [batch] as nm_verify_tree returns them."""
    done = (_quick or _bound()).nm_kv_compact(*cache, block_table, start, path, accepted)
    if done is not NotImplemented:
        return done
    import torch
    device = _device_of(block_table, "block_table")
    c = _cache_arg(cache, device)
    batch = block_table.shape[0]
    tp, sp, ap = _paging(block_table, start, "start", accepted, batch, device)
    if path.dim() != 2:
        raise ValueError("path must be [batch, nodes]")
    pp = _tensor(path, "path", torch.int32, (batch, path.shape[1]), device)
    _run("nm_kv_compact", device, c, tp, block_table.shape[1], sp, pp, ap, batch, path.shape[1])


def tree_attention_workspace(q, cache: KVCache, block_table):
    """A zeroed workspace for nm_tree_attention of these shapes (None where it takes none), made once
    for the largest step: it serves steps of fewer nodes, sequences or pages too, and the nm_verify
    calls, in stream order (a call that would take more splits as far as it goes)."""
    import torch
    device = _device_of(q, "q")
    c = _cache_arg(cache, device)
    with torch.cuda.device(device):
        n = _nm().lib().nm_tree_attention_workspace_bytes(c, q.shape[2], block_table.shape[1], q.shape[0], q.shape[1])
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def _workspace(workspace, device):
    import torch
    if workspace is None:
        return None, 0
    return _tensor(workspace, "workspace", torch.uint8, (workspace.numel(),), device), workspace.numel()


def nm_tree_attention(q, cache: KVCache, block_table, context, mask=None, count=None, scale: float | None = None,
                      workspace=None, out=None):
    """Attention of the nodes of each sequence's step: q fp16 [batch, tokens, heads, head_dim]
    over the context[b] cached positions and the nodes' own, which mask int64 [batch, tokens]
    allows by bits (None: a chain). count int32 [batch]: nodes of each sequence. scale: 1/sqrt of
    head_dim if None. workspace: from tree_attention_workspace, or None (long contexts are then
    not split over the GPU)."""
    done = (_quick or _bound()).nm_tree_attention(q, *cache, block_table, context, mask, count, scale, workspace, out)
    if done is not NotImplemented:
        return done
    import torch
    device = _device_of(q, "q")
    c = _cache_arg(cache, device)
    qp, qs = _rows(q, "q", 4, device)
    batch, tokens, heads, dim = q.shape
    if dim != c.head_dim:
        raise ValueError(f"q's heads have {dim} elements, the cache's {c.head_dim}")
    if out is None:
        out = q.new_empty((batch, tokens, heads, dim))
    op = _tensor(out, "out", torch.float16, (batch, tokens, heads, dim), device)
    tp, xp, np_ = _paging(block_table, context, "context", count, batch, device)
    mp = _tensor(mask, "mask", torch.int64, (batch, tokens), device)
    wp, wn = _workspace(workspace, device)
    _run("nm_tree_attention", device, c, qp, op, heads, qs, tp, block_table.shape[1], xp, mp, np_, batch, tokens,
         1.0 / math.sqrt(dim) if scale is None else scale, wp, wn)
    return out


def verify_workspace(batch: int, vocab: int, device=None):
    """A zeroed workspace for the nm_verify calls of these sizes, or fewer sequences (None where they
    take none)."""
    import torch
    device = torch.device("cuda" if device is None else device)
    with torch.cuda.device(device):
        n = _nm().lib().nm_verify_workspace_bytes(batch, vocab)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def _verify_args(target, tokens, uniforms, count, workspace):
    import torch
    device = _device_of(target, "target")
    if target.dim() != 3:
        raise ValueError("target must be [batch, nodes, vocab]")
    batch, nodes, vocab = target.shape
    given = (_tensor(tokens, "tokens", torch.int32, (batch, nodes), device),
             _tensor(uniforms, "uniforms", torch.float32, (batch, nodes), device),
             _tensor(count, "count", torch.int32, (batch,), device))
    made = tokens.new_empty((batch,)), tokens.new_empty((batch, nodes))
    return (device, _tensor(target, "target", torch.float32, (batch, nodes, vocab), device), given, made,
            (batch, nodes, vocab, *_workspace(workspace, device)))


def nm_verify_chain(target, draft, tokens, uniforms, count=None, workspace=None):
    """Rejection sampling of a drafted chain: target fp32 [batch, nodes, vocab], draft fp32 [batch,
    nodes-1, vocab], tokens int32 and uniforms fp32 [batch, nodes]. Returns (accepted int32 [batch],
    out_tokens int32 [batch, nodes]: the accepted drafts, the token drawn after them, then -1)."""
    done = (_quick or _bound()).nm_verify_chain(target, draft, tokens, uniforms, count, workspace)
    if done is not NotImplemented:
        return done
    import torch
    device, tp, (kp, up, np_), (accepted, out), rest = _verify_args(target, tokens, uniforms, count, workspace)
    batch, nodes, vocab = target.shape
    dp = _tensor(draft, "draft", torch.float32, (batch, nodes - 1, vocab), device)
    _run("nm_verify_chain", device, tp, dp or None, kp, up, np_, accepted.data_ptr(), out.data_ptr(), *rest)
    return accepted, out


def nm_verify_tree(target, tokens, parents, uniforms, count=None, workspace=None):
    """Verification of a tree of chosen tokens: parents int32 [batch, nodes], the rest as
    nm_verify_chain. Returns (accepted, out_tokens, path int32 [batch, nodes]: the nodes reached,
    from node 0 on, then -1)."""
    done = (_quick or _bound()).nm_verify_tree(target, parents, tokens, uniforms, count, workspace)
    if done is not NotImplemented:
        return done
    import torch
    device, tp, (kp, up, np_), (accepted, out), rest = _verify_args(target, tokens, uniforms, count, workspace)
    batch, nodes, _ = target.shape
    path = tokens.new_empty((batch, nodes))
    _run("nm_verify_tree", device, tp, kp, _tensor(parents, "parents", torch.int32, (batch, nodes), device), up, np_,
         accepted.data_ptr(), out.data_ptr(), path.data_ptr(), *rest)
    return accepted, out, path
