"""Python binding of include/nm_block.h: what a transformer block does around its sparse products.
Products with bias, activation, scale and residual, the gated feed-forward's two products as one,
the norms before and after a block with the residual addition between them, and the log
probabilities of its answers. Argument marshalling only, as in the rest of the package; every step
runs in the HIP kernels of libnmsparse.so. A call goes through _nmtorch.so (csrc/nm_torch.cpp), and
where that does not take it through the checks here, which raise or make the call, as in decode.py.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

from . import decode as _d

_c = ctypes
ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
NORMS = {"rms": 0, "layer": 1}
MAX_TOP = 64                         # alternatives of a row (nm_logprobs)

_P, _I, _L, _F, _Z = _c.c_void_p, _c.c_int, _c.c_int64, _c.c_float, _c.c_size_t
SIGNATURES = {
    "nm_linear": (_I, [_P, _P, _P, _P, _L, _L, _L, _I, _I, _P, _I, _F, _P, _P, _Z, _P]),
    "nm_gated": (_I, [_P, _P, _P, _P, _P, _P, _L, _L, _L, _I, _I, _P, _P, _I, _P, _Z, _P]),
    "nm_gated_workspace_bytes": (_Z, [_L, _L, _L, _I, _I]),
    "nm_norm": (_I, [_P, _P, _P, _P, _L, _L, _L, _L, _L, _I, _I, _F, _F, _P]),
    "nm_block_norm": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _L, _L, _L, _L, _L, _L, _L, _I, _I, _F, _F, _F, _P]),
    "nm_logprobs": (_I, [_P, _P, _P, _P, _P, _P, _L, _L, _L, _L, _I, _F, _P, _Z, _P]),
    "nm_logprobs_workspace_bytes": (_Z, [_L, _L]),
}


class LogProbs(NamedTuple):
    """What nm_logprobs returns; the last two are None where no alternatives were asked for, the first
    where no tokens were given."""
    logprob: Optional["torch.Tensor"]
    entropy: "torch.Tensor"
    top_tokens: Optional["torch.Tensor"]
    top_logprobs: Optional["torch.Tensor"]


def _nm():
    import semi_structured_sparse_amd as nm
    return nm


def _activation(name):
    if name not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {[a for a in ACTIVATIONS if a]} or None")
    return ACTIVATIONS[name]


def _kind(name):
    if name not in NORMS:
        raise ValueError(f"kind must be one of {sorted(NORMS)}")
    return NORMS[name]


def _matrix(values, masks, names, N, M, device):
    """Checks a packed matrix; returns its addresses, rows and columns."""
    import torch
    nm = _nm()
    nm._require(values, names[0], torch.float16, 2)
    nm._require(masks, names[1], torch.int32, 2)
    rows, words = masks.shape
    cols = words * 32
    if (N, M) in nm.ALL_PATTERNS and values.shape != (rows, cols * N // M):
        raise ValueError(f"{names[0]} shape {tuple(values.shape)} != {(rows, cols * N // M)}")
    if values.device != device or masks.device != device:
        raise ValueError(f"{names[0]}, {names[1]} and X must be on one device")
    return values.data_ptr(), masks.data_ptr(), rows, cols


def _vectors(X):
    """Checks X fp16 [cols] or [batch, cols]; returns its device and batch."""
    import torch
    device = _d._device_of(X, "X")
    if X.dim() not in (1, 2):
        raise ValueError(f"X must be [cols] or [batch, cols], got {X.dim()} dims")
    _nm()._require(X, "X", torch.float16, X.dim())
    return device, X.shape[0] if X.dim() == 2 else 1


def _product_out(X, rows, out, device):
    import torch
    shape = (*X.shape[:-1], rows)
    if out is None:
        out = X.new_empty(shape)
    return out, _d._tensor(out, "out", torch.float16, shape, device)


def linear_workspace(rows: int, cols: int, batch: int, N: int, M: int, device=None):
    """A zeroed workspace for nm_linear of this shape (None where it takes none): nm_spmm_ws's."""
    return _nm().spmm_workspace(rows, cols, batch, N, M, device)


def nm_linear(values, masks, X, N: int, M: int, bias=None, activation: str | None = None, scale: float = 1.0,
              residual=None, workspace=None, out=None):
    """scale * act(X W'^T + bias) + residual, of the packed (values, masks): X fp16 [cols] or [batch,
    cols] -> fp16 [rows] or [batch, rows]. bias fp16 [rows]; residual fp16 of the result's shape, and
    may be out. activation: None, "relu", "silu", "gelu" or "gelu_tanh". Products and sums in 32 bits,
    one rounding. workspace: as nm_spmm_ws."""
    done = (_d._quick or _d._bound()).nm_linear(values, masks, X, N, M, bias, ACTIVATIONS.get(activation, -1), scale, residual,
                                                workspace, out)
    if done is not NotImplemented:
        return done
    import torch
    device, batch = _vectors(X)
    vp, mp, rows, cols = _matrix(values, masks, ("values", "masks"), N, M, device)
    if X.shape[-1] != cols:
        raise ValueError(f"X has {X.shape[-1]} columns, masks describe {cols}")
    out, op = _product_out(X, rows, out, device)
    bp = _d._tensor(bias, "bias", torch.float16, (rows,), device)
    rp = _d._tensor(residual, "residual", torch.float16, out.shape, device)
    _d._run("nm_linear", device, vp, mp, X.data_ptr(), op, rows, cols, batch, N, M, bp, _activation(activation), scale, rp,
            *_d._workspace(workspace, device))
    return out


def gated_workspace(rows: int, cols: int, batch: int, N: int, M: int, device=None):
    """A zeroed workspace for nm_gated of this shape (None where it takes none)."""
    import torch
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(dev):
        n = _nm().lib().nm_gated_workspace_bytes(rows, cols, batch, N, M)
    return torch.zeros(n, dtype=torch.uint8, device=dev) if n else None


def nm_gated(gate, up, X, N: int, M: int, activation: str | None = "silu", gate_bias=None, up_bias=None, workspace=None,
             out=None):
    """act(X Wg'^T + gate_bias) * (X Wu'^T + up_bias), gate and up the packed (values, masks) of two
    matrices of one shape and pattern: X fp16 [cols] or [batch, cols] -> fp16 [rows] or [batch, rows].
    workspace: from gated_workspace, or None (columns are then not split)."""
    done = (_d._quick or _d._bound()).nm_gated(*gate, *up, X, N, M, ACTIVATIONS.get(activation, -1), gate_bias, up_bias,
                                               workspace, out)
    if done is not NotImplemented:
        return done
    import torch
    device, batch = _vectors(X)
    gv, gm, rows, cols = _matrix(*gate, ("gate[0]", "gate[1]"), N, M, device)
    uv, um, up_rows, up_cols = _matrix(*up, ("up[0]", "up[1]"), N, M, device)
    if (up_rows, up_cols) != (rows, cols):
        raise ValueError(f"gate is {(rows, cols)}, up {(up_rows, up_cols)}")
    if X.shape[-1] != cols:
        raise ValueError(f"X has {X.shape[-1]} columns, masks describe {cols}")
    out, op = _product_out(X, rows, out, device)
    _d._run("nm_gated", device, gv, gm, uv, um, X.data_ptr(), op, rows, cols, batch, N, M,
            _d._tensor(gate_bias, "gate_bias", torch.float16, (rows,), device),
            _d._tensor(up_bias, "up_bias", torch.float16, (rows,), device), _activation(activation),
            *_d._workspace(workspace, device))
    return out


def _spaced(t, name, dtypes, device):
    """Checks rows [..., width]: [width], [rows, width] with any row stride, or [(batch,) tokens, heads,
    width] as decode.py takes them. Returns (address, tokens, heads, width, token stride)."""
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    size, step, dims = t.shape, t.stride(), t.dim()
    if not 1 <= dims <= 4:
        raise ValueError(f"{name} must have 1 to 4 dims, got {dims}")
    if step[-1] != 1 and size[-1] > 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    heads = size[-2] if dims > 2 else 1
    if dims > 2 and step[-2] != size[-1] and heads > 1:
        raise ValueError(f"{name}'s heads must be contiguous")
    row = heads * size[-1]
    if dims == 1:
        return t.data_ptr(), 1, 1, size[0], row
    if dims == 2 or dims == 3:
        return t.data_ptr(), size[0], heads, size[-1], step[0] if size[0] > 1 else row
    if size[1] == 1:
        return t.data_ptr(), size[0], heads, size[-1], step[0] if size[0] > 1 else row
    if size[0] > 1 and step[0] != size[1] * step[1]:
        raise ValueError(f"{name}'s tokens must be evenly spaced over the batch")
    return t.data_ptr(), size[0] * size[1], heads, size[-1], step[1]


def nm_norm(x, weight=None, bias=None, kind: str = "rms", offset: float = 0.0, eps: float = 1e-6, out=None):
    """The norm of each row of x, fp16 or fp32 [rows, width] with any row stride, [width], or heads
    [(batch,) tokens, heads, width] as a slice of a fused projection's output: x / sqrt(mean(x^2) + eps)
    * (offset + weight) + bias, fp16 of x's shape; kind "layer" takes the mean off x first. weight and
    bias fp16 [width]. out: fp16 of x's shape, x itself included; made if not given."""
    done = (_d._quick or _d._bound()).nm_norm(x, weight, bias, NORMS.get(kind, -1), offset, eps, out)
    if done is not NotImplemented:
        return done
    import torch
    device = _d._device_of(x, "x")
    xp, tokens, heads, width, xs = _spaced(x, "x", (torch.float16, torch.float32), device)
    if out is None:
        out = torch.empty(x.shape, dtype=torch.float16, device=device)
    elif out.shape != x.shape:
        raise ValueError("out must have x's shape")
    yp, _, _, _, ys = _spaced(out, "out", (torch.float16,), device)
    _d._run("nm_norm", device, xp, yp, _d._tensor(weight, "weight", torch.float16, (width,), device),
            _d._tensor(bias, "bias", torch.float16, (width,), device), tokens, heads, width, xs, ys,
            int(x.dtype == torch.float32), _kind(kind), offset, eps)
    return out


def nm_block_norm(x, branch, weight=None, bias=None, post=None, gate=None, scale: float = 1.0, kind: str = "rms",
                  offset: float = 0.0, eps: float = 1e-6, h=None, out=None):
    """Between two blocks: h = x + scale * gate * post(branch), y = norm(h); returns (y, h). x, the
    residual stream, fp16 or fp32 [rows, width] with any row stride; branch fp16, likewise; post: the
    weight of the norm after the branch, fp16 [width], or None (the branch as it is); gate fp16 [width]
    or [rows, width], or None; weight and bias as nm_norm's. y fp16, h of x's type; h may be x, out may
    be branch; made if not given. y is the norm of h before its rounding."""
    done = (_d._quick or _d._bound()).nm_block_norm(x, branch, weight, bias, post, gate, scale, NORMS.get(kind, -1), offset,
                                                    eps, h, out)
    if done is not NotImplemented:
        return done
    import torch
    device = _d._device_of(x, "x")
    if x.dim() > 2 or x.shape != branch.shape:
        raise ValueError("x and branch must be [rows, width] or [width], of one shape")
    both = (torch.float16, torch.float32)
    xp, rows, _, width, xs = _spaced(x, "x", both, device)
    bp, _, _, _, bs = _spaced(branch, "branch", both[:1], device)
    h = torch.empty(x.shape, dtype=x.dtype, device=device) if h is None else h
    out = torch.empty(x.shape, dtype=torch.float16, device=device) if out is None else out
    if h.shape != x.shape or out.shape != x.shape:
        raise ValueError("h and out must have x's shape")
    hp, _, _, _, hs = _spaced(h, "h", (x.dtype,), device)
    yp, _, _, _, ys = _spaced(out, "out", both[:1], device)
    gp, gs = None, 0
    if gate is not None:
        if gate.dim() == 2:
            if gate.shape != x.shape:
                raise ValueError(f"gate must have shape {(width,)} or {tuple(x.shape)}, got {tuple(gate.shape)}")
            gp, _, _, _, gs = _spaced(gate, "gate", both[:1], device)
        else:
            gp = _d._tensor(gate, "gate", torch.float16, (width,), device)
    wp, cp, pp = (_d._tensor(t, name, torch.float16, (width,), device)
                  for t, name in ((weight, "weight"), (bias, "bias"), (post, "post")))
    _d._run("nm_block_norm", device, xp, bp, hp, yp, pp, gp, wp, cp, rows, width, xs, bs, hs, ys, gs,
            int(x.dtype == torch.float32), _kind(kind), scale, offset, eps)
    return out, h


def logprobs_workspace(rows: int, vocab: int, device=None):
    """A zeroed workspace for nm_logprobs of these sizes, or fewer rows (None where it takes none). It
    serves the calls of decode.py too, in stream order."""
    import torch
    device = torch.device("cuda" if device is None else device)
    with torch.cuda.device(device):
        n = _nm().lib().nm_logprobs_workspace_bytes(rows, vocab)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def nm_logprobs(logits, tokens=None, top: int = 0, scale: float = 1.0, workspace=None) -> LogProbs:
    """Of each row of logits, fp32 or fp16 [rows, vocab] with any row stride, times scale (a temperature's
    inverse): the log probability of tokens int32 [rows] (0 for negative ones), the entropy, and the
    `top` (at most 64) most likely tokens with their log probabilities, best first, ties to the lower
    token. fp32 and int32. Logits of -infinity are never listed (token -1, log probability -infinity) and
    are the mask to use where alternatives are asked for: finite ones are logits like others, whose ties
    take long. A row with NaN or +infinity gives NaN. workspace: from logprobs_workspace, or None (rows
    are then not split over the GPU)."""
    done = (_d._quick or _d._bound()).nm_logprobs(logits, tokens, top, scale, workspace)
    if done is not NotImplemented:
        return LogProbs(*done)
    import torch
    device = _d._device_of(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be [rows, vocab]")
    lp, rows, _, vocab, stride = _spaced(logits, "logits", (torch.float32, torch.float16), device)
    tp = _d._tensor(tokens, "tokens", torch.int32, (rows,), device)
    if not 0 <= top <= min(MAX_TOP, vocab):
        raise ValueError(f"top must be 0 .. {min(MAX_TOP, vocab)}, got {top}")
    entropy = torch.empty(rows, dtype=torch.float32, device=device)
    logprob = torch.empty_like(entropy) if tokens is not None else None
    top_tokens = torch.empty((rows, top), dtype=torch.int32, device=device) if top else None
    top_logprobs = torch.empty((rows, top), dtype=torch.float32, device=device) if top else None
    _d._run("nm_logprobs", device, lp, tp, *(None if t is None else t.data_ptr() for t in
                                             (logprob, entropy, top_tokens, top_logprobs)),
            rows, vocab, stride, top, int(logits.dtype == torch.float16), scale, *_d._workspace(workspace, device))
    return LogProbs(logprob, entropy, top_tokens, top_logprobs)
