"""CPU tests of the block operators: refusals (no HIP call is made before the arguments pass), the
binding's checks, and the reference forms against closed ones."""
import math

import pytest
import torch

import semi_structured_sparse_amd as nm
from semi_structured_sparse_amd import block
from tests import block_bounds as ref

A = 0x10000   # an aligned fake device address: checks never dereference it

LINEAR = dict(values=A, masks=A, X=A, Y=A, rows=16, cols=64, batch=2, N=2, M=4, bias=A, activation=2, scale=1.0, residual=A,
              workspace=None, workspace_bytes=0, stream=None)
GATED = dict(gate_values=A, gate_masks=A, up_values=A, up_masks=A, X=A, Y=A, rows=16, cols=64, batch=2, N=2, M=4, gate_bias=A,
             up_bias=A, activation=2, workspace=None, workspace_bytes=0, stream=None)
NORM = dict(x=A, y=A, weight=A, bias=A, tokens=3, heads=2, width=64, x_stride=128, y_stride=128, fp32_input=0, kind=0,
            offset=0.0, eps=1e-6, stream=None)
BLOCK_NORM = dict(x=A, branch=A, h=A, y=A, post=A, gate=A, weight=A, bias=A, rows=3, width=64, x_stride=64, branch_stride=64,
                  h_stride=64, y_stride=64, gate_stride=64, fp32_stream=1, kind=1, scale=1.0, offset=0.0, eps=1e-6, stream=None)
LOGPROBS = dict(logits=A, tokens=A, logprob=A, entropy=A, top_tokens=A, top_logprobs=A, rows=3, vocab=100, stride=100, top=5,
                fp16_logits=1, scale=1.0, workspace=None, workspace_bytes=0, stream=None)

PRODUCT = [(dict(X=None), nm.NM_ERR_NULL), (dict(Y=None), nm.NM_ERR_NULL), (dict(rows=0), nm.NM_ERR_SHAPE),
           (dict(cols=48), nm.NM_ERR_SHAPE), (dict(cols=0), nm.NM_ERR_SHAPE), (dict(batch=0), nm.NM_ERR_SHAPE),
           (dict(batch=(1 << 24) + 1), nm.NM_ERR_SHAPE), (dict(N=3), nm.NM_ERR_PATTERN), (dict(N=1, M=4), nm.NM_ERR_PATTERN),
           (dict(activation=5), nm.NM_ERR_FORMAT), (dict(activation=-1), nm.NM_ERR_FORMAT), (dict(X=A + 8), nm.NM_ERR_ALIGN),
           (dict(Y=A + 1), nm.NM_ERR_ALIGN), (dict(workspace=A + 8, workspace_bytes=4096), nm.NM_ERR_ALIGN)]
ROWS = [(dict(x=None), nm.NM_ERR_NULL), (dict(y=None), nm.NM_ERR_NULL), (dict(kind=2), nm.NM_ERR_FORMAT),
        (dict(kind=-1), nm.NM_ERR_FORMAT), (dict(width=0), nm.NM_ERR_SHAPE), (dict(width=32769), nm.NM_ERR_SHAPE),
        (dict(width=(1 << 32) + 64), nm.NM_ERR_SHAPE), (dict(x_stride=63), nm.NM_ERR_SHAPE), (dict(y_stride=63), nm.NM_ERR_SHAPE),
        (dict(x_stride=1 << 41), nm.NM_ERR_SHAPE), (dict(eps=-1.0), nm.NM_ERR_SHAPE), (dict(eps=math.nan), nm.NM_ERR_SHAPE),
        (dict(eps=math.inf), nm.NM_ERR_SHAPE), (dict(offset=math.nan), nm.NM_ERR_SHAPE), (dict(y=A + 1), nm.NM_ERR_ALIGN),
        (dict(weight=A + 1), nm.NM_ERR_ALIGN), (dict(bias=A + 1), nm.NM_ERR_ALIGN)]
REFUSED = (
    [("nm_linear", LINEAR, kw, st) for kw, st in PRODUCT + [
        (dict(values=None), nm.NM_ERR_NULL), (dict(masks=None), nm.NM_ERR_NULL), (dict(bias=A + 1), nm.NM_ERR_ALIGN),
        (dict(residual=A + 1), nm.NM_ERR_ALIGN), (dict(values=A + 8), nm.NM_ERR_ALIGN), (dict(rows=1 << 31), nm.NM_ERR_SHAPE),
        (dict(rows=1 << 26), nm.NM_ERR_SHAPE), (dict(rows=1 << 20, batch=(1 << 15) + 1), nm.NM_ERR_SHAPE)]] +
    [("nm_gated", GATED, kw, st) for kw, st in PRODUCT + [
        (dict(gate_values=None), nm.NM_ERR_NULL), (dict(gate_masks=None), nm.NM_ERR_NULL), (dict(up_values=None), nm.NM_ERR_NULL),
        (dict(up_masks=None), nm.NM_ERR_NULL), (dict(gate_bias=A + 1), nm.NM_ERR_ALIGN), (dict(up_bias=A + 1), nm.NM_ERR_ALIGN),
        (dict(up_values=A + 8), nm.NM_ERR_ALIGN), (dict(up_masks=A + 2), nm.NM_ERR_ALIGN), (dict(rows=1 << 30), nm.NM_ERR_SHAPE),
        (dict(rows=(1 << 63) - 1), nm.NM_ERR_SHAPE), (dict(rows=1 << 25), nm.NM_ERR_SHAPE),
        (dict(rows=1 << 20, batch=(1 << 14) + 1), nm.NM_ERR_SHAPE)]] +
    [("nm_norm", NORM, kw, st) for kw, st in ROWS + [
        (dict(tokens=0), nm.NM_ERR_SHAPE), (dict(heads=0), nm.NM_ERR_SHAPE), (dict(heads=1 << 25), nm.NM_ERR_SHAPE),
        (dict(tokens=1 << 40), nm.NM_ERR_SHAPE), (dict(tokens=(1 << 26) + 1, heads=1, width=64), nm.NM_ERR_SHAPE),
        (dict(x_stride=127), nm.NM_ERR_SHAPE), (dict(x=A + 1), nm.NM_ERR_ALIGN), (dict(x=A + 2, fp32_input=1), nm.NM_ERR_ALIGN)]] +
    [("nm_block_norm", BLOCK_NORM, kw, st) for kw, st in ROWS + [
        (dict(branch=None), nm.NM_ERR_NULL), (dict(rows=0), nm.NM_ERR_SHAPE), (dict(rows=(1 << 26) + 1), nm.NM_ERR_SHAPE),
        (dict(branch_stride=63), nm.NM_ERR_SHAPE), (dict(h_stride=63), nm.NM_ERR_SHAPE), (dict(gate_stride=63), nm.NM_ERR_SHAPE),
        (dict(scale=math.inf), nm.NM_ERR_SHAPE), (dict(x=A + 2), nm.NM_ERR_ALIGN), (dict(h=A + 2), nm.NM_ERR_ALIGN),
        (dict(post=A + 1), nm.NM_ERR_ALIGN), (dict(gate=A + 1), nm.NM_ERR_ALIGN), (dict(branch=A + 1), nm.NM_ERR_ALIGN)]] +
    [("nm_logprobs", LOGPROBS, kw, st) for kw, st in [
        (dict(logits=None), nm.NM_ERR_NULL), (dict(tokens=None), nm.NM_ERR_NULL), (dict(logprob=None), nm.NM_ERR_NULL),
        (dict(top_tokens=None), nm.NM_ERR_NULL), (dict(top_logprobs=None), nm.NM_ERR_NULL), (dict(rows=0), nm.NM_ERR_SHAPE),
        (dict(rows=(1 << 23) + 1), nm.NM_ERR_SHAPE), (dict(vocab=0), nm.NM_ERR_SHAPE),
        (dict(vocab=(1 << 24) + 1, stride=1 << 25), nm.NM_ERR_SHAPE), (dict(stride=99), nm.NM_ERR_SHAPE),
        (dict(stride=1 << 41), nm.NM_ERR_SHAPE), (dict(top=65), nm.NM_ERR_SHAPE), (dict(top=-1), nm.NM_ERR_SHAPE),
        (dict(top=5, vocab=4), nm.NM_ERR_SHAPE), (dict(scale=0.0), nm.NM_ERR_SHAPE), (dict(scale=-1.0), nm.NM_ERR_SHAPE),
        (dict(scale=math.nan), nm.NM_ERR_SHAPE), (dict(scale=math.inf), nm.NM_ERR_SHAPE), (dict(logits=A + 1), nm.NM_ERR_ALIGN),
        (dict(logits=A + 2, fp16_logits=0), nm.NM_ERR_ALIGN), (dict(tokens=A + 2), nm.NM_ERR_ALIGN),
        (dict(workspace=A + 8, workspace_bytes=1 << 20), nm.NM_ERR_ALIGN), (dict(entropy=A + 2), nm.NM_ERR_ALIGN)]])


@pytest.mark.parametrize("name,given,kw,status", REFUSED, ids=lambda v: str(v) if isinstance(v, (str, int)) else None)
def test_refused_before_any_hip_call(name, given, kw, status):
    assert getattr(nm.lib(), name)(*{**given, **kw}.values()) == status


def test_workspaces_of_bad_sizes_are_none():
    lib = nm.lib()
    for args in ((0, 64, 4, 2, 4), (16, 48, 4, 2, 4), (16, 64, 0, 2, 4), (16, 64, 4, 3, 4), (1 << 30, 64, 4, 2, 4), (1 << 62, 64, 4, 2, 4)):
        assert lib.nm_gated_workspace_bytes(*args) == 0
    for args in ((0, 100), (4, 0), (1 << 24, 100), (4, 1 << 25)):
        assert lib.nm_logprobs_workspace_bytes(*args) == 0


def test_the_binding_wants_gpu_tensors():
    h = torch.zeros(4, 64, dtype=torch.float16)
    w = (torch.zeros(8, 32, dtype=torch.float16), torch.zeros(8, 2, dtype=torch.int32))
    for call in (lambda: nm.nm_linear(*w, h, 2, 4), lambda: nm.nm_gated(w, w, h, 2, 4), lambda: nm.nm_norm(h),
                 lambda: nm.nm_block_norm(h, h), lambda: nm.nm_logprobs(h)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        nm.nm_norm([1.0])


def test_names():
    with pytest.raises(ValueError, match="activation"):
        block._activation("tanh")
    with pytest.raises(ValueError, match="kind"):
        block._kind("batch")
    assert block._activation(None) == block._activation("none") == 0
    assert nm.status_string(nm.NM_ERR_FORMAT).count("nm_block.h")


def test_reference_activations():
    x = torch.linspace(-9, 9, 4001, dtype=torch.float64)
    assert torch.allclose(ref.act(x, "silu"), x / (1 + torch.exp(-x)), rtol=1e-14)
    assert torch.allclose(ref.act(x, "gelu"), 0.5 * x * (1 + torch.erf(x / math.sqrt(2))), atol=1e-15)
    u = math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
    assert torch.allclose(ref.act(x, "gelu_tanh"), 0.5 * x * (1 + torch.tanh(u)), atol=1e-14)
    for name in ref.EXPONENTS:      # the slope that the slack of the sums is multiplied with
        y = ref.act(x, name)
        assert ((y[1:] - y[:-1]).abs() / (x[1] - x[0])).max() < ref.SLOPE


def test_reference_scores():
    z = torch.tensor([[0.0, math.log(3.0), -math.inf], [-math.inf] * 3, [1.0, math.nan, 0.0], [math.inf, 0.0, 0.0]],
                     dtype=torch.float64)
    lp, entropy = ref.scores(z)
    assert torch.allclose(lp[0, :2], torch.tensor([math.log(0.25), math.log(0.75)], dtype=torch.float64))
    assert abs(entropy[0].item() - (0.25 * math.log(4) + 0.75 * math.log(4 / 3))) < 1e-12
    assert (lp[1] == -math.inf).all() and entropy[1] == 0 and lp[2:].isnan().all() and entropy[2:].isnan().all()
    x = torch.tensor([[1.0, 3.0, 3.0, -math.inf, 2.0]])
    assert ref.best(x, 5).tolist() == [[1, 2, 4, 0, -1]]
