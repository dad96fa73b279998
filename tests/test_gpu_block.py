"""GPU tests of the block operators (nm_linear, nm_gated, nm_norm, nm_block_norm, nm_logprobs) against
their definitions in 64 bits, with the distances that fp32 arithmetic and one rounding allow
(block_bounds.py)."""
import itertools
import math

import pytest
import torch

import semi_structured_sparse_amd as nm
from tests import block_bounds as ref
from tests.gpu_helpers import device, say

pytestmark = pytest.mark.gpu


def generator(*seed):
    return torch.Generator(device=device()).manual_seed(hash(seed) & 0x7FFFFFFF)


def normal(gen, *shape, spread=1.0, dtype=torch.float16):
    return (torch.randn(shape, generator=gen, device=gen.device) * spread).to(dtype)


def packed(gen, rows, cols, N, M):
    """((values, masks), the pruned matrix in 64 bits)."""
    w = nm.nm_pack(normal(gen, rows, cols, spread=cols ** -0.5), N, M)
    return w, nm.nm_unpack(*w, N, M).double()


def wide(t):
    return None if t is None else t.double()


def near(got, want, slack, what):
    off = (got.double() - want).abs()
    worst = (off / slack.clamp(min=1e-300)).max().item()
    assert torch.isfinite(got).all() and worst <= 1.0, f"{what}: {worst:.3g} of the allowed distance"


# --------------------------------------------------------------------------- the products
# batches on each side of every change of route: one vector, the small-batch kernels, the 16-vector
# launches and their rests, the column splits and the prompt kernels
BATCHES = [1, 2, 3, 4, 5, 8, 9, 16, 17, 21, 32, 33, 49, 65, 130, 200]
SHAPES = [(37, 96), (64, 256), (300, 1056), (1000, 4096), (2056, 512), (4104, 2080)]
EVERY = [(p, b, s) for p in nm.PATTERNS for b, s in itertools.product(BATCHES, SHAPES) if b * s[0] * s[1] <= 3e8]
# two long matrices of few rows, whose columns are split from 9 (16:32: 12) vectors on; X in several phases;
# 16:32 on many rows, from 6 vectors on the matrix instructions and from 17, 24 or 33 on the prompt kernels
EVERY += [(p, b, s) for p in nm.PATTERNS for b, s in itertools.product([9, 12, 16], [(300, 8192), (2048, 8224), (40, 14368)])]
EVERY += [((16, 32), b, (8200, 160)) for b in (5, 6, 7, 12, 14, 16, 17, 23, 24, 33, 40)]


@pytest.mark.parametrize("pattern,batch,shape", EVERY, ids=str)
def test_products(pattern, batch, shape):
    """Both products at every route, with and without a workspace; the options turn with the case."""
    (N, M), (rows, cols) = pattern, shape
    gen = generator(N, batch, rows)
    k = batch + rows + N
    name = list(ref.EXPONENTS)[k % 6]
    X = normal(gen, batch, cols)
    a, wa = packed(gen, rows, cols, N, M)
    b, wb = packed(gen, rows, cols, N, M)
    bias, other = normal(gen, rows), normal(gen, rows)
    residual = normal(gen, batch, rows) if k % 3 else None
    if k % 2:
        bias = None
    scale = 1.0 if k % 5 else -0.375
    say(f"linear and gated {N}:{M} {rows}x{cols} batch {batch} {name}")
    want, slack = ref.linear(X.double(), wa, wide(bias), name, scale, wide(residual))
    gwant, gslack = ref.gated(X.double(), wa, wb, wide(bias), wide(other), name)
    for ws, gws in ((None, None), (nm.linear_workspace(rows, cols, batch, N, M), nm.gated_workspace(rows, cols, batch, N, M))):
        y = nm.nm_linear(*a, X, N, M, bias=bias, activation=name, scale=scale, residual=residual, workspace=ws)
        near(y, want, slack, "linear")
        y = nm.nm_gated(a, b, X, N, M, activation=name, gate_bias=bias, up_bias=other, workspace=gws)
        near(y, gwant, gslack, "gated")
        for w in (ws, gws):
            if w is not None:
                assert not w[:1024].any(), "the counters are left at zero"


@pytest.mark.parametrize("pattern", nm.ALL_PATTERNS, ids=str)
@pytest.mark.parametrize("rows,cols", [(1, 32), (5, 64), (37, 288), (520, 4096), (3000, 1120), (40, 9248)])
def test_one_vector(pattern, rows, cols):
    """A vector without a batch dimension, the 25% patterns among them."""
    N, M = pattern
    gen = generator(N, M, rows)
    x = normal(gen, cols)
    a, wa = packed(gen, rows, cols, N, M)
    b, wb = packed(gen, rows, cols, N, M)
    bias, other, residual = normal(gen, rows), normal(gen, rows), normal(gen, rows)
    y = nm.nm_linear(*a, x, N, M, bias=bias, activation="gelu", scale=0.5, residual=residual)
    assert y.shape == (rows,)
    want, slack = ref.linear(x.double()[None], wa, wide(bias), "gelu", 0.5, wide(residual))
    near(y, want[0], slack[0], "linear")
    y = nm.nm_gated(a, b, x, N, M, activation="gelu_tanh", gate_bias=bias, up_bias=other)
    want, slack = ref.gated(x.double()[None], wa, wb, wide(bias), wide(other), "gelu_tanh")
    near(y, want[0], slack[0], "gated")


@pytest.mark.parametrize("pattern", nm.PATTERNS, ids=str)
@pytest.mark.parametrize("batch", [1, 3])
def test_rows_wider_than_one_workgroup_holds(pattern, batch):
    """Columns past what the single-vector kernel stages go through the small-batch kernel in phases."""
    N, M = pattern
    gen = generator(N, batch)
    rows, cols = 24, nm.max_cols() // 32 * 32 + 640
    X = normal(gen, batch, cols)
    a, wa = packed(gen, rows, cols, N, M)
    b, wb = packed(gen, rows, cols, N, M)
    residual = normal(gen, batch, rows)
    near(nm.nm_linear(*a, X, N, M, activation="silu", residual=residual),
         *ref.linear(X.double(), wa, None, "silu", 1.0, residual.double()), "linear")
    near(nm.nm_gated(a, b, X, N, M), *ref.gated(X.double(), wa, wb, None, None, "silu"), "gated")


@pytest.mark.parametrize("pattern", nm.PATTERNS, ids=str)
@pytest.mark.parametrize("batch", [1, 2, 6, 12, 24, 40, 150])
@pytest.mark.parametrize("rows,cols", [(72, 512), (1024, 8192), (90, 1024)])
def test_no_end_is_the_plain_product(pattern, batch, rows, cols):
    """Without bias, activation, scale and residual the linear product is nm_spmm_ws's, bit for bit where
    16 vectors or fewer fit 128 KiB. More go through LDS in phases, whose widths are the plain product's
    own: sums of the same products in another order."""
    N, M = pattern
    gen = generator(N, batch, rows)
    X = normal(gen, batch, cols)
    a, wa = packed(gen, rows, cols, N, M)
    for ws, plain in ((nm.linear_workspace(rows, cols, batch, N, M), nm.nm_spmm_ws), (None, nm.nm_spmm)):
        y = nm.nm_linear(*a, X, N, M, workspace=ws)
        if 2 * min(batch, 16) * cols <= 1 << 17:
            more = {} if ws is None else {"workspace": ws}
            assert torch.equal(y, plain(*a, X, N, M, **more))
        else:
            near(y, *ref.linear(X.double(), wa, None, None, 1.0, None), "linear")


@pytest.mark.parametrize("batch", [1, 3, 10, 24, 200])
@pytest.mark.parametrize("rows", [64, 83])
def test_the_residual_may_be_the_result(batch, rows):
    gen = generator(batch, rows)
    X = normal(gen, batch, 1024)
    a, _ = packed(gen, rows, 1024, 2, 4)
    residual = normal(gen, batch, rows)
    want = nm.nm_linear(*a, X, 2, 4, activation="relu", residual=residual)
    got = nm.nm_linear(*a, X, 2, 4, activation="relu", residual=residual, out=residual)
    assert got is residual and torch.equal(got, want)


@pytest.mark.parametrize("batch", [1, 4, 9, 40, 140])
def test_arrays_of_any_alignment(batch):
    """Rows a multiple of 8 with a result, biases and a residual that start 2 bytes past a 16-byte
    boundary are read and written one by one."""
    gen = generator(batch)
    rows, cols = 136, 512
    X = normal(gen, batch, cols)
    a, wa = packed(gen, rows, cols, 2, 4)
    b, wb = packed(gen, rows, cols, 2, 4)

    def odd(*shape):
        n = math.prod(shape)
        return torch.zeros(n + 9, dtype=torch.float16, device=device())[1:n + 1].view(shape)

    bias, residual, out = odd(rows).copy_(normal(gen, rows)), odd(batch, rows).copy_(normal(gen, batch, rows)), odd(batch, rows)
    assert bias.data_ptr() % 16 == 2 and out.data_ptr() % 16 == 2
    near(nm.nm_linear(*a, X, 2, 4, bias=bias, residual=residual, out=out),
         *ref.linear(X.double(), wa, bias.double(), None, 1.0, residual.double()), "linear")
    near(nm.nm_gated(a, b, X, 2, 4, up_bias=bias, out=out), *ref.gated(X.double(), wa, wb, None, bias.double(), "silu"), "gated")


@pytest.mark.parametrize("batch", [1, 4, 12, 30, 150])
def test_what_lies_behind_the_result_stays(batch):
    """Nothing is written past the last row of the last vector."""
    gen = generator(batch)
    rows, cols = 90, 512
    X = normal(gen, batch, cols)
    a, _ = packed(gen, rows, cols, 4, 8)
    room = torch.full((batch * rows + 512,), 7.0, dtype=torch.float16, device=device())
    nm.nm_linear(*a, X, 4, 8, out=room[:batch * rows].view(batch, rows))
    nm.nm_gated(a, a, X, 4, 8, out=room[:batch * rows].view(batch, rows))
    assert (room[batch * rows:] == 7.0).all()


@pytest.mark.parametrize("batch", [1, 4, 12, 30, 150])
def test_values_at_the_ends_of_the_range(batch):
    """Large sums: the logistic forms' limits, fp16's infinity where the result is past it, NaN of a NaN."""
    rows, cols = 64, 512
    w = torch.zeros(rows, cols, dtype=torch.float16, device=device())
    w[:, 0] = 1.0
    a = nm.nm_pack(w, 2, 4)
    X = torch.zeros(batch, cols, dtype=torch.float16, device=device())
    X[:, 0] = torch.tensor([60000.0, -60000.0, 1000.0, -1000.0, 0.0], device=device())[torch.arange(batch) % 5].half()
    up = X[:, :1].expand(batch, rows)
    for name in ("silu", "gelu", "gelu_tanh"):
        y = nm.nm_linear(*a, X, 2, 4, activation=name)
        assert torch.equal(y, up.clamp(min=0)), name            # the far sides are x and 0
    assert torch.equal(nm.nm_linear(*a, X, 2, 4, scale=4.0), (up.float() * 4.0).half())
    assert torch.equal(nm.nm_gated(a, a, X, 2, 4, activation="relu"), (up.clamp(min=0).float() * up.float()).half())
    X[0, 0] = math.nan
    for name in (None, "relu", "silu", "gelu", "gelu_tanh"):
        y = nm.nm_linear(*a, X, 2, 4, activation=name)
        assert y[0].isnan().all() and not y[1:].isnan().any(), name


# ------------------------------------------------------------------------------ the norms
WIDTHS = [1, 2, 7, 8, 64, 80, 127, 128, 129, 500, 512, 513, 1024, 1100, 2048, 2050, 4096, 5120, 8192, 8200, 16384, 25600, 32768]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("rows", [1, 5, 67])
def test_norm(kind, width, rows):
    gen = generator(width, rows)
    for wide_x, (weight, bias, offset) in itertools.product((False, True), ((None, None, 0.0), (1, None, 1.0), (1, 1, 0.0))):
        x = normal(gen, rows, width + 3, spread=3.0, dtype=torch.float32 if wide_x else torch.float16)[:, 1:width + 1] + 0.5
        weight = normal(gen, width) if weight is not None else None
        bias = normal(gen, width) if bias is not None else None
        y = nm.nm_norm(x, weight, bias, kind=kind, offset=offset, eps=1e-5)
        want, slack = ref.norm(x.double(), wide(weight), wide(bias), kind, offset, 1e-5)
        near(y, want, slack + ref.half_rounding(want), f"norm {kind} {rows}x{width}")


@pytest.mark.parametrize("shape,heads", [((7, 6, 128), 5), ((2, 9, 4, 64), 3), ((33, 3, 80), 3), ((3, 1, 10, 256), 8)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_of_heads_in_place(shape, heads, kind):
    """Heads of a fused projection's output, normalised where they are; the others stay."""
    gen = generator(*shape)
    fused = normal(gen, *shape)
    before = fused.clone()
    q = fused[..., :heads, :]
    weight = normal(gen, shape[-1])
    want, slack = ref.norm(q.double(), weight.double(), None, kind, 0.0, 1e-6)
    out = nm.nm_norm(q, weight, kind=kind)
    assert nm.nm_norm(q, weight, kind=kind, out=q) is q
    near(q, want, slack + ref.half_rounding(want), "heads")
    assert torch.equal(out, q) and torch.equal(fused[..., heads:, :], before[..., heads:, :])


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("width", [3, 96, 500, 1000, 2048, 4100, 8192, 10000, 32768])
@pytest.mark.parametrize("stream", [torch.float16, torch.float32])
def test_block_norm(kind, width, stream):
    gen = generator(width)
    rows = 6
    for post, gate, given in itertools.product((None, 1), (None, 1, 2), (False, True)):
        x = normal(gen, rows, width, spread=2.0, dtype=stream)
        branch = normal(gen, rows, width + 5)[:, 2:width + 2]
        weight, bias = normal(gen, width), normal(gen, width)
        post = normal(gen, width) if post is not None else None
        gate = None if gate is None else normal(gen, width) if gate == 1 else normal(gen, rows, width)
        (want, slack), (hw, hs) = ref.block_norm(x.double(), branch.double(), weight.double(), bias.double(), wide(post),
                                                 wide(gate), 0.7, kind, 1.0, 1e-5)
        scale = torch.tensor(0.7, dtype=torch.float32).item()    # what the kernel is given
        (want, slack), (hw, hs) = ref.block_norm(x.double(), branch.double(), weight.double(), bias.double(), wide(post),
                                                 wide(gate), scale, kind, 1.0, 1e-5)
        more = dict(h=x, out=branch) if given else {}            # in place, or made
        y, h = nm.nm_block_norm(x, branch, weight, bias, post=post, gate=gate, scale=0.7, kind=kind, offset=1.0, eps=1e-5, **more)
        near(y, want, slack + ref.half_rounding(want), f"y {post is None} {gate is None}")
        rounding = ref.half_rounding(hw) if stream == torch.float16 else ref.U * hw.abs() + 1e-45
        near(h, hw, hs + rounding, "h")
        assert h.dtype == stream and (not given or (h is x and y is branch))


def test_norm_of_what_is_not_finite():
    """A NaN or an infinity stays with its row; zeros are zeros, with an eps of 0 they are not."""
    x = normal(generator(3), 6, 700)
    x[1, 5], x[2, 699], x[3] = math.nan, math.inf, 0.0
    y = nm.nm_norm(x)
    assert y[1].isnan().all() and y[2, 699].isnan() and (y[2, :699] == 0).all() and (y[3] == 0).all()
    assert torch.equal(y[[0, 4, 5]], nm.nm_norm(x[[0, 4, 5]]))
    assert nm.nm_norm(x, eps=0.0)[3].isnan().all()


# ----------------------------------------------------------------------------- the scores
def check_scores(x, tokens, top, scale, got):
    """Log probabilities and entropies within fp32's reach of the definition; tokens exactly its own."""
    z = x.double() * scale
    lp, entropy = ref.scores(z)
    n = x.shape[1]
    m = torch.where(z.isfinite(), z, torch.full_like(z, -math.inf)).amax(-1)
    bad = entropy.isnan()
    # log p = scale (x - M) - log1p(S): two roundings of the difference, a sum of n terms each of which
    # exp moves by its argument's rounding (2 |d| U, weighed with its share) and 4 U, log1p and the last
    # subtraction; sums run over 64 lanes and their tiles, so that n / 64 + 64 additions follow one another
    run = n / 64 + 64
    p = lp.exp()
    d = torch.where(p > 0, (m[:, None] - z), torch.zeros_like(z))
    mean_d = (p * d).sum(-1)
    sum_slack = (run + 4.0) * ref.U + 2.0 * ref.U * mean_d
    log1p = torch.where(bad, torch.zeros_like(m), (-lp.gather(1, z.argmax(-1, keepdim=True)).squeeze(1)))
    share = -torch.expm1(-log1p.clamp(min=0))          # S / (1 + S): what S's slack does to log1p
    common = sum_slack * share + 4.0 * ref.U * log1p.abs()

    def allowed(value, dist):
        return 1.01 * (common + 4.0 * ref.U * dist + 4.0 * ref.U * value.abs()) + 1e-37

    def compare(a, b, slack, what):
        same = (a.double() == b) | (a.isnan() & b.isnan())
        share = torch.where(same, torch.zeros_like(b), (a.double() - b).abs() / slack)
        worst = share.max().item() if share.numel() else 0.0
        assert worst <= 1.0, f"{what}: {worst:.3g} of the allowed distance"

    if tokens is not None:
        at = tokens.long()
        ok = (at >= 0) & (at < n)
        want = lp.gather(1, at.clamp(0, n - 1)[:, None]).squeeze(1)
        dist = (m - z.gather(1, at.clamp(0, n - 1)[:, None]).squeeze(1)).nan_to_num(0.0, 0.0, 0.0).abs()
        want = torch.where(at < 0, torch.zeros_like(want), torch.where(ok, want, torch.full_like(want, math.nan)))
        compare(got.logprob, want, allowed(want.nan_to_num(0.0, 0.0, 0.0), dist), "logprob")
    # entropy = log1p(S) + T / (1 + S): T's terms move as S's, by another d of theirs
    mean_d2 = (p * d * d).sum(-1)
    slack = common + sum_slack * mean_d * 2.0 + 2.0 * ref.U * mean_d2 + 8.0 * ref.U * entropy.abs().nan_to_num(0.0)
    compare(got.entropy, entropy, 1.01 * slack + 1e-37, "entropy")
    if top:
        want = ref.best(x, top)
        want = torch.where(bad[:, None], torch.full_like(want, -1), want)
        assert torch.equal(got.top_tokens.long(), want)
        values = lp.gather(1, want.clamp(min=0))
        values = torch.where(bad[:, None], torch.full_like(values, math.nan),
                             torch.where(want < 0, torch.full_like(values, -math.inf), values))
        dist = (m[:, None] - z.gather(1, want.clamp(min=0))).nan_to_num(0.0, 0.0, 0.0).abs()
        slack = 1.01 * (common[:, None] + 4.0 * ref.U * dist + 4.0 * ref.U * values.abs().nan_to_num(0.0, 0.0, 0.0)) + 1e-37
        compare(got.top_logprobs, values, slack, "top_logprobs")
    else:
        assert got.top_tokens is None and got.top_logprobs is None


def score(x, tokens, top, scale=1.0):
    """With and without a workspace; the counters are left at zero."""
    ws = nm.logprobs_workspace(*x.shape)
    for w in (None, ws, ws):
        got = nm.nm_logprobs(x, tokens, top=top, scale=scale, workspace=w)
        check_scores(x, tokens, top, scale, got)
        assert w is None or not w[:65536].any()
    return got


@pytest.mark.parametrize("type_", [torch.float16, torch.float32])
@pytest.mark.parametrize("vocab", [1, 2, 63, 65, 300, 1000, 4096, 4099, 32000, 50257, 151936])
@pytest.mark.parametrize("rows", [1, 3, 33])
def test_scores(type_, vocab, rows):
    gen = generator(vocab, rows)
    for top, scale in ((0, 1.0), (1, 1.25), (5, 0.5), (20, 1.0), (64, 2.0)):
        top = min(top, vocab)
        x = normal(gen, rows, vocab + 1, spread=3.0, dtype=type_)[:, 1:]     # rows at odd elements
        tokens = torch.randint(-1, vocab, (rows,), generator=gen, device=device()).to(torch.int32)
        say(f"scores {rows}x{vocab} {type_} top {top}")
        score(x, tokens, top, scale)


@pytest.mark.parametrize("type_", [torch.float16, torch.float32])
@pytest.mark.parametrize("vocab", [40, 3000, 70000])
def test_scores_of_masked_and_equal_logits(type_, vocab):
    """Rows with nothing left, a single token, all equal, the type's lowest value in most places, rising
    and falling ones, the best of a row in one lane's places, NaN and infinities."""
    gen = generator(vocab)
    top = 20
    x = normal(gen, 14, vocab, spread=2.0, dtype=type_)
    low = torch.finfo(type_).min
    x[0] = -math.inf
    x[1] = -math.inf
    x[1, vocab // 2] = 1.0
    x[2] = 0.25
    x[3] = low
    x[4] = low
    x[4, [1, vocab - 1, 7]] = torch.tensor([2.0, 2.0, 3.0], device=device()).to(type_)
    x[5] = torch.linspace(-8, 8, vocab, device=device()).to(type_)
    x[6] = x[5].flip(0)
    x[7] = 0.0
    x[7, ::3] = -0.0
    x[8, 3] = math.nan
    x[9, vocab - 1] = math.inf
    x[10] = -math.inf
    x[10, :: max(1, vocab // 10)] = 0.5
    x[11, : vocab // 2] = -math.inf
    x[12] = low
    x[12, 8 * torch.arange(5, device=device())] = 0.0
    lanes = torch.arange(vocab, device=device())
    x[13] = torch.where(lanes % 2048 < 64, x[13].abs() + 5.0, x[13])          # a few lanes hold all of the best
    tokens = torch.full((14,), vocab // 2, dtype=torch.int32, device=device())
    tokens[13] = vocab                                                         # past the vocabulary
    score(x, tokens, top)
    score(x, tokens, min(64, vocab))
    score(x, None, 0)


def test_a_nearly_certain_token_keeps_its_digits():
    """log p of 2^-30 and less below 0 is what the others' sum says, not 0."""
    x = torch.full((4, 50000), -60.0, device=device())
    x[:, 777] = torch.tensor([-10.0, -8.0, 0.0, 20.0], device=device())
    got = score(x, torch.full((4,), 777, dtype=torch.int32, device=device()), 1)
    others = 49999 * torch.exp(-60.0 - x[:, 777].double())
    assert (got.logprob.double() / -torch.log1p(others) - 1.0).abs().max() < 1e-5
    assert (got.entropy > 0).all() and (got.logprob < 0).all()


@pytest.mark.parametrize("rows", [600, 4000])
def test_many_rows(rows):
    gen = generator(rows)
    x = normal(gen, rows, 2500, spread=2.0)
    tokens = torch.randint(0, 2500, (rows,), generator=gen, device=device()).to(torch.int32)
    score(x, tokens, 5)


class _Counts:
    """Stands before the extension and counts the calls that it takes and leaves."""

    def __init__(self, quick):
        self.quick, self.took, self.left = quick, [], []

    def __getattr__(self, name):
        def call(*args):
            done = getattr(self.quick, name)(*args)
            (self.left if done is NotImplemented else self.took).append(name)
            return done
        return call


def test_both_ways_to_the_library(monkeypatch):
    """The extension and block.py's own checks make the same calls."""
    from semi_structured_sparse_amd import block, decode

    def calls():
        gen = generator(1)
        w, _ = packed(gen, 96, 512, 2, 4)
        X, bias, residual = normal(gen, 30, 512), normal(gen, 96), normal(gen, 30, 96)
        ws, gws = nm.linear_workspace(96, 512, 30, 2, 4), nm.gated_workspace(96, 512, 30, 2, 4)
        made = [nm.nm_linear(*w, X, 2, 4, bias, "gelu", 0.5, residual, ws), nm.nm_linear(*w, X[3], 2, 4),
                nm.nm_gated(w, w, X, 2, 4, "relu", bias, None, gws), nm.nm_gated(w, w, X[1], 2, 4)]
        fused = normal(gen, 7, 5, 64)
        made += [nm.nm_norm(fused[:, :3], bias[:64].contiguous(), kind="layer"), nm.nm_norm(X[0]),
                 nm.nm_norm(fused.view(7, 1, 5, 64)[:, :, 1:3], out=torch.empty(7, 1, 2, 64, dtype=torch.float16, device=device()))]
        stream = normal(gen, 30, 96, dtype=torch.float32)
        made += nm.nm_block_norm(stream, residual, bias, None, bias, bias, 0.5, "layer", 1.0)
        made += nm.nm_block_norm(residual, residual.clone(), gate=residual, out=torch.empty_like(residual))
        logits = normal(gen, 9, 5001)[:, :5000]
        tokens = torch.arange(9, dtype=torch.int32, device=device())
        made += [t for t in nm.nm_logprobs(logits, tokens, 5, 0.5, nm.logprobs_workspace(9, 5000))]
        made += [t for t in nm.nm_logprobs(logits.float()) if t is not None]
        return made

    counts = _Counts(decode._bound())
    monkeypatch.setattr(decode, "_quick", counts)
    quick = calls()
    assert not counts.left and set(counts.took) == set(decode._QUICK_BLOCK)
    monkeypatch.setattr(decode, "_quick", decode._Absent())
    for a, b in zip(quick, calls()):
        assert a.dtype == b.dtype and torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert block.MAX_TOP == 64
