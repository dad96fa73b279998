"""GPU tests of the block operators as a program uses them: together, captured into graphs and replayed,
on other streams, with shared workspaces, far strides and optional arguments left out; and what their
binding refuses."""
import math

import pytest
import torch

import semi_structured_sparse_amd as nm
from tests import block_bounds as ref
from tests.gpu_helpers import device
from tests.test_gpu_block import generator, near, normal, packed, wide

pytestmark = pytest.mark.gpu
N, M = 2, 4


class Block:
    """A block's weights, and its step from the residual stream and the last branch on."""

    def __init__(self, gen, width=512, inner=1376, heads=8, vocab=1000):
        self.width, self.heads, self.dim = width, heads, width // heads
        self.qkv, self.qkv64 = packed(gen, 3 * width, width, N, M)
        self.out, self.out64 = packed(gen, width, width, N, M)
        self.gate, self.gate64 = packed(gen, inner, width, N, M)
        self.up, self.up64 = packed(gen, inner, width, N, M)
        self.down, self.down64 = packed(gen, width, inner, N, M)
        self.head = normal(gen, vocab, width, spread=width ** -0.5)
        self.norms = [normal(gen, width, spread=0.1) for _ in range(3)]
        self.head_norm = normal(gen, self.dim, spread=0.1)
        self.bias = normal(gen, 3 * width, spread=0.1)
        self.inner, self.vocab = inner, vocab

    def workspaces(self, batch):
        self.ws = {"qkv": nm.linear_workspace(3 * self.width, self.width, batch, N, M),
                   "out": nm.linear_workspace(self.width, self.width, batch, N, M),
                   "gated": nm.gated_workspace(self.inner, self.width, batch, N, M),
                   "down": nm.linear_workspace(self.width, self.inner, batch, N, M),
                   "score": nm.logprobs_workspace(batch, self.vocab)}

    def step(self, stream, branch, tokens):
        """Everything that the operators make, in order."""
        t = stream.shape[0]
        y, h = nm.nm_block_norm(stream, branch, self.norms[0], offset=1.0)
        qkv = nm.nm_linear(*self.qkv, y, N, M, bias=self.bias, workspace=self.ws["qkv"])
        heads = qkv.view(t, 3 * self.heads, self.dim)
        q = nm.nm_norm(heads[:, :2 * self.heads], self.head_norm, offset=1.0)
        mixed = (q[:, :self.heads] + heads[:, 2 * self.heads:]).reshape(t, self.width)     # in attention's place
        branch = nm.nm_linear(*self.out, mixed, N, M, workspace=self.ws["out"])
        y2, h2 = nm.nm_block_norm(h, branch, self.norms[1], post=self.norms[2], offset=1.0)
        g = nm.nm_gated(self.gate, self.up, y2, N, M, workspace=self.ws["gated"])
        last = nm.nm_linear(*self.down, g, N, M, residual=h2, workspace=self.ws["down"])
        y3 = nm.nm_norm(last, self.norms[0], offset=1.0)
        logits = nm.nm_gemm_dense(self.head, y3)
        scores = nm.nm_logprobs(logits, tokens, top=5, workspace=self.ws["score"])
        return [y, h, qkv, q, mixed, branch, y2, h2, g, last, y3, logits, *scores]

    def check(self, stream, branch, tokens, made):
        """Each result against its definition on the operands that the call had."""
        y, h, qkv, q, mixed, out, y2, h2, g, last, y3, logits, logprob, entropy, top_tokens, top_logprobs = made
        d = torch.double
        n0, n1, n2 = (w.to(d) for w in self.norms)

        def block(x, b, weight, post, got_y, got_h):
            (want, slack), (hw, hs) = ref.block_norm(x.to(d), b.to(d), weight, None, post, None, 1.0, "rms", 1.0, 1e-6)
            near(got_y, want, slack + ref.half_rounding(want), "y")
            near(got_h, hw, hs + ref.half_rounding(hw), "h")

        block(stream, branch, n0, None, y, h)
        near(qkv, *ref.linear(y.to(d), self.qkv64, self.bias.to(d), None, 1.0, None), "qkv")
        heads = qkv.view(len(y), 3 * self.heads, self.dim)[:, :2 * self.heads]
        want, slack = ref.norm(heads.to(d), self.head_norm.to(d), None, "rms", 1.0, 1e-6)
        near(q, want, slack + ref.half_rounding(want), "heads")
        near(out, *ref.linear(mixed.to(d), self.out64, None, None, 1.0, None), "out")
        block(h, out, n1, n2, y2, h2)
        near(g, *ref.gated(y2.to(d), self.gate64, self.up64, None, None, "silu"), "gated")
        near(last, *ref.linear(g.to(d), self.down64, None, None, 1.0, h2.to(d)), "down")
        lp, e = ref.scores(logits.to(d))
        assert (logprob - lp.gather(1, tokens.long()[:, None]).squeeze(1)).abs().max() < 2e-5
        assert (entropy - e).abs().max() < 2e-5
        assert torch.equal(top_tokens.long(), ref.best(logits, 5))
        assert (top_logprobs - lp.gather(1, top_tokens.long())).abs().max() < 2e-5


def inputs(gen, batch, width=512, vocab=1000):
    return (normal(gen, batch, width), normal(gen, batch, width),
            torch.randint(0, vocab, (batch,), generator=gen, device=device()).to(torch.int32))


@pytest.mark.parametrize("batch", [1, 3, 12, 24, 40, 300])
def test_a_block_of_them(batch):
    gen = generator(batch)
    block = Block(gen)
    block.workspaces(batch)
    given = inputs(gen, batch)
    block.check(*given, block.step(*given))


@pytest.mark.parametrize("batch", [1, 12, 24, 40])
def test_captured_and_replayed(batch):
    """Several replays with other inputs, with eager calls on the same workspaces and synchronisations
    between them: each gives what the eager calls give, to the bit."""
    gen = generator(batch, 1)
    block = Block(gen)
    block.workspaces(batch)
    held = inputs(gen, batch)
    block.step(*held)                                   # the first calls, outside the capture
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.step(*held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made = block.step(*held)
    for k in range(4):
        given = inputs(gen, batch)
        for to, t in zip(held, given):
            to.copy_(t)
        graph.replay()
        if k % 2:
            torch.cuda.synchronize()
        got = [t.clone() for t in made]
        want = block.step(*given)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    block.check(*given, got)


def test_two_graphs_share_workspaces():
    """Replayed in turn on one stream, each leaves the counters as the other needs them."""
    gen = generator(5)
    block = Block(gen)
    block.workspaces(40)
    graphs = []
    for batch in (40, 12):
        held = inputs(gen, batch)
        block.step(*held)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            made = block.step(*held)
        graphs.append((graph, held, made))
    for _ in range(3):
        for graph, held, made in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for graph, held, made in graphs:
        block.check(*held, made)


def test_on_another_stream():
    """A call's work goes to the current stream: behind a long product there, and before what follows."""
    gen = generator(6)
    block = Block(gen)
    block.workspaces(24)
    given = inputs(gen, 24)
    want = block.step(*given)
    slow = torch.randn(4096, 4096, device=device())
    side = torch.cuda.Stream()
    late = [torch.zeros_like(t) for t in given]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(10):
            slow = slow @ slow * 1e-3
        for to, t in zip(late, given):
            to.copy_(t)
        got = block.step(*late)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_the_same_bits_each_time():
    gen = generator(7)
    for batch in (1, 7, 16, 24, 33, 260):
        block = Block(gen)
        block.workspaces(batch)
        given = inputs(gen, batch)
        first = block.step(*given)
        for _ in range(3):
            for a, b in zip(block.step(*given), first):
                assert torch.equal(a, b)


def test_a_scores_workspace_serves_the_decoding_calls():
    """One workspace in stream order for nm_logprobs and nm_verify_chain: both find its counters at zero."""
    gen = generator(8)
    rows, vocab = 6, 20000
    room = torch.zeros(max(t.numel() for t in (nm.logprobs_workspace(rows, vocab), nm.verify_workspace(2, vocab))),
                       dtype=torch.uint8, device=device())
    x = normal(gen, rows, vocab, dtype=torch.float32)
    tokens = torch.zeros(rows, dtype=torch.int32, device=device())
    p = torch.softmax(x.view(2, 3, vocab), -1)
    chain = torch.randint(0, vocab, (2, 3), generator=gen, device=device()).to(torch.int32)
    u = torch.rand(2, 3, generator=gen, device=device())

    def calls(ws):
        return [*nm.nm_logprobs(x, tokens, 20, workspace=ws), *nm.nm_verify_chain(p, p[:, 1:].contiguous(), chain, u, workspace=ws)]

    apart = [*nm.nm_logprobs(x, tokens, 20, workspace=nm.logprobs_workspace(rows, vocab)),
             *nm.nm_verify_chain(p, p[:, 1:].contiguous(), chain, u, workspace=nm.verify_workspace(2, vocab))]
    for _ in range(3):
        for a, b in zip(calls(room), apart):
            assert torch.equal(a, b)
    few = nm.nm_logprobs(x[:2], tokens[:2], 20, workspace=room)      # fewer rows than it was made for
    near(few.entropy, ref.scores(x[:2].double())[1], torch.full((2,), 1e-4, dtype=torch.double, device=device()), "entropy")
    short = nm.nm_logprobs(x, tokens, 20, workspace=room[:4096])     # too little: not split
    assert torch.equal(short.top_tokens, apart[2])


def test_rows_more_than_four_billion_elements_apart():
    far = (1 << 32) + 8
    room = torch.empty(2 * far + 1024, dtype=torch.float16, device=device())
    x = room.as_strided((3, 700), (far, 1))
    gen = generator(9)
    x.copy_(normal(gen, 3, 700))
    tokens = torch.tensor([1, 2, 699], dtype=torch.int32, device=device())
    near_by = x.contiguous()
    got, want = nm.nm_logprobs(x, tokens, 5), nm.nm_logprobs(near_by, tokens, 5)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    y = nm.nm_norm(near_by)
    assert torch.equal(nm.nm_norm(x), y)
    assert nm.nm_norm(x, out=x) is x and torch.equal(x, y)
    del room


@pytest.mark.parametrize("batch", [17, 40, 400])
def test_a_result_past_two_to_the_31_bytes(batch):
    """Rows of Y and of the residual far from the first, in each family's own arithmetic."""
    rows = (1 << 31) // (2 * batch) // 64 * 64 + 128
    gen = generator(batch, 2)
    X = normal(gen, batch, 32)
    w, w64 = packed(gen, 64, 32, N, M)
    v, m = (t.repeat(rows // 64, 1) for t in w)
    residual = torch.zeros(batch, rows, dtype=torch.float16, device=device())
    residual[-1, -64:] = 1.0
    assert residual.numel() * 2 > 1 << 31
    y = nm.nm_linear(v, m, X, N, M, residual=residual)
    g = nm.nm_gated((v, m), (v, m), X, N, M, activation="relu") if 2 * rows < 1 << 26 else None
    for first in (0, rows // 128 * 64, rows - 64):
        part = slice(first, first + 64)
        near(y[:, part], *ref.linear(X.double(), w64, None, None, 1.0, residual[:, part].double()), f"linear {first}")
        if g is not None:
            near(g[:, part], *ref.gated(X.double(), w64, w64, None, None, "relu"), f"gated {first}")
    del v, m, residual, y, g


def test_what_may_be_left_out():
    """The C calls without optional outputs and inputs."""
    gen = generator(10)
    lib, stream = nm.lib(), torch.cuda.current_stream().cuda_stream
    x, b = normal(gen, 5, 300), normal(gen, 5, 300)
    y = torch.zeros_like(x)
    want, h = nm.nm_block_norm(x, b)
    before = x.clone()
    assert lib.nm_block_norm(x.data_ptr(), b.data_ptr(), None, y.data_ptr(), None, None, None, None, 5, 300, 300, 300, 0, 300, 0,
                             0, 0, 1.0, 0.0, 1e-6, stream) == 0
    assert torch.equal(y, want) and torch.equal(x, before)
    tokens = torch.arange(5, dtype=torch.int32, device=device())
    full = nm.nm_logprobs(x, tokens, 3)
    lp, e = (torch.zeros(5, device=device()) for _ in range(2))
    tt, tl = torch.zeros(5, 3, dtype=torch.int32, device=device()), torch.zeros(5, 3, device=device())
    assert lib.nm_logprobs(x.data_ptr(), tokens.data_ptr(), lp.data_ptr(), None, None, None, 5, 300, 300, 0, 1, 1.0, None, 0,
                           stream) == 0
    assert lib.nm_logprobs(x.data_ptr(), None, None, e.data_ptr(), None, None, 5, 300, 300, 0, 1, 1.0, None, 0, stream) == 0
    assert lib.nm_logprobs(x.data_ptr(), None, None, None, tt.data_ptr(), tl.data_ptr(), 5, 300, 300, 3, 1, 1.0, None, 0,
                           stream) == 0
    for a, c in zip((lp, e, tt, tl), full):
        assert torch.equal(a, c)


def test_vectors_and_rows_of_one_dimension():
    gen = generator(11)
    x, b, g = normal(gen, 700), normal(gen, 700), normal(gen, 700)
    assert torch.equal(nm.nm_norm(x, g), nm.nm_norm(x[None], g)[0])
    y, h = nm.nm_block_norm(x, b, g, gate=g)
    y2, h2 = nm.nm_block_norm(x[None], b[None], g, gate=g[None])
    assert y.shape == (700,) and torch.equal(y, y2[0]) and torch.equal(h, h2[0])


def test_refused_by_the_binding():
    gen = generator(12)
    w, _ = packed(gen, 64, 128, N, M)
    other, _ = packed(gen, 32, 128, N, M)
    X, bias, res = normal(gen, 3, 128), normal(gen, 64), normal(gen, 3, 64)
    ws = torch.zeros(4096, dtype=torch.uint8, device=device())
    stream, logits = normal(gen, 3, 128, dtype=torch.float32), normal(gen, 3, 100)
    tokens = torch.zeros(3, dtype=torch.int32, device=device())
    bad = [
        lambda: nm.nm_linear(*w, X.float(), N, M), lambda: nm.nm_linear(*w, X[:, :64], N, M), lambda: nm.nm_linear(*w, X.t(), N, M),
        lambda: nm.nm_linear(*w, X[None], N, M), lambda: nm.nm_linear(*w, X, 4, 16), lambda: nm.nm_linear(*w, X, N, M, bias=X[0]),
        lambda: nm.nm_linear(*w, X, N, M, bias=bias.float()), lambda: nm.nm_linear(*w, X, N, M, residual=res[:2]),
        lambda: nm.nm_linear(*w, X, N, M, residual=res.t().contiguous().t()), lambda: nm.nm_linear(*w, X, N, M, activation="tanh"),
        lambda: nm.nm_linear(*w, X, N, M, out=res[:2]), lambda: nm.nm_linear(*w, X, N, M, workspace=ws.view(2, 2048)),
        lambda: nm.nm_linear(*w, X, N, M, workspace=ws.int()), lambda: nm.nm_linear(*w, X, N, M, workspace=ws[4:]),
        lambda: nm.nm_linear(*w, X[:0], N, M), lambda: nm.nm_linear(w[0].cpu(), w[1], X, N, M),
        lambda: nm.nm_linear(*w, X, N, M, bias=bias.cpu()),
        lambda: nm.nm_gated(w, other, X, N, M), lambda: nm.nm_gated(w, w, X, N, M, activation="tanh"),
        lambda: nm.nm_gated(w, w, X, N, M, up_bias=X[0]), lambda: nm.nm_gated(w, w, X[:, :64].contiguous(), N, M),
        lambda: nm.nm_norm(X.t()), lambda: nm.nm_norm(X.int()), lambda: nm.nm_norm(X, bias), lambda: nm.nm_norm(X, kind="batch"),
        lambda: nm.nm_norm(X, eps=-1.0), lambda: nm.nm_norm(X, out=res), lambda: nm.nm_norm(X, out=stream),
        lambda: nm.nm_norm(X.expand(3, 3, 128)), lambda: nm.nm_norm(X[:0]), lambda: nm.nm_norm(X[0, 0]),
        lambda: nm.nm_block_norm(X, res), lambda: nm.nm_block_norm(stream, stream), lambda: nm.nm_block_norm(stream, X, h=X),
        lambda: nm.nm_block_norm(X, X, gate=X[:2]), lambda: nm.nm_block_norm(X, X, gate=X.float()),
        lambda: nm.nm_block_norm(X, X, post=bias), lambda: nm.nm_block_norm(X[None], X[None]),
        lambda: nm.nm_block_norm(X, X, scale=math.inf),
        lambda: nm.nm_logprobs(logits.int()), lambda: nm.nm_logprobs(logits[0]), lambda: nm.nm_logprobs(logits, tokens[:2]),
        lambda: nm.nm_logprobs(logits, tokens.long()), lambda: nm.nm_logprobs(logits, top=65), lambda: nm.nm_logprobs(logits, top=-1),
        lambda: nm.nm_logprobs(logits[:, :4], top=5), lambda: nm.nm_logprobs(logits, scale=0.0),
        lambda: nm.nm_logprobs(logits, workspace=ws[4:]), lambda: nm.nm_logprobs(logits.t()), lambda: nm.nm_logprobs(logits[:0]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    torch.cuda.synchronize()
    assert wide(None) is None and math.isfinite(nm.nm_linear(*w, X, N, M).float().sum().item())
