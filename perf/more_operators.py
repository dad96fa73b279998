"""The operators around the sparse products of a transformer block, as they are measured.

A block on packed weights is norms, projections with their bias and residual, a gated
feed-forward, and after the last one the scores of its answers. Each case below is one of these:

  norm    the branch of a block scaled, gated and added to the residual stream, with the norm
          after the branch and the norm before the next block; or the norm of query/key heads
  linear  a packed product with bias, activation, scale and residual, for 1 .. thousands of tokens
  gated   act(X Wg'^T + bg) * (X Wu'^T + bu) of two packed matrices
  score   log probabilities of given tokens from logits, their entropy and the best alternatives

`run` computes them in their plain form, or with the package's kernels where `own` is true;
`exact` computes them once more in 64 bits, from their definitions.
"""
import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
EPS = 1e-5
ACTIVATIONS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


# ------------------------------------------------------------------------------ the cases
def listed():
    return [
        # the step of a few sequences: the attention's output joins the stream, the next norm follows
        {"name": "norm step", "op": "norm", "rows": 8, "width": 4096, "kind": "rms", "stream": "fp16",
         "branch": True, "post": False, "gate": "none", "scale": 1.0, "offset": 0.0, "bias": False},
        # query and key heads of a fused projection's output, each head normalised
        {"name": "norm heads", "op": "heads", "tokens": 2048, "heads": 40, "width": 48, "dim": 128, "kind": "rms"},
        # a long prompt with an fp32 stream, norms on both sides of the block, a gate per channel
        {"name": "norm prompt", "op": "norm", "rows": 8191, "width": 8192, "kind": "rms", "stream": "fp32",
         "branch": True, "post": True, "gate": "channel", "scale": 0.5, "offset": 1.0, "bias": False},
        # one sequence's token through the down projection, added to the residual stream
        {"name": "linear token", "op": "linear", "batch": 1, "rows": 4096, "cols": 14336, "n": 2, "m": 4,
         "activation": "none", "bias": False, "residual": True, "scale": 1.0},
        # a serving batch's fused q/k/v projection with its bias
        {"name": "linear batch", "op": "linear", "batch": 13, "rows": 7168, "cols": 5120, "n": 4, "m": 8,
         "activation": "none", "bias": True, "residual": False, "scale": 1.0},
        # a prompt through an ungated feed-forward's first layer
        {"name": "linear prompt", "op": "linear", "batch": 2047, "rows": 14336, "cols": 4096, "n": 2, "m": 4,
         "activation": "gelu_tanh", "bias": True, "residual": False, "scale": 1.0},
        # one sequence's token through the gated feed-forward
        {"name": "gated token", "op": "gated", "batch": 1, "rows": 14336, "cols": 4096, "n": 2, "m": 4,
         "activation": "silu", "bias": False},
        # the drafted tokens of a speculative step
        {"name": "gated batch", "op": "gated", "batch": 12, "rows": 17408, "cols": 5120, "n": 8, "m": 16,
         "activation": "silu", "bias": False},
        # a prompt of an uneven length
        {"name": "gated prompt", "op": "gated", "batch": 1000, "rows": 14336, "cols": 4096, "n": 2, "m": 4,
         "activation": "silu", "bias": False},
        # the answers of a decoding step, with five alternatives each
        {"name": "score step", "op": "score", "rows": 8, "vocab": 128256, "type": "fp32", "top": 5, "scale": 1.0},
        # a serving batch that asks for twenty alternatives, at a temperature
        {"name": "score batch", "op": "score", "rows": 64, "vocab": 151936, "type": "fp16", "top": 20, "scale": 1.25},
        # the perplexity of a text
        {"name": "score text", "op": "score", "rows": 2047, "vocab": 128256, "type": "fp16", "top": 0, "scale": 1.0},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "heads", "linear", "linear", "gated", "gated", "score"])
    if op == "norm":
        width = rng.choice([_spread(rng, 64, 16384), 128 * rng.randint(1, 64)])
        rows = min(_spread(rng, 1, 8191), max(1, 8191 * 8192 // width))
        branch = rng.random() < 0.7
        return {"op": op, "rows": rows, "width": width, "kind": rng.choice(["rms", "rms", "layer"]),
                "stream": rng.choice(["fp16", "fp32"]), "branch": branch, "post": branch and rng.random() < 0.5,
                "gate": rng.choice(["none", "channel", "row"]) if branch else "none",
                "scale": rng.choice([1.0, 0.5, 0.22]) if branch else 1.0, "offset": rng.choice([0.0, 1.0]),
                "bias": rng.random() < 0.3}
    if op == "heads":
        heads, dim = rng.choice([5, 8, 10, 32, 40, 64]), rng.choice([64, 128, 128, 256, 80])
        return {"op": op, "tokens": min(_spread(rng, 1, 8191), 8191 * 8192 // (heads * dim)), "heads": heads,
                "width": heads + rng.choice([0, 1, 8]), "dim": dim, "kind": rng.choice(["rms", "rms", "layer"])}
    if op == "score":
        vocab = _spread(rng, 300, 151936)
        rows = min(_spread(rng, 1, 2047), 2047 * 128256 // (vocab * 2))
        return {"op": op, "rows": rows, "vocab": vocab, "type": rng.choice(["fp16", "fp32"]),
                "top": rng.choice([0, 1, 5, 20, 64]), "scale": rng.choice([1.0, 1.25, 0.5])}
    n = rng.choice([2, 2, 4, 8, 16])
    batch = rng.choice([1, _spread(rng, 1, 16), _spread(rng, 17, 2047)])
    rows = rng.choice([_spread(rng, 64, 17408), 64 * rng.randint(4, 224)])
    cols = 32 * rng.choice([_spread(rng, 8, 448), 16 * rng.randint(2, 28)])
    m = 2 * n
    if batch == 1 and rng.random() < 0.3:
        n, m = rng.choice([(1, 4), (2, 8), (4, 16), (8, 32)])
    most = 2047 * 14336 * 4096 // ((1 if m == 4 and n == 2 else 2) * (2 if op == "gated" else 1) * 2)
    batch = max(1, min(batch, most // (rows * cols)))
    case = {"op": op, "batch": batch, "rows": rows, "cols": cols, "n": n, "m": m, "bias": rng.random() < 0.5}
    if op == "gated":
        return {**case, "activation": rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"])}
    return {**case, "activation": rng.choice(ACTIVATIONS), "residual": rng.random() < 0.6,
            "scale": rng.choice([1.0, 0.5])}


def _packed_bytes(case):
    return case["rows"] * case["cols"] * case["n"] // case["m"] * 2 + case["rows"] * case["cols"] // 8


def work(case):
    if case["op"] == "heads":
        n = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": 4 * n + 2 * case["dim"], "flops": 4 * n}
    if case["op"] == "norm":
        n = case["rows"] * case["width"]
        wide = 4 if case["stream"] == "fp32" else 2
        each = 2 + wide
        if case["branch"]:
            each += 2 + wide + (2 if case["gate"] == "row" else 0)
        return {"bytes": each * n + 2 * case["width"], "flops": (4 + 3 * case["branch"] + 4 * case["post"]) * n}
    if case["op"] == "score":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (2 if case["type"] == "fp16" else 4) + case["rows"] * (12 + 8 * case["top"]), "flops": 5 * n}
    kept = case["rows"] * case["cols"] * case["n"] // case["m"]
    ends = case["batch"] * (case["cols"] + case["rows"]) * 2
    if case["op"] == "gated":
        return {"bytes": 2 * _packed_bytes(case) + ends + 4 * case["rows"] * case["bias"],
                "flops": 4 * case["batch"] * kept}
    ends += 2 * case["rows"] * case["bias"] + 2 * case["batch"] * case["rows"] * case["residual"]
    return {"bytes": _packed_bytes(case) + ends, "flops": 2 * case["batch"] * kept}


# ----------------------------------------------------------------------------- the inputs
def _packed(case, gen):
    """A pruned weight: (values fp16 [rows, cols n/m] in row order, masks int32 [rows, cols/32])."""
    rows, cols, n, m = case["rows"], case["cols"], case["n"], case["m"]
    w = (torch.randn((rows, cols), generator=gen, device=DEVICE) / math.sqrt(cols)).to(torch.float16)
    groups = w.view(-1, m)
    best = groups.abs().float().sort(dim=-1, descending=True, stable=True).indices[:, :n]
    bits = torch.zeros(groups.shape, dtype=torch.bool, device=DEVICE).scatter_(1, best, True)
    values = groups[bits].view(rows, cols * n // m)
    at = torch.arange(32, device=DEVICE)
    masks = (bits.view(rows, cols // 32, 32).long() << at).sum(-1)
    return values.contiguous(), masks.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    s = {"case": case}

    def normal(*shape, spread=1.0, dtype=torch.float16):
        return (torch.randn(shape, generator=gen, device=DEVICE) * spread).to(dtype)

    if case["op"] == "heads":
        fused = normal(case["tokens"], case["width"], case["dim"])
        s["x"] = fused[:, : case["heads"]]
        s["weight"] = (1.0 + normal(case["dim"], spread=0.1, dtype=torch.float32)).to(torch.float16)
        return s
    if case["op"] == "norm":
        rows, width = case["rows"], case["width"]
        wide = 1.0 + 9.0 * (torch.rand(width, generator=gen, device=DEVICE) < 0.01)      # a few wide channels
        s["x"] = (normal(rows, width, dtype=torch.float32) * wide).to(torch.float32 if case["stream"] == "fp32" else torch.float16)
        shift = 1.0 - case["offset"]
        s["weight"] = (shift + normal(width, spread=0.1, dtype=torch.float32)).to(torch.float16)
        s["bias"] = normal(width, spread=0.1) if case["bias"] else None
        s["branch"] = normal(rows, width, spread=0.5) if case["branch"] else None
        s["post"] = (shift + normal(width, spread=0.1, dtype=torch.float32)).to(torch.float16) if case["post"] else None
        s["gate"] = None
        if case["gate"] == "channel":
            s["gate"] = normal(width, spread=0.5)
        elif case["gate"] == "row":
            s["gate"] = normal(rows, width, spread=0.5)
        return s
    if case["op"] == "score":
        logits = normal(case["rows"], case["vocab"], spread=2.5, dtype=torch.float32)
        liked = torch.randint(0, case["vocab"], (case["rows"], 4), generator=gen, device=DEVICE)
        logits.scatter_add_(1, liked, normal(case["rows"], 4, spread=4.0, dtype=torch.float32) + 8.0)
        barred = torch.randint(0, case["vocab"], (case["vocab"] // 64,), generator=gen, device=DEVICE)
        logits[:, barred] = -math.inf                                    # tokens that a grammar forbids
        s["logits"] = logits.to(torch.float16 if case["type"] == "fp16" else torch.float32)
        s["tokens"] = liked[:, 0].to(torch.int32)
        return s
    X = normal(case["batch"], case["cols"])
    s["x"] = X[0] if case["batch"] == 1 else X
    if case["op"] == "linear":
        s["w"] = _packed(case, gen)
        s["bias"] = normal(case["rows"], spread=0.2) if case["bias"] else None
        shape = s["x"].shape[:-1] + (case["rows"],)
        s["residual"] = normal(*shape) if case["residual"] else None
        return s
    s["gate"], s["up"] = _packed(case, gen), _packed(case, gen)
    s["gate_bias"], s["up_bias"] = (normal(case["rows"], spread=0.2) if case["bias"] else None for _ in range(2))
    return s


# ------------------------------------------------------------------------ the plain forms
def _act(x, name):
    if name == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if name == "silu":
        return x / (1.0 + torch.exp(-x))
    if name == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))
    return x


def _dense(packed):
    """The fp32 matrix that values and masks stand for: a bit's rank in its row finds its value."""
    values, masks = packed
    at = torch.arange(32, dtype=torch.int32, device=masks.device)
    bits = ((masks[..., None] >> at) & 1).view(masks.shape[0], -1)
    rank = (bits.cumsum(-1, dtype=torch.int32) - 1).clamp(min=0).long()
    return torch.where(bits.bool(), values.gather(1, rank).float(), torch.zeros((), device=masks.device))


def _product(x, packed, bias):
    y = torch.matmul(x.float(), _dense(packed).t())
    return y if bias is None else y + bias.float()


def _plain_norm(x, weight, bias, kind, offset):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * (offset + weight.float())
    return y if bias is None else y + bias.float()


def _plain_score(s):
    case = s["case"]
    x = s["logits"].float()
    rows, vocab = x.shape
    top = x.amax(-1, keepdim=True)
    z = (x - top) * case["scale"]
    e = torch.exp(z)
    total = e.sum(-1, dtype=torch.float64)
    low = torch.where(e > 0, e * z, torch.zeros_like(e)).sum(-1, dtype=torch.float64)
    log_total = torch.log(total)
    given = z.gather(1, s["tokens"].long()[:, None]).squeeze(1).double() - log_total
    out = {"logprob": given.float(), "entropy": (log_total - low / total).float()}
    if case["top"]:
        # the order of the floats as whole numbers, then the lower index
        b = (x + 0.0).view(torch.int32).long()          # -0 as 0
        b = torch.where(b < 0, -(b + 2 ** 31) - 1, b)
        key = (b << 20) + (2 ** 20 - 1 - torch.arange(vocab, device=x.device))
        at = torch.topk(key, case["top"], dim=-1, sorted=True).indices
        best = z.gather(1, at).double() - log_total[:, None]
        out["top_tokens"] = torch.where(best > -math.inf, at, -1).to(torch.int32)
        out["top_logprobs"] = best.float()
    return out


# ---------------------------------------------------------------------------- the kernels
def _own(s):
    import semi_structured_sparse_amd as nm
    case = s["case"]
    if case["op"] == "heads":
        return nm.nm_norm(s["x"], s["weight"], kind=case["kind"], eps=EPS)
    if case["op"] == "norm":
        if not case["branch"]:
            return nm.nm_norm(s["x"], s["weight"], bias=s["bias"], kind=case["kind"], offset=case["offset"], eps=EPS)
        return nm.nm_block_norm(s["x"], s["branch"], s["weight"], bias=s["bias"], post=s["post"], gate=s["gate"],
                                scale=case["scale"], kind=case["kind"], offset=case["offset"], eps=EPS)
    if case["op"] == "score":
        return dict(nm.nm_logprobs(s["logits"], s["tokens"], top=case["top"], scale=case["scale"],
                                   workspace=_workspace(s, lambda: nm.logprobs_workspace(*s["logits"].shape, device=DEVICE)))._asdict())
    sizes = case["rows"], case["cols"], case["batch"], case["n"], case["m"]
    if case["op"] == "gated":
        return nm.nm_gated(s["gate"], s["up"], s["x"], case["n"], case["m"], activation=case["activation"],
                           gate_bias=s["gate_bias"], up_bias=s["up_bias"],
                           workspace=_workspace(s, lambda: nm.gated_workspace(*sizes, device=DEVICE)))
    return nm.nm_linear(*s["w"], s["x"], case["n"], case["m"], bias=s["bias"], activation=case["activation"],
                        scale=case["scale"], residual=s["residual"],
                        workspace=_workspace(s, lambda: nm.linear_workspace(*sizes, device=DEVICE)))


def _workspace(s, make):
    if "workspace" not in s:
        s["workspace"] = make()
    return s["workspace"]


def run(state):
    if own:
        return _own(state)
    s, case = state, state["case"]
    if case["op"] == "heads":
        return _plain_norm(s["x"].float(), s["weight"], None, case["kind"], 0.0).to(torch.float16)
    if case["op"] == "norm":
        h = s["x"].float()
        if case["branch"]:
            b = s["branch"].float()
            if case["post"]:
                b = _plain_norm(b, s["post"], None, case["kind"], case["offset"])
            if s["gate"] is not None:
                b = b * s["gate"].float()
            h = h + case["scale"] * b
        y = _plain_norm(h, s["weight"], s["bias"], case["kind"], case["offset"]).to(torch.float16)
        return (y, h.to(s["x"].dtype)) if case["branch"] else y
    if case["op"] == "score":
        return _plain_score(s)
    if case["op"] == "gated":
        g, u = _product(s["x"], s["gate"], s["gate_bias"]), _product(s["x"], s["up"], s["up_bias"])
        return (_act(g, case["activation"]) * u).to(torch.float16)
    y = case["scale"] * _act(_product(s["x"], s["w"], s["bias"]), case["activation"])
    return (y if s["residual"] is None else y + s["residual"].float()).to(torch.float16)


# ----------------------------------------------------------------- the definitions, 64 bits
def _act64(x, name):
    if name == "relu":
        return x.clamp(min=0)
    if name == "silu":
        return x * torch.special.expit(x)
    if name == "gelu":
        return x * torch.special.ndtr(x)
    if name == "gelu_tanh":     # (1 + tanh t) / 2 is the logistic function of 2 t
        return x * torch.special.expit(2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3))
    return x


def _dense64(packed):
    """Row by row, the kept values fill the set bits in order."""
    values, masks = packed
    at = torch.arange(32, device=masks.device)
    bits = ((masks.long()[..., None] >> at) & 1).bool().flatten(1)
    return torch.zeros(bits.shape, dtype=torch.float64, device=masks.device).masked_scatter_(bits, values.double())


def _product64(x, packed, bias):
    y = x.double() @ _dense64(packed).t()
    return y if bias is None else y + bias.double()


def _norm64(x, weight, bias, kind, offset):
    if kind == "layer":
        x = (x - x.mean(-1, keepdim=True)) / torch.sqrt(x.var(-1, keepdim=True, correction=0) + EPS)
    else:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    y = x * (offset + weight.double())
    return y if bias is None else y + bias.double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "heads":
        return _norm64(s["x"].double(), s["weight"], None, case["kind"], 0.0)
    if case["op"] == "norm":
        h = s["x"].double()
        if case["branch"]:
            b = s["branch"].double()
            if case["post"]:
                b = _norm64(b, s["post"], None, case["kind"], case["offset"])
            if s["gate"] is not None:
                b = b * s["gate"].double()
            h = h + case["scale"] * b
            return _norm64(h, s["weight"], s["bias"], case["kind"], case["offset"]), h
        return _norm64(h, s["weight"], s["bias"], case["kind"], case["offset"])
    if case["op"] == "score":
        out = {"logprob": [], "entropy": [], "top_logprobs": []}
        for i in range(0, case["rows"], 256):          # a part of the rows at a time
            z = s["logits"][i:i + 256].double() * case["scale"]
            lp = z - torch.logsumexp(z, -1, keepdim=True)
            out["logprob"].append(lp.gather(1, s["tokens"][i:i + 256].long()[:, None]).squeeze(1))
            out["entropy"].append(torch.special.entr(lp.exp()).sum(-1))
            if case["top"]:
                out["top_logprobs"].append(lp.sort(-1, descending=True).values[:, :case["top"]].contiguous())
            del z, lp
        out = {k: torch.cat(v) for k, v in out.items() if v}
        return {**out, "top_tokens": None} if case["top"] else out
    if case["op"] == "gated":
        g, u = _product64(s["x"], s["gate"], s["gate_bias"]), _product64(s["x"], s["up"], s["up_bias"])
        return _act64(g, case["activation"]) * u
    y = case["scale"] * _act64(_product64(s["x"], s["w"], s["bias"]), case["activation"])
    return y if s["residual"] is None else y + s["residual"].double()
