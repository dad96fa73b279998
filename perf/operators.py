"""The operators of a speculative decoding step, as they are measured.

Between the sparse products of a decoding step stand the rotary positions, the key/value
cache, the attention of the drafted tokens over it, and the verification of the drafts
against the target's probabilities. Each case below is one of these:

  rope    rotary positions on the query and key heads of a fused projection's output
  cache   appending to a paged cache (with the rotation of q and k, or without), moving the
          accepted nodes of a draft tree together, and reading the tokens back
  attend  attention of 1 .. 64 drafted tokens (a tree, a chain, or a single token) over a
          paged cache in fp16, int8 or e4m3
  verify  acceptance of a drafted chain or tree and the draw of the token after it

`run` computes them in their plain form, or with the package's kernels where `own` is true;
`exact` computes them once more in 64 bits, from their definitions.
"""
import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
LARGEST = {"int8": 127.0, "e4m3": 448.0}          # the largest code of a cache format
TINY = 1e-30                                      # rows below it are held as zeros
BANDS = dict(factor=8.0, length=8192.0, low=1.0, high=4.0)   # rotary scaling by frequency bands
BASE = 500000.0


# ------------------------------------------------------------------------------ the cases
def listed():
    return [
        # q and k heads of eight sequences' tokens in one decoding step
        {"name": "rope step", "op": "rope", "tokens": 8, "heads": 40, "width": 48, "dim": 128, "rot": 128,
         "layout": "half", "scaling": "none", "far": 8192},
        # a long prompt, half of each head rotated, positions far beyond the original length
        {"name": "rope prompt", "op": "rope", "tokens": 8191, "heads": 72, "width": 80, "dim": 128, "rot": 64,
         "layout": "interleaved", "scaling": "bands", "far": 1000000},
        # one token for each of 16 sequences: rotated, quantised into the cache, read back
        {"name": "cache step", "op": "cache", "batch": 16, "tokens": 1, "heads": 32, "kv": 8, "dim": 128,
         "format": "int8", "page": 16, "context": 4000, "rope": True, "layout": "half", "rot": 128, "tree": False},
        # draft trees of 24 nodes: appended, the accepted path moved together, read back
        {"name": "cache tree", "op": "cache", "batch": 8, "tokens": 24, "heads": 64, "kv": 8, "dim": 128,
         "format": "e4m3", "page": 32, "context": 2500, "rope": True, "layout": "half", "rot": 128, "tree": True},
        # ragged prompts written whole, already rotated, and gathered for a later use
        {"name": "cache prompt", "op": "cache", "batch": 4, "tokens": 4096, "heads": 0, "kv": 8, "dim": 128,
         "format": "int8", "page": 64, "context": 100, "rope": False, "layout": "half", "rot": 128, "tree": False},
        # a single user's next token over a short context
        {"name": "attend token", "op": "attend", "batch": 1, "tokens": 1, "heads": 32, "kv": 8, "dim": 128,
         "format": "fp16", "page": 16, "context": 777, "tree": False},
        # a serving batch's next tokens over ragged contexts
        {"name": "attend batch", "op": "attend", "batch": 32, "tokens": 1, "heads": 32, "kv": 8, "dim": 128,
         "format": "int8", "page": 64, "context": 8192, "tree": False},
        # draft trees over contexts of a few thousand tokens
        {"name": "attend tree", "op": "attend", "batch": 4, "tokens": 24, "heads": 64, "kv": 8, "dim": 128,
         "format": "e4m3", "page": 32, "context": 4097, "tree": True},
        # drafted chains at the end of very long contexts, five query heads a key head
        {"name": "attend long", "op": "attend", "batch": 2, "tokens": 8, "heads": 40, "kv": 8, "dim": 128,
         "format": "int8", "page": 128, "context": 131071, "tree": False},
        # four drafted tokens for each of eight sequences
        {"name": "verify chain", "op": "verify", "batch": 8, "tokens": 5, "vocab": 32000, "tree": False},
        # a serving batch with a large vocabulary
        {"name": "verify batch", "op": "verify", "batch": 64, "tokens": 8, "vocab": 128256, "tree": False},
        # draft trees of 32 nodes
        {"name": "verify tree", "op": "verify", "batch": 16, "tokens": 32, "vocab": 151936, "tree": True},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "cache", "attend", "attend", "verify"])
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 4, 5, 8])
    dim = rng.choice([64, 128, 128, 256])
    form = rng.choice(["fp16", "int8", "e4m3"])
    page = rng.choice([16, 32, 64, 128])
    if op == "rope":
        width = heads + 2 * kv
        tokens = min(_spread(rng, 1, 8191), 8191 * 72 * 128 // ((heads + kv) * dim))
        return {"op": op, "tokens": tokens, "heads": heads + kv, "width": width, "dim": dim,
                "rot": rng.choice([dim, dim, dim // 2]), "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["none", "bands"]), "far": _spread(rng, 16, 1000000)}
    if op == "cache":
        batch = _spread(rng, 1, 32)
        tree = rng.random() < 0.4
        tokens = _spread(rng, 2, 64) if tree else _spread(rng, 1, 2048)
        tokens = max(1, min(tokens, 16384 * 8 * 128 // (batch * (heads // 2 + kv) * dim)))
        return {"op": op, "batch": batch, "tokens": tokens, "heads": heads, "kv": kv, "dim": dim, "format": form,
                "page": page, "context": _spread(rng, 1, 4000), "rope": tree or rng.random() < 0.6,
                "layout": rng.choice(["half", "interleaved"]), "rot": rng.choice([dim, dim // 2]),
                "tree": tree and tokens > 1}
    if op == "attend":
        batch = _spread(rng, 1, 48)
        tokens = rng.choice([1, 1, _spread(rng, 2, 64)])
        most = min(131072 * 2 * 8 * 128 // (batch * kv * dim * (2 if form == "fp16" else 1)),
                   131072 * 2 * 8 * 40 * 128 // (batch * tokens * heads * dim))
        return {"op": op, "batch": batch, "tokens": tokens, "heads": heads, "kv": kv, "dim": dim, "format": form,
                "page": page, "context": min(_spread(rng, 1, 131071), max(1, most - tokens)),
                "tree": tokens > 1 and rng.random() < 0.6}
    batch, vocab = _spread(rng, 1, 64), _spread(rng, 500, 151936)
    tree = rng.random() < 0.5
    tokens = min(_spread(rng, 2, 48 if tree else 12), max(2, 64 * 8 * 128256 // (batch * vocab)))
    return {"op": op, "batch": batch, "tokens": tokens, "vocab": vocab, "tree": tree}


def _contexts(case):
    """The sequences' context lengths: from the longest down to a quarter of it."""
    b, c = case["batch"], case["context"]
    return [c - (3 * c * i) // (4 * b) for i in range(b)]


def _counts(case):
    """The sequences' numbers of tokens: ragged where a sequence has many."""
    b, t = case["batch"], case["tokens"]
    return [t - (t * i) // (3 * b) for i in range(b)]


def _wide(case):
    return 2 if case["format"] == "fp16" else 1


def work(case):
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": 4 * n + 4 * case["tokens"] + 4 * case["rot"], "flops": 3 * n}
    if case["op"] == "cache":
        n = sum(_counts(case))
        heads = case["heads"] if case["rope"] else 0
        row = case["kv"] * case["dim"]
        held = row * _wide(case) + (4 * case["kv"] if case["format"] != "fp16" else 0)
        # q in and out, k and v in, the cache written and read, k and v out
        moved = 4 * heads * case["dim"] + 2 * (2 * row + 2 * held + 2 * row)
        return {"bytes": n * moved, "flops": n * (3 * heads * case["dim"] + 12 * row)}
    if case["op"] == "attend":
        keys = sum(c + t for c, t in zip(_contexts(case), _counts(case)))
        row = case["kv"] * case["dim"] * _wide(case) + (4 * case["kv"] if case["format"] != "fp16" else 0)
        rows = sum(_counts(case))
        pairs = sum((c + t) * t for c, t in zip(_contexts(case), _counts(case)))
        return {"bytes": 2 * keys * row + 4 * rows * case["heads"] * case["dim"],
                "flops": 4 * pairs * case["heads"] * case["dim"]}
    rows = 1 if case["tree"] else 2     # the last row of the target, and of the draft
    return {"bytes": case["batch"] * (4 * case["vocab"] * rows + 24 * case["tokens"]),
            "flops": 3 * case["batch"] * case["vocab"]}


# ----------------------------------------------------------------------------- the inputs
def _turns(rot, scaling):
    """Turns a position for each pair of a head's rotated part, in 64 bits."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    turns = BASE ** (-2.0 * i / rot) / (2.0 * math.pi)
    if scaling == "bands":
        ramp = ((turns * BANDS["length"] - BANDS["low"]) / (BANDS["high"] - BANDS["low"])).clamp(0.0, 1.0)
        turns = turns * ramp + turns / BANDS["factor"] * (1.0 - ramp)
    return turns


def _parents(batch, tokens, tree, gen):
    """[batch, tokens] parents of the nodes (the first has none), their depths, and the
    [batch, tokens, tokens] truth of 'the row's node is below, or is, the column's'."""
    parents = torch.full((batch, tokens), -1, dtype=torch.int64)
    depth = torch.zeros((batch, tokens), dtype=torch.int64)
    sees = torch.zeros((batch, tokens, tokens), dtype=torch.bool)
    sees[:, 0, 0] = True
    rows = torch.arange(batch)
    for i in range(1, tokens):
        back = torch.randint(0, min(i, 6), (batch,), generator=gen) if tree else torch.zeros(batch, dtype=torch.int64)
        parents[:, i] = i - 1 - back
        depth[:, i] = depth[rows, parents[:, i]] + 1
        sees[:, i] = sees[rows, parents[:, i]]
        sees[:, i, i] = True
    return parents, depth, sees


def _bits(sees):
    """The rows of a truth matrix of up to 64 columns as int64 words, column 0 lowest."""
    t = sees.shape[-1]
    at = torch.arange(t, dtype=torch.int64)
    return (sees.to(torch.int64) << at).sum(-1)     # distinct bits: the sum is their union


def _quantise(x, form):
    """Rows of fp32 in a cache format: codes and, for the 8-bit ones, a scale a row."""
    if form == "fp16":
        return x.to(torch.float16), None
    most = LARGEST[form]
    amax = x.abs().amax(-1, keepdim=True)
    held = amax >= TINY
    up = torch.where(held, most / amax.clamp(min=TINY), torch.zeros_like(amax))
    y = (x * up).clamp(-most, most)
    codes = y.round().to(torch.int8) if form == "int8" else y.to(torch.float8_e4m3fn)
    return codes, torch.where(held, amax / most, torch.zeros_like(amax)).squeeze(-1)


def _table(lengths, page, gen):
    """A page table of shuffled blocks (-1 past a sequence's end) and the number of blocks."""
    need = [-(-n // page) for n in lengths]
    blocks = sum(need) + 3
    order = torch.randperm(blocks, generator=gen).to(torch.int32)
    table = torch.full((len(need), max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, blocks


def _cache(case, blocks, gen):
    """A cache's tensors, full of tokens: keys with a few wide channels, values without."""
    shape = (blocks, case["kv"], case["page"], case["dim"])
    wide = torch.ones(case["dim"], device=DEVICE)
    wide[:: case["dim"] // 4] = 4.0
    held = []
    for spread in (wide, torch.ones_like(wide)):
        codes, scale = _quantise(torch.randn(shape, generator=gen, device=DEVICE) * spread, case["format"])
        held.append((codes, scale))
    return {"k": held[0][0], "v": held[1][0], "k_scale": held[0][1], "v_scale": held[1][1]}


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=DEVICE).manual_seed(seed + 1)
    s = {"case": case}

    def halves(*shape):
        return torch.randn(shape, generator=gen, device=DEVICE).to(torch.float16)

    def whole(v):
        return torch.as_tensor(v).to(torch.int32).to(DEVICE)

    if case["op"] == "rope":
        fused = halves(case["tokens"], case["width"], case["dim"])
        s["x"] = fused[:, : case["heads"]]
        last = torch.randint(case["far"] // 2, case["far"], (1,), generator=host)
        s["positions"] = whole(last - torch.arange(case["tokens"]).flip(0)).clamp(min=0)
        s["turns"] = _turns(case["rot"], case["scaling"]).to(DEVICE)
        return s
    b, t = case["batch"], case["tokens"]
    if case["op"] == "verify":
        parents, _, _ = _parents(b, t, case["tree"], host)
        logits = torch.randn((b, t, case["vocab"]), generator=gen, device=DEVICE) * 4.0
        s["target"] = torch.softmax(logits, -1)
        from_row = parents.clamp(min=0).to(DEVICE)
        if case["tree"]:
            drawn_from = s["target"]
        else:
            logits += torch.randn(logits.shape, generator=gen, device=DEVICE) * 0.7
            drawn_from = torch.softmax(logits, -1)
            s["draft"] = drawn_from[:, : t - 1].contiguous()
        del logits
        picked = torch.multinomial(drawn_from.reshape(b * t, -1), 6, generator=gen).view(b, t, 6)
        which = torch.randint(0, 3 if case["tree"] else 1, (b, t), generator=gen, device=DEVICE)
        rows = torch.arange(b, device=DEVICE)[:, None]
        s["tokens"] = picked[rows, from_row, which].to(torch.int32)
        s["parents"] = whole(parents)
        s["uniforms"] = torch.rand((b, t), generator=gen, device=DEVICE)
        s["count"] = whole(_counts(case))
        return s
    contexts, counts = _contexts(case), _counts(case)
    table, blocks = _table([c + t for c in contexts], case["page"], host)
    s.update(_cache(case, blocks, gen))
    parents, depth, sees = _parents(b, t, case["tree"], host)
    s["table"], s["context"], s["count"] = table.to(DEVICE), whole(contexts), whole(counts)
    if case["op"] == "attend":
        s["q"] = halves(b, t, case["heads"], case["dim"])
        s["mask"] = _bits(sees).to(DEVICE) if case["tree"] else None
        s["longest"] = case["context"] + t
        return s
    fused = halves(b, t, case["heads"] + 2 * case["kv"], case["dim"])
    s["q"], s["k_new"], s["v_new"] = fused.split([case["heads"], case["kv"], case["kv"]], dim=2)
    s["positions"] = whole(torch.tensor(contexts)[:, None] + depth)
    s["turns"] = _turns(case["rot"], "none").to(DEVICE)
    if case["tree"]:        # the accepted path: from the root to a node of each sequence
        leaf = (torch.rand(b, generator=host) * torch.tensor(counts)).to(torch.int64)
        on = sees[torch.arange(b), leaf]
        nodes = torch.where(on, torch.arange(t), torch.full((b, t), t)).sort(-1).values
        s["path"] = whole(torch.where(nodes < t, nodes, -1))
        s["accepted"] = whole(on.sum(-1) - 1)
    return s


# ------------------------------------------------------------------------ the plain forms
def _rotate(x, positions, turns, layout):
    """Rows [..., heads, dim] in fp32 turned by their positions; the angles in 64 bits."""
    half = turns.shape[0]
    angle = (positions.to(torch.float64)[..., None] * turns) * (2.0 * math.pi)
    c, n = torch.cos(angle).float()[..., None, :], torch.sin(angle).float()[..., None, :]
    y = x.clone()
    if layout == "half":
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * c - b * n, b * c + a * n
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * c - b * n, b * c + a * n
    return y


def _places(s, first, tokens):
    """Blocks and slots [batch, tokens] of the positions first + 0 .. tokens - 1."""
    page = s["case"]["page"]
    at = first[:, None].long() + torch.arange(tokens, device=first.device)
    column = (at // page).clamp(max=s["table"].shape[1] - 1)
    return s["table"].gather(1, column).clamp(min=0).long(), at % page


def _raw(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _put(s, name, rows, first, counts):
    codes, scale = _quantise(rows, s["case"]["format"])
    block, slot = _places(s, first, rows.shape[1])
    block, slot = block[..., None], slot[..., None]
    head = torch.arange(rows.shape[2], device=rows.device)
    old = _raw(s[name])[block, head, slot]
    live = (torch.arange(rows.shape[1], device=rows.device) < counts[:, None])[..., None]
    _raw(s[name])[block, head, slot] = torch.where(live[..., None], _raw(codes), old)
    if scale is not None:
        kept = s[name + "_scale"]
        kept[block, head, slot] = torch.where(live, scale, kept[block, head, slot])


def _get(s, name, first, tokens):
    """[batch, tokens, kv, dim] fp32 values the cache stands for."""
    block, slot = _places(s, first, tokens)
    rows = _raw(s[name])[block, :, slot]
    rows = (rows.view(torch.float8_e4m3fn) if s[name].dtype == torch.float8_e4m3fn else rows).float()
    if s[name + "_scale"] is not None:
        rows = rows * s[name + "_scale"][block, :, slot][..., None]
    return rows


def _move(s, name, path, first, accepted):
    """Rows at first + path[d] to first + d, for 1 <= d <= accepted."""
    d = torch.arange(path.shape[1], device=path.device)
    live = ((d >= 1) & (d <= accepted[:, None]))
    block, slot = _places(s, first, path.shape[1])
    node = torch.where(live, path.long(), d)
    from_block, from_slot = block.gather(1, node), slot.gather(1, node)
    for held in (s[name], s[name + "_scale"]):
        if held is not None:
            raw = _raw(held)
            raw[block, :, slot] = raw[from_block, :, from_slot]


def _plain_cache(s):
    case = s["case"]
    q, k, v = s["q"].float(), s["k_new"].float(), s["v_new"].float()
    tokens = case["tokens"]
    live = torch.arange(tokens, device=k.device) < s["count"][:, None]
    out = {}
    if case["rope"]:
        k = _rotate(k, s["positions"], s["turns"], case["layout"])
        q = _rotate(q, s["positions"], s["turns"], case["layout"])
        out["q"] = torch.where(live[..., None, None], q, torch.zeros_like(q)).to(torch.float16)
    counts = s["count"]
    for name, rows in (("k", k), ("v", v)):
        _put(s, name, rows, s["context"], counts)
        if case["tree"]:
            _move(s, name, s["path"], s["context"], s["accepted"])
    if case["tree"]:
        live = torch.arange(tokens, device=k.device) <= s["accepted"][:, None]
    for name in ("k", "v"):
        rows = _get(s, name, s["context"], tokens)
        out[name] = torch.where(live[..., None, None], rows, torch.zeros_like(rows)).to(torch.float16)
    return out


def _plain_attend(s):
    case = s["case"]
    b, t, kv, dim = case["batch"], case["tokens"], case["kv"], case["dim"]
    group, longest = case["heads"] // kv, s["longest"]
    zero = torch.zeros_like(s["context"])
    k, v = _get(s, "k", zero, longest), _get(s, "v", zero, longest)
    q = s["q"].float().view(b, t, kv, group, dim).permute(0, 2, 1, 3, 4).reshape(b, kv, t * group, dim)
    scores = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()) * (1.0 / math.sqrt(dim))
    at = torch.arange(longest, device=q.device)
    node = at - s["context"][:, None]                           # [b, longest], < 0 in the context
    row = torch.arange(t, device=q.device)
    inside = (node[:, None, :] < s["count"][:, None, None]) & (row[:, None] < s["count"][:, None, None])
    if s["mask"] is None:
        seen = node[:, None, :] <= row[:, None]
    else:
        seen = (node < 0)[:, None, :] | ((s["mask"][:, :, None] >> node.clamp(0, 63)[:, None, :]) & 1).bool()
    seen = (seen & inside)[:, None, :, None, :].expand(b, kv, t, group, longest).reshape(b, kv, t * group, longest)
    scores = torch.where(seen, scores, torch.full_like(scores, -math.inf))
    top = scores.amax(-1, keepdim=True)
    weights = torch.exp(scores - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = weights.sum(-1, keepdim=True)
    out = torch.matmul(weights, v.permute(0, 2, 1, 3).contiguous()) / torch.where(total > 0, total, torch.ones_like(total))
    return out.view(b, kv, t, group, dim).permute(0, 2, 1, 3, 4).reshape(b, t, case["heads"], dim).to(torch.float16)


def _pick(weights, uniform):
    """The first index whose running sum of the weights (64 bits) exceeds uniform * total."""
    running = weights.double().cumsum(-1)
    return (running > uniform.double()[:, None] * running[:, -1:]).to(torch.int8).argmax(-1)


def _plain_chain(s):
    p, q, tokens, u = s["target"], s["draft"], s["tokens"].long(), s["uniforms"].double()
    b, t, _ = p.shape
    rows = torch.arange(b, device=p.device)
    node = torch.arange(t, device=p.device)
    p_at = p[:, : t - 1].gather(2, tokens[:, 1:, None]).squeeze(2).double()
    q_at = q.gather(2, tokens[:, 1:, None]).squeeze(2).double()
    good = (u[:, 1:] * q_at < p_at) & (node[1:] < s["count"][:, None])
    n = good.long().cumprod(1).sum(1)
    drafted = n < s["count"] - 1                                # stopped at a drafted token
    last = p[rows, n]
    other = q[rows, n.clamp(max=t - 2)]
    rest = (last.double() - other.double()).clamp(min=0.0)
    pick = _pick(torch.where(drafted[:, None] & (rest.sum(1, keepdim=True) > 0), rest, last.double()), s["uniforms"][:, 0])
    after = torch.cat([tokens[:, 1:], tokens[:, :1]], 1)
    out = torch.where(node < n[:, None], after, torch.where(node == n[:, None], pick[:, None], -1))
    return n.to(torch.int32), out.to(torch.int32)


def _plain_tree(s):
    p, tokens, u, parents = s["target"], s["tokens"].long(), s["uniforms"].double(), s["parents"].long()
    b, t, _ = p.shape
    rows = torch.arange(b, device=p.device)[:, None]
    node = torch.arange(t, device=p.device)
    above = parents.clamp(min=0)
    live = (node < s["count"][:, None]) & (node > 0)
    siblings = (parents[:, :, None] == parents[:, None, :]) & (node[None, :] < node[:, None]) & live[:, :, None] & live[:, None, :]
    again = (siblings & (tokens[:, :, None] == tokens[:, None, :])).any(2)
    mass = torch.where(again | ~live, 0.0, p[rows, above, tokens].double())
    left = 1.0 - (siblings.double() * mass[:, None, :]).sum(2)
    good = (u * left < mass) & live
    first = good & ~(siblings & good[:, None, :]).any(2)       # the child its parent goes on to
    links = torch.eye(t, dtype=torch.float64, device=p.device).repeat(b, 1, 1)
    links[rows, node, above] += live.double()
    below = torch.linalg.matrix_power(links, t) > 0            # [node, ancestor], itself included
    on = ~(below & ~first[:, None, :] & (node > 0)).any(2) & (live | (node == 0))
    n = on.sum(1) - 1
    path = torch.where(on, node, t).sort(1).values
    path = torch.where(path < t, path, -1)
    end = path.gather(1, n[:, None])
    tried = (parents == end) & live                            # its children, all refused
    refused = torch.zeros_like(p[:, 0], dtype=torch.bool).scatter_add_(1, tokens, tried)
    last = p[rows, end].squeeze(1)
    rest = torch.where(refused, torch.zeros_like(last), last)
    pick = _pick(torch.where(rest.double().sum(1, keepdim=True) > 0, rest, last), s["uniforms"][:, 0])
    next_node = torch.cat([path[:, 1:], path[:, :1]], 1).clamp(min=0)
    out = torch.where(node < n[:, None], tokens.gather(1, next_node), torch.where(node == n[:, None], pick[:, None], -1))
    return n.to(torch.int32), out.to(torch.int32), path.to(torch.int32)


# ---------------------------------------------------------------------------- the kernels
def _own(s):
    import semi_structured_sparse_amd as nm
    case = s["case"]
    if case["op"] == "rope":
        return nm.nm_rope(s["x"], s["positions"], s["turns"], layout=case["layout"])
    if case["op"] == "verify":
        if "workspace" not in s:
            s["workspace"] = nm.verify_workspace(case["batch"], case["vocab"], device=DEVICE)
        if case["tree"]:
            return nm.nm_verify_tree(s["target"], s["tokens"], s["parents"], s["uniforms"], count=s["count"],
                                     workspace=s["workspace"])
        return nm.nm_verify_chain(s["target"], s["draft"], s["tokens"], s["uniforms"], count=s["count"],
                                  workspace=s["workspace"])
    cache = nm.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if case["op"] == "attend":
        if "workspace" not in s:
            s["workspace"] = nm.tree_attention_workspace(s["q"], cache, s["table"])
        return nm.nm_tree_attention(s["q"], cache, s["table"], s["context"], mask=s["mask"], count=s["count"],
                                    workspace=s["workspace"])
    out, count = {}, s["count"]
    if case["rope"]:
        out["q"] = nm.nm_rope_kv_append(cache, s["q"], s["k_new"], s["v_new"], s["positions"], s["turns"], s["table"],
                                        s["context"], count=count, layout=case["layout"])
    else:
        nm.nm_kv_append(cache, s["k_new"], s["v_new"], s["table"], s["context"], count=count)
    if case["tree"]:
        nm.nm_kv_compact(cache, s["table"], s["context"], s["path"], s["accepted"])
        count = s["accepted"] + 1
    out["k"], out["v"] = nm.nm_kv_read(cache, s["table"], s["context"], case["tokens"], count=count)
    return out


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "rope":
        return _rotate(state["x"].float(), state["positions"], state["turns"], state["case"]["layout"]).to(torch.float16)
    if op == "cache":
        return _plain_cache(state)
    if op == "attend":
        return _plain_attend(state)
    return _plain_tree(state) if state["case"]["tree"] else _plain_chain(state)


# ----------------------------------------------------------------- the definitions, 64 bits
def _turned(x, positions, turns, layout):
    """Each pair as a complex number, times exp(2 pi i position turns)."""
    half = turns.shape[0]
    whole = positions.double()[:, None] * turns
    angle = 2.0 * math.pi * (whole - whole.round())
    z = torch.polar(torch.ones_like(angle), angle)[:, None, :]
    x = x.double().clone()
    if layout == "half":
        w = torch.complex(x[..., :half], x[..., half:2 * half]) * z
        x[..., :half], x[..., half:2 * half] = w.real, w.imag
    else:
        w = torch.view_as_complex(x[..., :2 * half].unflatten(-1, (half, 2)).contiguous()) * z
        x[..., :2 * half] = torch.view_as_real(w).flatten(-2)
    return x


def _held(x, form):
    """The values a cache in this format has for fp64 rows."""
    if form == "fp16":
        return x.to(torch.float16).double()
    step = x.abs().amax(-1, keepdim=True) / LARGEST[form]
    step = torch.where(step > 0, step, torch.ones_like(step))
    y = x / step
    if form == "int8":
        return y.round() * step
    # e4m3: three bits after the leading one, from 2^-6 up; steps of 2^-9 below
    power = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    grain = 2.0 ** (power - 3.0)
    return ((y / grain).round() * grain).clamp(-448.0, 448.0) * step


def exact(case, seed):
    if case["op"] == "verify":
        return None                     # whole numbers
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _turned(s["x"], s["positions"], s["turns"], case["layout"])
    contexts, counts, tokens = _contexts(case), _counts(case), case["tokens"]
    if case["op"] == "cache":
        out = {name: torch.zeros(s[src].shape, dtype=torch.float64, device=DEVICE)
               for name, src in (("q", "q"), ("k", "k_new"), ("v", "v_new")) if name != "q" or case["rope"]}
        for b in range(case["batch"]):
            n = counts[b]
            k, v = s["k_new"][b, :n].double(), s["v_new"][b, :n].double()
            if case["rope"]:
                where = s["positions"][b, :n]
                k = _turned(k, where, s["turns"], case["layout"])
                out["q"][b, :n] = _turned(s["q"][b, :n], where, s["turns"], case["layout"])
            k, v = _held(k, case["format"]), _held(v, case["format"])
            if case["tree"]:
                nodes = s["path"][b, : int(s["accepted"][b]) + 1].long()
                k, v = k[nodes], v[nodes]
            out["k"][b, : k.shape[0]], out["v"][b, : v.shape[0]] = k, v
        return out
    kv, dim, page = case["kv"], case["dim"], case["page"]
    group = case["heads"] // kv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    for b in range(case["batch"]):
        n, length = counts[b], contexts[b] + counts[b]
        blocks = s["table"][b, : -(-length // page)].long()
        rows = []
        for name in ("k", "v"):         # [kv, length, dim]
            x = _raw(s[name])[blocks]
            x = (x.view(torch.float8_e4m3fn) if s[name].dtype == torch.float8_e4m3fn else x).double()
            if s[name + "_scale"] is not None:
                x = x * s[name + "_scale"][blocks].double()[..., None]
            rows.append(x.permute(1, 0, 2, 3).reshape(kv, -1, dim)[:, :length])
        q = s["q"][b, :n].double().view(n, kv, group, dim).permute(1, 0, 2, 3).reshape(kv, n * group, dim)
        scores = q @ rows[0].transpose(1, 2).contiguous() / math.sqrt(dim)
        open_ = torch.ones(n, length, dtype=torch.bool, device=DEVICE)
        if case["tree"]:
            at = torch.arange(n, device=DEVICE)
            open_[:, contexts[b]:] = ((s["mask"][b, :n, None] >> at) & 1).bool()
        else:
            open_[:, contexts[b]:] = torch.ones(n, n, dtype=torch.bool, device=DEVICE).tril()
        scores = scores.masked_fill(~open_.repeat_interleave(group, 0), -math.inf)
        mixed = torch.softmax(scores, -1) @ rows[1].contiguous()
        out[b, :n] = mixed.view(kv, n, group, dim).permute(1, 0, 2, 3).reshape(n, case["heads"], dim)
        del rows, scores, mixed
    return out
