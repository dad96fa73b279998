"""Speculative decoding with packed N:M weights: the sparse products of nm_sparse.h and the
operators of nm_decode.h in one loop.

A small transformer with random weights, pruned to 2:4, generates greedily twice: one token at
a time, and with draft trees. A step of the latter runs the last accepted token and a tree of
drafts through the model together (nm_spmm_ws, nm_rope_kv_append, nm_tree_attention), verifies
the tree against the target's probabilities (nm_verify_tree) and moves the accepted path's
cache rows together (nm_kv_compact). Greedy means a target distribution with all its mass on
the best token, so both must give the same text; the drafts come from the text itself (what
followed the last tokens before), padded with guesses, and decide only how many tokens a step
yields.

    python examples/speculative_decode.py [--tokens 96] [--format int8|e4m3|fp16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import semi_structured_sparse_amd as nm  # noqa: E402

N, M = 2, 4
FORMATS = {"fp16": torch.float16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}


class Linear:
    """A packed 2:4 layer: y = x W'^T for a batch of tokens."""

    def __init__(self, rows, cols, gen, batch):
        w = torch.randn(rows, cols, generator=gen, device="cuda") / cols ** 0.5
        self.values, self.masks = nm.nm_pack(w.half(), N, M)
        self.workspace = nm.spmm_workspace(rows, cols, batch, N, M)

    def __call__(self, x):
        return nm.nm_spmm_ws(self.values, self.masks, x, N, M, workspace=self.workspace)


class Model:
    def __init__(self, nodes, form, layers=2, width=512, heads=8, kv=2, dim=64, vocab=512, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv, self.dim, self.vocab = heads, kv, dim, vocab
        self.embedding = torch.randn(vocab, width, generator=gen, device="cuda").half()
        self.layers = [{"qkv": Linear((heads + 2 * kv) * dim, width, gen, nodes), "out": Linear(width, heads * dim, gen, nodes),
                        "up": Linear(2 * width, width, gen, nodes), "down": Linear(width, 2 * width, gen, nodes)}
                       for _ in range(layers)]
        self.turns = nm.rope_turns(dim, device="cuda")
        self.page, pages = 16, 64
        self.table = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)[None]
        self.caches = [nm.kv_cache(pages, self.page, kv, dim, FORMATS[form]) for _ in range(layers)]
        # made once, for the largest step; steps of fewer nodes (the prompt's tokens) use them too
        step = torch.empty(1, nodes, heads, dim, dtype=torch.float16, device="cuda")
        self.workspace = nm.tree_attention_workspace(step, self.caches[0], self.table)
        self.verify_workspace = nm.verify_workspace(1, vocab)

    def __call__(self, tokens, positions, context, mask):
        """Probabilities fp32 [1, nodes, vocab] after each node; its k and v go into the caches."""
        nodes = tokens.shape[1]
        x = self.embedding[tokens[0]]
        for layer, cache in zip(self.layers, self.caches):
            fused = layer["qkv"](norm(x)).view(1, nodes, self.heads + 2 * self.kv, self.dim)
            q, k, v = fused.split([self.heads, self.kv, self.kv], dim=2)
            q = nm.nm_rope_kv_append(cache, q, k, v, positions, self.turns, self.table, context)
            o = nm.nm_tree_attention(q, cache, self.table, context, mask=mask, workspace=self.workspace)
            x = x + layer["out"](o.view(nodes, -1))
            x = x + layer["down"](torch.relu(layer["up"](norm(x))))
        logits = nm.nm_gemm_dense(self.embedding, norm(x)).float()
        best = logits.argmax(-1, keepdim=True)
        return torch.zeros_like(logits).scatter_(1, best, 1.0)[None]     # greedy


def norm(x):
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).half()


def drafts(text, nodes, vocab):
    """A tree of guesses below the last token: two chains of what followed it before, and single
    guesses. Returns tokens [nodes], parents [nodes]."""
    tokens, parents = [text[-1]], [-1]
    before = [i for i in range(len(text) - 2, -1, -1) if text[i] == text[-1]][:2]
    for i in before:
        at = 0
        for x in text[i + 1:i + 1 + nodes // 3]:
            tokens.append(x)
            parents.append(at)
            at = len(tokens) - 1
    while len(tokens) < nodes:
        tokens.append((text[-1] * 7 + 13 * len(tokens)) % vocab)
        parents.append(0)
    return tokens[:nodes], parents[:nodes]


def generate(model, prompt, count, nodes):
    """`count` tokens after the prompt; nodes 1 is plain decoding. Returns (text, steps)."""
    def device(v, dtype=torch.int32):
        return torch.tensor(v, dtype=dtype, device="cuda")

    text, steps = list(prompt), 0
    for i in range(len(prompt) - 1):                   # the prompt, a token at a time
        model(device([[prompt[i]]]), device([[i]]), device([i]), None)
    while len(text) < len(prompt) + count:
        context = len(text) - 1
        tokens, parents = drafts(text, nodes, model.vocab)
        depth, sees = [0] * nodes, [1] * nodes
        for i in range(1, nodes):
            depth[i] = depth[parents[i]] + 1
            sees[i] = sees[parents[i]] | 1 << i
        start, tokens = device([context]), device([tokens])
        target = model(tokens, device([[context + d for d in depth]]), start, device([sees], torch.int64))
        uniforms = torch.full((1, nodes), 0.5, device="cuda")
        accepted, out, path = nm.nm_verify_tree(target, tokens, device([parents]), uniforms,
                                                workspace=model.verify_workspace)
        for cache in model.caches:
            nm.nm_kv_compact(cache, model.table, start, path, accepted)
        text += out[0, :int(accepted[0]) + 1].tolist()
        steps += 1
    return text[:len(prompt) + count], steps


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=96)
    ap.add_argument("--nodes", type=int, default=12)
    ap.add_argument("--format", choices=sorted(FORMATS), default="int8")
    a = ap.parse_args(argv)
    prompt = [1, 5, 9, 1, 5]
    plain, plain_steps = generate(Model(a.nodes, a.format), prompt, a.tokens, 1)
    tree, tree_steps = generate(Model(a.nodes, a.format), prompt, a.tokens, a.nodes)
    same = plain == tree
    print(f"{a.tokens} tokens, {a.format} cache: {plain_steps} steps one at a time, {tree_steps} with trees of "
          f"{a.nodes} nodes; same text: {same}")
    return plain, tree, tree_steps


if __name__ == "__main__":
    result = main()
    sys.exit(0 if result[0] == result[1] else 1)
