"""GPU tests that what decode.py refuses never passes by way of the extension: each bad argument
raises whether the extension looks at the call first or not, with the same message, and calls of
odd but allowed layouts give the same bits both ways."""
import ctypes

import pytest
import torch

import semi_structured_sparse_amd as nm
from semi_structured_sparse_amd import decode
from tests.gpu_helpers import device

pytestmark = pytest.mark.gpu
BATCH, NODES, HEADS, KV, DIM, VOCAB = 2, 3, 4, 2, 64, 50


class Neither:
    def __getattr__(self, name):
        return lambda *args: NotImplemented


def good():
    """The arguments of a call of each function, by name."""
    dev = device()
    g = torch.Generator().manual_seed(3)

    def halves(*shape):
        return torch.randn(shape, generator=g).half().to(dev)

    def whole(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    cache = nm.kv_cache(8, 16, KV, DIM, torch.int8, dev)
    table = torch.arange(8, dtype=torch.int32, device=dev).view(BATCH, 4)
    q, k, v = halves(BATCH, NODES, HEADS, DIM), halves(BATCH, NODES, KV, DIM), halves(BATCH, NODES, KV, DIM)
    turns = nm.rope_turns(DIM, device=dev)
    where = dict(block_table=table, start=whole([3, 0]), count=whole([3, 2]))
    p = torch.rand(BATCH, NODES, VOCAB, generator=g).to(dev)
    tokens, uniforms = whole([[0, 5, 7]] * BATCH), torch.rand(BATCH, NODES, generator=g).to(dev)
    verify = dict(tokens=tokens, uniforms=uniforms, count=whole([3, 3]), workspace=None)
    return {
        "nm_rope": dict(x=q[0], positions=whole([0, 1, 2]), turns=turns, layout="half", scale=1.0, out=None),
        "nm_kv_append": dict(cache=cache, k=k, v=v, **where),
        "nm_rope_kv_append": dict(cache=cache, q=q, k=k, v=v, positions=whole([[3, 4, 5], [0, 1, 2]]), turns=turns, **where,
                                  layout="half", scale=1.0, out=None),
        "nm_kv_read": dict(cache=cache, block_table=table, start=whole([3, 0]), tokens=NODES, count=whole([3, 2]), out=None),
        "nm_kv_compact": dict(cache=cache, block_table=table, start=whole([3, 0]), path=whole([[0, 2, -1]] * BATCH),
                              accepted=whole([1, 1])),
        "nm_tree_attention": dict(q=q, cache=cache, block_table=table, context=whole([3, 0]), mask=None, count=None,
                                  scale=None, workspace=None, out=None),
        "nm_verify_chain": dict(target=p, draft=p[:, 1:].contiguous(), **verify),
        "nm_verify_tree": dict(target=p, parents=whole([[-1, 0, 1]] * BATCH), **verify),
    }


def both(monkeypatch, call):
    """What call() gives or raises with the extension and without."""
    made = []
    for quick in (decode._bound(), Neither()):
        monkeypatch.setattr(decode, "_quick", quick)
        try:
            made.append(call())
        except (ValueError, TypeError, AttributeError, RuntimeError, ctypes.ArgumentError) as e:
            made.append((type(e), str(e)))
        torch.cuda.synchronize()
    monkeypatch.undo()
    return made


def test_good_calls_are_taken():
    for name, kw in good().items():
        getattr(nm, name)(**kw)
    torch.cuda.synchronize()


def strided(t):      # every second element of the last dim
    return torch.stack([t, t], -1).flatten(-2)[..., ::2]


BAD = {
    "x": [torch.Tensor.float, torch.Tensor.cpu, strided, lambda t: t[0], lambda t: t.transpose(0, 1), lambda t: t[:0]],
    "q": [torch.Tensor.float, torch.Tensor.cpu, strided, lambda t: t[0], lambda t: t.transpose(1, 2), lambda t: t[:1],
          lambda t: t[..., :32], lambda t: t.expand(BATCH, NODES, HEADS, DIM)[:, :, :, :0], lambda t: t[:, :0]],
    "k": [torch.Tensor.double, torch.Tensor.cpu, strided, lambda t: t[:, :, :1], lambda t: t[:1], lambda t: t[:, ::2],
          lambda t: t[:, :2], lambda t: t[:, :1].expand(-1, NODES, -1, -1)],
    "v": [torch.Tensor.bfloat16, torch.Tensor.cpu, strided, lambda t: t[:, :, :1], lambda t: t[:, ::2], lambda t: None],
    "positions": [torch.Tensor.long, torch.Tensor.cpu, lambda t: t[:1], lambda t: t.repeat(2, 1)],
    "turns": [torch.Tensor.float, torch.Tensor.cpu, lambda t: t[:0], lambda t: t[::2], lambda t: t[None],
              lambda t: t.repeat(2), lambda t: t.repeat(40)],
    "block_table": [torch.Tensor.long, torch.Tensor.cpu, lambda t: t[:1], lambda t: t[:, ::2], lambda t: t[0], lambda t: t[:, :0]],
    "start": [torch.Tensor.long, torch.Tensor.cpu, lambda t: t[:1], lambda t: t[:, None], lambda t: None],
    "context": [torch.Tensor.long, torch.Tensor.cpu, lambda t: t[:1], lambda t: None],
    "count": [lambda t: torch.zeros(BATCH, dtype=torch.int64, device=device()), lambda t: torch.zeros(BATCH, dtype=torch.int32),
              lambda t: torch.zeros(BATCH + 1, dtype=torch.int32, device=device())],
    "mask": [lambda t: torch.ones(BATCH, NODES, dtype=torch.int32, device=device()),
             lambda t: torch.ones(BATCH, NODES + 1, dtype=torch.int64, device=device()),
             lambda t: torch.ones(BATCH, NODES, dtype=torch.int64)],
    "workspace": [lambda t: torch.zeros(1 << 17, dtype=torch.int8, device=device()), lambda t: torch.zeros(1 << 17, dtype=torch.uint8),
                  lambda t: torch.zeros(1 << 17, dtype=torch.uint8, device=device())[1:],
                  lambda t: torch.zeros(2, 1 << 16, dtype=torch.uint8, device=device())],
    "layout": [lambda t: "other", lambda t: 7],
    "tokens": [torch.Tensor.long, torch.Tensor.cpu, lambda t: t[:1], lambda t: t[:, :1]],
    "uniforms": [torch.Tensor.double, torch.Tensor.cpu, lambda t: t[:1], lambda t: t[:, :2], lambda t: None],
    "target": [torch.Tensor.half, torch.Tensor.cpu, lambda t: t[0], lambda t: t[..., :40], lambda t: t[:, :, :0]],
    "draft": [torch.Tensor.half, torch.Tensor.cpu, lambda t: t[:1], lambda t: t[..., :40], lambda t: None],
    "parents": [torch.Tensor.long, torch.Tensor.cpu, lambda t: t[:1], lambda t: None],
    "path": [torch.Tensor.long, torch.Tensor.cpu, lambda t: t[:1], lambda t: t[0], lambda t: t.repeat(1, 30)],
    "accepted": [torch.Tensor.long, torch.Tensor.cpu, lambda t: t[:1], lambda t: None],
    "scale": [lambda t: "one", lambda t: float("inf")],
    "cache": [lambda c: c._replace(k=c.k.view(torch.uint8)), lambda c: c._replace(v=c.v[:4]), lambda c: c._replace(k_scale=None),
              lambda c: c._replace(v_scale=c.v_scale.double()), lambda c: c._replace(k=c.k.cpu()),
              lambda c: c._replace(k=c.k[:, :, ::2]), lambda c: nm.kv_cache(8, 16, KV, 48, torch.int8, device()),
              lambda c: nm.kv_cache(8, 24, KV, DIM, torch.int8, device()), lambda c: c._replace(k_scale=c.k_scale[:4])],
}
CASES = [(name, arg, i) for name, kw in (("nm_rope", "x positions turns layout"),
                                         ("nm_kv_append", "cache k v block_table start count"),
                                         ("nm_rope_kv_append", "cache q k v positions turns block_table start count layout"),
                                         ("nm_kv_read", "cache block_table start count"),
                                         ("nm_kv_compact", "cache block_table start path accepted"),
                                         ("nm_tree_attention", "q cache block_table context mask count scale workspace"),
                                         ("nm_verify_chain", "target draft tokens uniforms count workspace"),
                                         ("nm_verify_tree", "target parents tokens uniforms count workspace"))
         for arg in kw.split() for i in range(len(BAD[arg]))]


@pytest.mark.parametrize("name,arg,i", CASES)
def test_bad_arguments_raise_either_way(name, arg, i, monkeypatch):
    kw = good()[name]
    kw[arg] = BAD[arg][i](kw[arg])
    quick, slow = both(monkeypatch, lambda: getattr(nm, name)(**kw))
    assert isinstance(slow, tuple) and isinstance(slow[0], type), f"decode.py takes it: {slow}"
    assert quick == slow


@pytest.mark.parametrize("bad", [dict(tokens=0), dict(tokens=-1), dict(tokens=1.5), dict(out=(1, 2))])
def test_bad_reads_raise_either_way(bad, monkeypatch):
    kw = {**good()["nm_kv_read"], **bad}
    quick, slow = both(monkeypatch, lambda: nm.nm_kv_read(**kw))
    assert isinstance(slow[0], type) and quick == slow


@pytest.mark.parametrize("name", ["nm_rope", "nm_rope_kv_append", "nm_tree_attention"])
def test_bad_outputs_raise_either_way(name, monkeypatch):
    kw = good()[name]
    like = kw["x"] if name == "nm_rope" else kw["q"]
    for out in (like.float(), like.cpu(), like[..., :32].contiguous(), strided(like), like[:1].contiguous()):
        quick, slow = both(monkeypatch, lambda: getattr(nm, name)(**{**kw, "out": out}))
        assert isinstance(slow, tuple) and isinstance(slow[0], type) and quick == slow


def test_odd_layouts_are_taken_either_way(monkeypatch):
    """One sequence, one token, one head, slices of a fused tensor: strides that mean nothing there."""
    kw = good()
    fused = torch.randn(BATCH, NODES, 12, DIM, generator=torch.Generator().manual_seed(1)).half().to(device())
    calls = [
        ("nm_rope", dict(x=fused[0, :, 2:6])), ("nm_rope", dict(x=fused[0, :, 2:3])),
        ("nm_tree_attention", dict(q=fused[:, :, 1:5])), ("nm_tree_attention", dict(q=fused[:, :1, 4:8])),
        ("nm_tree_attention", dict(q=fused[:, 1:2].transpose(0, 1)[:, :1, :4].expand(1, 1, 4, DIM),
                                   block_table=kw["nm_tree_attention"]["block_table"][:1],
                                   context=kw["nm_tree_attention"]["context"][:1])),
        ("nm_rope_kv_append", dict(q=fused[:, :, :4], k=fused[:, :, 4:6], v=fused[:, :, 10:])),
    ]
    for name, over in calls:
        quick, slow = both(monkeypatch, lambda: getattr(nm, name)(**{**kw[name], **over}))
        assert isinstance(quick, torch.Tensor) and torch.equal(quick, slow) and quick.stride() == slow.stride()
