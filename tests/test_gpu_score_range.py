"""GPU tests of nm_logprobs where logits times scale are large. The distances are check_scores': its run of
n / 64 + 64 additions is 50 or more longer than any lane's, which covers what these rows add to a term's
exponent d (a rounding or two of d, and one of the part below 1 that a rounded reference leaves in it)."""
import math

import pytest
import torch

from tests.gpu_helpers import device, say
from tests.test_gpu_block import generator, normal, score

pytestmark = pytest.mark.gpu


def as_float(v):
    """The scale that the kernel is given."""
    return torch.tensor(v, dtype=torch.float32).item()


@pytest.mark.parametrize("offset", [3e3, -4.5e4, 1e6, -1e6, 8e6])
@pytest.mark.parametrize("vocab", [300, 4099, 70000])
def test_entropy_beside_a_large_offset(offset, vocab):
    """Ordinary rows moved by a constant keep the entropy of their own, rounded, logits."""
    gen = generator(vocab)
    x = normal(gen, 5, vocab, spread=3.0, dtype=torch.float32) + offset
    tokens = torch.randint(0, vocab, (5,), generator=gen, device=device()).to(torch.int32)
    say(f"scores {vocab} around {offset}")
    score(x, tokens, 0)
    score(x, tokens, min(20, vocab), 0.25)


@pytest.mark.parametrize("offset", [4e4, -6e4])
@pytest.mark.parametrize("scale", [0.03125, 0.25, 64.0])
def test_entropy_of_large_halves(offset, scale):
    gen = generator(int(offset))
    x = normal(gen, 5, 5000, spread=300.0) + offset
    assert torch.isfinite(x).all()
    tokens = torch.randint(0, 5000, (5,), generator=gen, device=device()).to(torch.int32)
    score(x, tokens, 20, scale)


SCALES = [1.0, as_float(1 / 0.7), as_float(1 / 0.3), 10.0]


@pytest.mark.parametrize("fill", [-1e9, -5e9, -1e10, -1e12, -1e15, -1e20, -1e30, 5e9, 1e12, 1e30])
@pytest.mark.parametrize("vocab", [40, 3000, 70000])
def test_finite_fills(fill, vocab):
    """Masks far below the logits that are not the type's lowest value, and lone logits far above: the whole
    row, its first tiles, its last ones, all but a few tokens, and a single place."""
    gen = generator(vocab)
    x = normal(gen, 8, vocab, spread=2.0, dtype=torch.float32)
    x[0] = fill
    x[1, : vocab // 2] = fill
    x[2, vocab - vocab // 3:] = fill
    keep = x[3, [1, vocab // 2, vocab - 1]]
    x[3] = fill
    x[3, [1, vocab // 2, vocab - 1]] = keep
    x[4, vocab // 3] = fill
    x[5, ::2] = fill
    x[6] = fill + x[6] * abs(fill) * 2.0 ** -20           # near each other, many steps apart
    x[7] = torch.where(x[7] > 0, x[7], x[7] * abs(fill))
    tokens = torch.randint(0, vocab, (8,), generator=gen, device=device()).to(torch.int32)
    tokens[3] = 1
    for scale in SCALES:
        say(f"scores {vocab} filled with {fill} scale {scale}")
        score(x, tokens, 0, scale)
        score(x, tokens, min(20, vocab), scale)


@pytest.mark.parametrize("type_", [torch.float16, torch.float32])
@pytest.mark.parametrize("scale", [3e3, 1e5, 1e9, 1e20, 1e30])
def test_large_scales(type_, scale):
    """A temperature near 0: the largest logits share the row, every other has log p far below 0."""
    scale = as_float(scale)
    gen = generator(11)
    for vocab in (50, 5000, 70000):
        x = normal(gen, 12, vocab, spread=3.0, dtype=type_) + 20.0
        x[0, : vocab // 2] = torch.finfo(torch.float16).min
        x[1] = torch.finfo(torch.float16).min
        x[2, ::7] = x[2].max()
        tokens = torch.randint(0, vocab, (12,), generator=gen, device=device()).to(torch.int32)
        tokens[3:] = x[3:].argmax(-1).to(torch.int32)
        say(f"scores {vocab} {type_} scale {scale}")
        score(x, tokens, 0, scale)
        score(x, tokens, 20, scale)


@pytest.mark.parametrize("scale", [0.1, 1e-3, 1e-37, 1e-38])
def test_differences_past_the_largest_float(scale):
    """Logits of both ends of the type: their difference is no float, its product with the scale is."""
    scale = as_float(scale)
    gen = generator(5)
    x = normal(gen, 6, 3000, dtype=torch.float32) * 1e38
    x = x.clamp(-3.4e38, 3.4e38)
    x[0, ::2] = torch.finfo(torch.float32).min
    x[1] = torch.finfo(torch.float32).min
    x[1, [5, 2000]] = torch.finfo(torch.float32).max
    x[2] = torch.linspace(-3.4e38, 3.4e38, 3000, device=device())
    x[3] = x[2].flip(0)
    tokens = x.argmin(-1).to(torch.int32)
    score(x, tokens, 0, scale)
    score(x, tokens, 64, scale)


@pytest.mark.parametrize("scale", [2.3e38, 2.5e38, 3.4e38])
def test_scales_past_what_log2_e_leaves(scale):
    """Where scale * log2 e is no float."""
    scale = as_float(scale)
    gen = generator(6)
    x = normal(gen, 6, 3000, spread=1.0, dtype=torch.float32)
    x[:3] *= 1e-37
    x[3:5] *= 1e-30
    x[5] = 0.0
    score(x, x.argmax(-1).to(torch.int32), 0, scale)
    score(x, x.argmax(-1).to(torch.int32), 20, scale)


@pytest.mark.parametrize("type_", [torch.float16, torch.float32])
@pytest.mark.parametrize("vocab", [257, 1300, 2047, 4104, 4616, 9500, 14328, 50257])
def test_runs_that_leave_waves_empty(type_, vocab):
    """The last run of a row ends before some of its waves' places, or masks leave a wave fewer values than it
    is asked for: everything there meets the limit, and more than a key a thread is put in order."""
    gen = generator(vocab)
    x = normal(gen, 6, vocab, spread=2.0, dtype=type_)
    x[1, -1200:] = x[1, -1200:] + 40.0                    # the best of the row are in its last run
    x[2, -1200:] = 50.0                                   # all equal
    places = torch.arange(vocab, device=device())
    x[3] = torch.where(places % 128 < 2, x[3], torch.full_like(x[3], -float("inf")))      # in few lanes
    x[4] = torch.where(places % 512 < 8, x[4].round(), torch.full_like(x[4], -float("inf")))
    x[5] = x[5].round()                                   # long runs of ties
    tokens = torch.randint(0, vocab, (6,), generator=gen, device=device()).to(torch.int32)
    for top in (1, 5, 20, 64):
        score(x, tokens, top)
        score(x[:1], tokens[:1], top)


@pytest.mark.parametrize("type_", [torch.float16, torch.float32])
@pytest.mark.parametrize("vocab", [9000, 70000, 200001])
def test_lanes_with_many_of_the_best(type_, vocab):
    """Values that recur with every tile: the lanes that hold the best hold them in all of their tiles."""
    gen = generator(vocab)
    places = torch.arange(vocab, device=device())
    x = normal(gen, 4, vocab, spread=0.01, dtype=torch.float32)
    for i, period in enumerate((2048, 4096, 8192, 1000)):
        x[i] += normal(gen, period, spread=3.0, dtype=torch.float32)[places % period]
    x = x.to(type_)
    tokens = torch.randint(0, vocab, (4,), generator=gen, device=device()).to(torch.int32)
    for top in (1, 20, 64):
        score(x, tokens, top)


@pytest.mark.parametrize("type_", [torch.float16, torch.float32])
def test_the_longest_row_and_the_most_rows(type_):
    gen = generator(24)
    x = normal(gen, 1, 1 << 24, spread=3.0, dtype=type_)
    score(x, x.argmax(-1).to(torch.int32), 64, 0.5)
    x = normal(gen, 1 << 23, 3, spread=3.0, dtype=type_)
    tokens = torch.randint(-1, 3, (1 << 23,), generator=gen, device=device()).to(torch.int32)
    score(x, tokens, 2)
