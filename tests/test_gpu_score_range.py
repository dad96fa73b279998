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
