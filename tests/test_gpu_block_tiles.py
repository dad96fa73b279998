"""GPU tests of the block products on the tiles of long prompts: between them, the cases take every tile that
the launcher's cost model chooses from on 256 CUs, whole and with split columns, in both products."""
import pytest
import torch

import semi_structured_sparse_amd as nm
from tests import block_bounds as ref
from tests.gpu_helpers import say
from tests.test_gpu_block import generator, near, normal, packed

pytestmark = pytest.mark.gpu

# (rows, cols, vectors): split over columns in tiles of 128 x 128 and (2:4) 256 x 128, then whole ones from
# 64 x 128 to 256 x 256; rows that are not whole tiles, and half of them not groups of 8 either
SPLIT = [(1000, 8192, 260), (2100, 8224, 300), (2377, 4096, 256), (4090, 14336, 512)]
WHOLE = [(821, 288, 2385), (5700, 224, 153), (8828, 192, 204), (5566, 192, 602), (5437, 192, 1292), (16616, 192, 212),
         (26653, 192, 274), (33760, 192, 157), (4100, 1024, 1024), (14330, 544, 2047)]


@pytest.mark.parametrize("pattern", nm.PATTERNS, ids=str)
@pytest.mark.parametrize("shape", SPLIT + WHOLE, ids=str)
def test_tiles(pattern, shape):
    (N, M), (rows, cols, batch) = pattern, shape
    gen = generator(N, rows, batch)
    X = normal(gen, batch, cols)
    a, wa = packed(gen, rows, cols, N, M)
    bias, residual = normal(gen, rows), normal(gen, batch, rows)
    ws = nm.linear_workspace(rows, cols, batch, N, M)
    say(f"linear {N}:{M} {rows}x{cols} batch {batch} workspace {0 if ws is None else ws.numel()}")
    want, slack = ref.linear(X.double(), wa, bias.double(), "gelu_tanh", 0.5, residual.double())
    for w in {None, ws}:
        near(nm.nm_linear(*a, X, N, M, bias, "gelu_tanh", 0.5, residual, w), want, slack, "linear")
    out = residual.clone()
    nm.nm_linear(*a, X, N, M, bias, "gelu_tanh", 0.5, out, ws, out)
    near(out, want, slack, "linear onto its residual")
    del want, slack, out
    b, wb = packed(gen, rows, cols, N, M)
    gws = nm.gated_workspace(rows, cols, batch, N, M)
    say(f"gated {N}:{M} {rows}x{cols} batch {batch} workspace {0 if gws is None else gws.numel()}")
    want, slack = ref.gated(X.double(), wa, wb, bias.double(), None, "silu")
    for w in {None, gws}:
        near(nm.nm_gated(a, b, X, N, M, "silu", bias, None, w), want, slack, "gated")
    for w in (ws, gws):
        assert w is None or not w[:1024].any(), "the counters are left at zero"
    assert shape not in SPLIT or (ws is not None or gws is not None)
