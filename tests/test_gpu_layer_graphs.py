"""Captured steps of one layer at several shapes, replayed in turn (GPU)."""
import numpy as np
import pytest
import torch

import gqe_inputs as gi
from helpers import bf16_dev

pytestmark = pytest.mark.gpu

gq = pytest.importorskip("moe_gqa_query_b200")


@pytest.fixture(autouse=True)
def _cuda_and_error_word():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield
    torch.cuda.synchronize()
    assert gq.gqe_device_error() == 0


def make(dims, window):
    cfg = gq.GQEConfig(B=dims.B, T=dims.T, D=dims.D, G=dims.G, E=dims.E, k=dims.k, d=dims.d, n_shared=dims.n_shared,
                       sg=dims.sg, window=window, sinks=2 if window else 0)
    return gq.GQELayer(cfg, {k: torch.from_numpy(v.view(np.int16)) for k, v in gi.layer_weights(dims, 5).items()})


DIMS = gi.GQEDims(B=2, T=96, D=128, G=2, E=4, k=2, d=64, sg=1)


def fill_freed_memory():
    """Takes what the allocator has free and writes to it: a buffer that was let go would show it."""
    return [torch.full((1 << n,), 7.0, device="cuda") for n in range(8, 22) for _ in range(4)]


@pytest.mark.parametrize("window", [0, 20])
def test_forward_graphs_of_two_shapes(window):
    layer = make(DIMS, window)
    xs = [bf16_dev(gi.normal_bf16(3, "x", (2, T, DIMS.D))) for T in (96, 41)]
    want = [layer.forward(x).clone() for x in xs]
    for _ in range(3):
        for x, w in zip(xs, want):
            y = layer.forward_graph(x)
            junk = fill_freed_memory()
            y = layer.forward_graph(x)
            assert torch.equal(y, w)
            assert all((t == 7).all() for t in junk)


@pytest.mark.parametrize("window", [0, 20])
def test_captured_trees_of_two_sizes(window):
    """Two decode_tree captures of one layer; each replays on its own buffers, whatever ran between."""
    layer = make(DIMS, window)
    L = 64
    Kc, Vc = (bf16_dev(gi.normal_bf16(4, n, (2, DIMS.G, L, DIMS.d))) for n in ("K", "V"))
    lens = torch.tensor([50, 33], dtype=torch.int32, device="cuda")
    steps = []
    for T in (8, 5):
        x = bf16_dev(gi.normal_bf16(6, "x", (2, T, DIMS.D)))
        parent = torch.arange(-1, T - 1, dtype=torch.int32, device="cuda").repeat(2, 1)
        want = layer.decode_tree(x, parent, Kc, Vc, lens)[0].clone()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y, draft = layer.decode_tree(x, parent, Kc, Vc, lens)
        steps.append((g, y, want, draft["K"], x, parent))
    layer.decode_tree(steps[0][4][:, :3].contiguous(), steps[0][5][:, :3].contiguous(), Kc, Vc, lens)
    for _ in range(3):
        for g, y, want, K, *_ in steps:
            junk = fill_freed_memory()
            K.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want) and K.any()
            assert all((t == 7).all() for t in junk)
