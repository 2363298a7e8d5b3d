"""Shared helpers of the GPU tests of a state-space block's operators (inputs, bounds), beside
those of layer_helpers."""

import numpy as np

from layer_helpers import TINY, U, check, f64, half, offsets, rand, tdt  # noqa: F401


def split(a, lens):
    """a's rows cut into the sequences."""
    return np.split(a[:sum(lens)], np.cumsum(lens)[:-1])


def strided(t, more=24):
    """The same values as a view of rows `more` entries longer (a multiple of 16 bytes in every type)."""
    import torch
    none = 0x7f if t.dtype == torch.uint8 else float("nan")     # 0x7f: NaN of e4m3
    big = torch.full(t.shape[:-1] + (t.shape[-1] + more,), none, dtype=t.dtype, device=t.device)
    big[..., :t.shape[-1]] = t
    return big[..., :t.shape[-1]]


def same_in_graph(call, rounds=3):
    """Captures call() (a list of tensors), replays it between eager calls, and compares bits."""
    import torch
    want = call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(rounds):
        for t in got:
            t.zero_()
        graph.replay()
        eager = call()
        torch.cuda.synchronize()
        for a, b, c in zip(got, want, eager):
            assert torch.equal(a, b) and torch.equal(c, b)
