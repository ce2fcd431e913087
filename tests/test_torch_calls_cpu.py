"""The extension module of the tensor-level block calls, without a GPU: it
makes no call on tensors that are not on one, and raises nothing itself."""

import torch

import cross_rank_collective_amd as crc
from cross_rank_collective_amd import block as K


def test_it_leaves_what_does_not_fit():
    K._torch is None and K._init()
    x, w = torch.zeros(4, 64), torch.ones(64)
    k = crc.checkpoint_empty(4, 64, "cpu")
    none = [None]
    calls = {
        "block_norm": [[x], x, *none * 5, 1e-6, 0.0, 1.0, 1.0, *none * 7],
        "block_norm_backward": [x, x, x, w[:4], *none * 7, 0.0, 0.0, 1.0, 1.0, *none * 5],
        "checkpoint_pack": [x, k, None],
        "checkpoint_unpack": [k, x, None],
        "checkpoint_wgrad": [x, k, torch.zeros(64, 64), False, None, None],
    }
    for name, args in calls.items():
        call = getattr(K._native, name)
        assert call(*args) is None, name
        assert call() is None and call(*args, None) is None, name
        assert call(*["no tensor"] * len(args)) is None, name
        for i in range(len(args)):
            assert call(*args[:i], object(), *args[i + 1:]) is None, (name, i)


def test_workspaces_serve_every_type():
    """The query knows no type: its answer is enough for the one whose rows
    are cut finest, and rows do not make it grow."""
    for cols in (8, 640, 4096, 8200, 16384):
        sizes = [crc.block_norm_backward_workspace(rows, cols) for rows in (1, 100, 5000, 1 << 20)]
        assert sizes == sorted(sizes) and sizes[-1] <= 8 * 4 * 5120 * 640 + (1 << 20), (cols, sizes)
