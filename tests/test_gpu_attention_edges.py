"""Attention of drafted tokens with the largest call's workspace."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_skinny_amd as B
from test_gpu_serving import attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_one_workspace_serves_smaller_calls(dim):
    """The workspace of 24 sequences of 20 nodes and 700 positions, its contents whatever they were, through smaller batches,
    fewer nodes and shorter contexts; what follows it stays untouched."""
    hq, hkv, top = 8, 1, (24, 20, 700)
    need = B.bsfp8_attention_workspace_bytes(top[0], top[1], hq, hkv, dim, top[2])
    room = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")

    def launch(args, kw):
        return B.bsfp8_tree_attention(*args, **kw, ws=room[:need])
    r = np.random.default_rng(dim)
    for n, T, most in ((24, 20, 700), (1, 20, 700), (24, 3, 700), (2, 2, 650), (7, 13, 600), (1, 1, 700), (24, 1, 300)):
        lens = [most] + [int(x) for x in r.integers(0, most + 1, n - 1)]
        attend(180 + T, T, hq, hkv, dim, 32, lens, tree=T > 1, max_len=most, launch=launch)
        assert (room[need:] == 0xFF).all()
