"""Clusters of the tree attention that end right after their last output: the
pair's signals to each other have all arrived by then, and whatever takes the
shared memory next finds nothing written into it."""
import pytest
import torch

from mla_latent_kv_23_b200 import mla
from test_tree_gpu import D_C, D_R, SCALE, W, check, draw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_h,sizes,lens,splits", [
    (128, (1,) * 40, (70,) * 40, 0),      # one segment of two tiles in each cluster
    (128, (1,) * 60, (30,) * 60, 0),      # of one tile
    (16, (9, 30, 5), (700, 65, 129), 0),  # a few tiles, split and whole
    (128, (3, 2), (64, 130), 200),        # most clusters have none
    (128, (20, 33), (200, 100), 3),       # many segments in each
])
def test_calls_back_to_back(n_h, sizes, lens, splits):
    inp = draw(sizes, lens, n_h, seed=n_h + len(sizes))
    g = torch.Generator().manual_seed(5)
    # the append's CTAs fill as much shared memory with sums that stay there
    h = torch.randn((200, 1024), generator=g).to(torch.bfloat16).cuda()
    wd, wk = ((torch.randn((d, 1024), generator=g) / 32).to(torch.bfloat16).cuda() for d in (D_C, D_R))
    slots = torch.arange(200, dtype=torch.int32, device="cuda")
    rows = torch.zeros((200, W), dtype=torch.bfloat16, device="cuda")
    u = torch.zeros((inp["q"].shape[0], n_h, D_C), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(u.shape[:2], device="cuda")
    p = mla.tree_params(inp["q"], inp["cache"], inp["table"], inp["lens"], inp["cu"], inp["mask"], u, lse, 64, D_R, SCALE, splits)
    ws = torch.empty(mla.mla_decode_tree_workspace_size(p), dtype=torch.uint8, device="cuda")
    first = None
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(100):
        mla.mla_decode_tree(p, ws)
        mla.mla_append_latent_slots(h, wd, wk, slots, slots, rows)
        if first is None:
            first = u.clone(), lse.clone(), rows.clone()
        n = sum(sizes)
        wrong += (u[:n] != first[0][:n]).sum() + (lse[:n] != first[1][:n]).sum() + (rows != first[2]).sum()
    mla.mla_check_device_errors()
    assert wrong.item() == 0
    check(inp, *first[:2])
