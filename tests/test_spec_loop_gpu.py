"""Speculative decoding over many steps, as a server's loop runs it: two sets
of step state that take turns, rejected drafts, prompts beside trees."""
import numpy as np
import pytest
import torch

from gpu_pipeline import f64
from mla_latent_kv_23_b200 import mla
from test_tables_gpu import append_reference, random_parents
from test_tree_gpu import D_C, D_R, SCALE, W, reference, rows_of

pytestmark = pytest.mark.gpu

PAGE, D_MODEL = 64, 256


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def weights(g):
    return tuple((torch.randn((d, D_MODEL), generator=g) / 16).to(torch.bfloat16).cuda() for d in (D_C, D_R))


def test_a_loop_of_steps():
    g, rng = torch.Generator().manual_seed(2), np.random.default_rng(2)
    B, max_pages, T = 5, 6, 5 * 64
    wd, wk = weights(g)
    free = i32(rng.permutation(40))
    cache = torch.full((40 * PAGE, W), float("nan"), dtype=torch.bfloat16, device="cuda")
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    old, new = ({k: torch.zeros(n, dtype=torch.int32, device="cuda") for k, n in (("lens", B), ("held", B), ("used", 1))} for _ in range(2))
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    seq, pos, slots, path = (torch.zeros(T, dtype=torch.int32, device="cuda") for _ in range(4))
    mask = torch.zeros(T, dtype=torch.int64, device="cuda")
    kept = [[] for _ in range(B)]
    for _ in range(14):
        sizes = rng.integers(0, 65, B)
        total = int(sizes.sum())
        parents = random_parents(sizes.tolist(), rng)
        up = i32(parents + [-1] * (T - total))
        h = torch.randn((T, D_MODEL), generator=g).to(torch.bfloat16).cuda()
        slots.fill_(-1)  # the append skips what no request has
        mla.mla_build_tables(mla.tables_params(old["lens"], i32(sizes), table, free, old["used"], new["used"], new["lens"],
                                               cu, seq, pos, slots, PAGE, 40, parents=up, tree_mask=mask,
                                               pages_held=old["held"], pages_held_out=new["held"]))
        mla.mla_append_latent_slots(h, wd, wk, slots, pos, cache)
        at = np.concatenate([[0], np.cumsum(sizes)])
        accepted = [int(rng.integers(-1, at[b + 1] - at[b])) if at[b + 1] > at[b] else -1 for b in range(B)]
        mla.mla_accept_tree(mla.accept_params(cache, table, new["lens"], cu, mask, i32(accepted), new["lens"], path, PAGE))
        mla.mla_check_device_errors()
        for b in range(B):
            k, branch = accepted[b], []
            while k >= 0:
                branch.append(k)
                k = parents[at[b] + k]
            kept[b] += [h[at[b] + k] for k in branch[::-1]]
        assert new["lens"].tolist() == [len(x) for x in kept] and cu.tolist() == at.tolist()
        pages = [p for row, n in zip(table.tolist(), new["held"].tolist()) for p in row[:n]]
        assert sorted(pages) == sorted(free[:int(new["used"])].tolist())
        old, new = new, old
    assert min(len(x) for x in kept) > 0
    for b in range(B):
        hs = torch.stack(kept[b])
        want, e = append_reference(hs, wd, wk, torch.arange(len(hs)))
        got = cache[rows_of(dict(table=table, page=PAGE), b, len(hs))]
        assert (np.abs(f64(got) - want) <= e).all()


def test_prompts_beside_trees():
    # the trees first: the attention and the accept take them, by B, and leave
    # the prompt's rows, length and cache as they are
    g, rng = torch.Generator().manual_seed(4), np.random.default_rng(4)
    wd, wk = weights(g)
    ctx, new, n_h, trees = [70, 129, 10], [9, 64, 150], 16, 2
    T, max_pages = sum(new), 4
    table = i32(rng.permutation(12).reshape(3, max_pages))
    cache = torch.randn((30 * PAGE, W), generator=g).to(torch.bfloat16).cuda()
    free = i32(12 + rng.permutation(18))
    lens, cu, used = i32([0] * 3), i32([0] * 4), i32([0])
    seq, pos, slots, path = (i32([-7] * T) for _ in range(4))
    mask = torch.full((T,), -7, dtype=torch.int64, device="cuda")
    mla.mla_build_tables(mla.tables_params(i32(ctx), i32(new), table, free, i32([0]), used, lens, cu, seq, pos, slots,
                                           PAGE, 30, parents=i32(random_parents(new, rng)), tree_mask=mask))
    h = torch.randn((T, D_MODEL), generator=g).to(torch.bfloat16).cuda()
    mla.mla_append_latent_slots(h, wd, wk, slots, pos, cache)
    mla.mla_check_device_errors()
    q = torch.randn((T, n_h, W), generator=g).to(torch.bfloat16).cuda()
    u = torch.full((T, n_h, D_C), -7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, n_h), -7.0, device="cuda")
    p = mla.tree_params(q, cache, table[:trees], lens[:trees], cu[:trees + 1], mask, u, lse, PAGE, D_R, SCALE)
    mla.mla_decode_tree(p, torch.empty(mla.mla_decode_tree_workspace_size(p), dtype=torch.uint8, device="cuda"))
    mla.mla_check_device_errors()
    n = sum(new[:trees])
    assert (u[n:] == -7).all() and (lse[n:] == -7).all()
    for t, (ur, lr, du, dl) in reference(dict(q=q, cache=cache, table=table, lens=lens, cu=cu, mask=mask, page=PAGE,
                                              sizes=new[:trees], n_h=n_h)).items():
        assert ((u[t].double() - ur).abs() <= du + 2.0 ** -8 * (ur.abs() + du)).all() and ((lse[t].double() - lr).abs() <= dl).all()
    prompt = cache[rows_of(dict(table=table, page=PAGE), 2, ctx[2] + new[2])].clone()
    want, e = append_reference(h[n:], wd, wk, torch.arange(ctx[2], ctx[2] + new[2]))
    assert (np.abs(f64(prompt[ctx[2]:]) - want) <= e).all()
    mla.mla_accept_tree(mla.accept_params(cache, table[:trees], lens[:trees], cu[:trees + 1], mask, i32([8, 63]), lens[:trees], path, PAGE))
    mla.mla_check_device_errors()
    kept = [bin(int(mask[t]) & (2 ** 64 - 1)).count("1") for t in (8, n - 1)]
    assert lens.tolist() == [ctx[0] + kept[0], ctx[1] + kept[1], ctx[2] + new[2]]
    assert path[n:].tolist() == [-7] * new[2]
    assert torch.equal(cache[rows_of(dict(table=table, page=PAGE), 2, ctx[2] + new[2])], prompt)
