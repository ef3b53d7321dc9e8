"""The speculative-decoding operators at the sizes of whole prompts, long
contexts and large caches, where their tiles, pieces and offsets take other
forms than in small calls."""
import math

import numpy as np
import pytest
import torch

from gpu_pipeline import f64
from mla_latent_kv_23_b200 import mla
from test_tables_gpu import append_reference
from test_tree_gpu import D_C, D_R, SCALE, W, behind_is_untouched, check, draw, run

pytestmark = pytest.mark.gpu

D_MODEL = 7168


@pytest.mark.parametrize("T", [300, 513, 1024, 2048, 2049, 4097, 8129])
def test_append_of_many_tokens(T):
    # three to nine boxes of 32 features a CTA, of 18 in all (so last tiles of
    # fewer, and two products side by side at nine), 8 to 1 CTAs along K, last
    # tiles of one token
    g = torch.Generator().manual_seed(T)
    rows = T + 70
    h = torch.randn((T, D_MODEL), generator=g).to(torch.bfloat16)
    wd = (torch.randn((D_C, D_MODEL), generator=g) / math.sqrt(D_MODEL)).to(torch.bfloat16)
    wk = (torch.randn((D_R, D_MODEL), generator=g) / math.sqrt(D_MODEL)).to(torch.bfloat16)
    slots = torch.randperm(rows, generator=g)[:T].to(torch.int32)
    pos = torch.randint(0, 131072, (T,), generator=g).to(torch.int32)
    slots[[1, T - 2]] = -1
    before = torch.randn((rows, W), generator=g).to(torch.bfloat16).cuda()
    cache = before.clone()
    mla.mla_append_latent_slots(h.cuda(), wd.cuda(), wk.cuda(), slots.cuda(), pos.cuda(), cache)
    mla.mla_check_device_errors()
    live = (slots >= 0).numpy()
    got = f64(cache)[slots[live].long().numpy()]
    ref, e = append_reference(h, wd, wk, pos)
    assert (np.abs(got - ref[live]) <= e[live]).all()
    rest = torch.ones(rows, dtype=torch.bool)
    rest[slots[live].long()] = False
    assert torch.equal(cache[rest.cuda()], before[rest.cuda()])


@pytest.mark.parametrize("n_h,sizes,lens,page,splits", [
    (128, (1,), (20000,), 64, 0),            # one block in as many pieces as there are clusters
    (128, (1,), (20000,), 64, 157),          # 157 pieces of one or two tiles: five groups of chunks
    (128, (2, 1), (12345, 4160), 128, 1),    # one chunk: page lookups of 32 tiles, again and again
    (16, (9, 3), (9000, 5000), 64, 2),       # a cut in the middle of a long block
    (16, (8,), (2049,), 64, 33),             # 33 tiles in 17 pieces
    (16, (8,), (4225,), 64, 200),            # 67 tiles in 34
])
def test_trees_over_long_contexts(n_h, sizes, lens, page, splits):
    inp = draw(sizes, lens, n_h, page=page, seed=n_h + lens[0])
    for dt in (torch.bfloat16, torch.float32):
        u, lse = run(inp, splits, dt)
        mla.mla_check_device_errors()
        check(inp, u, lse)
        behind_is_untouched(inp, u, lse)


@pytest.mark.parametrize("dtype,width", [(torch.bfloat16, (192, 64)), (torch.float32, (64, 16))])
@pytest.mark.parametrize("splits", [0, 1, 120])
def test_small_latents_over_long_contexts(dtype, width, splits):
    inp = draw((3, 1), (9000, 4161), 20, seed=splits, width=width, dtype=dtype)
    u, lse = run(inp, splits, dtype)
    mla.mla_check_device_errors()
    check(inp, u, lse)
    behind_is_untouched(inp, u, lse)


def test_rows_past_32_bit_offsets():
    # a cache of more than 2^31 values and 2^32 bytes, the sequence's pages at
    # its end: append, attention and the accepted branch
    page, pages = 64, 59000
    rows = page * pages
    assert rows * W > 2 ** 31 and 2 * rows * W > 2 ** 32
    g = torch.Generator().manual_seed(1)
    cache = torch.empty((rows, W), dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[pages - 1, 58500, pages - 3]], dtype=torch.int32, device="cuda")
    n, L, n_h = 6, 150, 16
    at = table[0].long().repeat_interleave(page) * page + torch.arange(page, device="cuda").repeat(3)
    cache[at] = torch.randn((3 * page, W), generator=g).to(torch.bfloat16).cuda()
    h = torch.randn((n, 256), generator=g).to(torch.bfloat16)
    wd, wk = ((torch.randn((d, 256), generator=g) / 16).to(torch.bfloat16) for d in (D_C, D_R))
    pos = torch.arange(L - n, L, dtype=torch.int32)
    slots = at[L - n:L].int()
    assert int(slots.min()) * W > 2 ** 31
    mla.mla_append_latent_slots(h.cuda(), wd.cuda(), wk.cuda(), slots, pos.cuda(), cache)
    mla.mla_check_device_errors()
    ref, e = append_reference(h, wd, wk, pos)
    assert (np.abs(f64(cache[at[L - n:L]]) - ref) <= e).all()
    mask = torch.tensor([0b1, 0b11, 0b101, 0b1001, 0b10101, 0b110101], dtype=torch.int64, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    inp = dict(q=torch.randn((n, n_h, W), generator=g).to(torch.bfloat16).cuda(), cache=cache, d_c=D_C, table=table,
               lens=i32(L), cu=i32(0, n), mask=mask, page=page, sizes=(n,), n_h=n_h)
    u, lse = run(inp)
    mla.mla_check_device_errors()
    check(inp, u, lse)
    before = cache[at].clone()
    lens, path = i32(0), i32(*[-7] * n)
    mla.mla_accept_tree(mla.accept_params(cache, table, inp["lens"], inp["cu"], mask, i32(5), lens, path, page))
    mla.mla_check_device_errors()
    assert path.tolist() == [0, 2, 4, 5, -1, -1] and lens.tolist() == [L - 2]
    want = before.clone()
    want[L - n:L - n + 4] = before[[L - n, L - n + 2, L - n + 4, L - n + 5]]
    assert torch.equal(cache[at], want)
