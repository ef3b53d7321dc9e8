"""Attention of drafted trees over the paged latent cache (mla_decode_tree)
against its definition in 64 bits, at the head counts, tree sizes, masks and
lengths where its row blocks, tiles and pieces end."""
import math

import numpy as np
import pytest
import torch

from mla_latent_kv_23_b200 import mla

pytestmark = pytest.mark.gpu

D_C, D_R, W = 512, 64, 576
SCALE = 1 / math.sqrt(192.0)


def draw(sizes, lens, n_h, page=64, seed=0, masks="tree", spare_rows=3, width=(D_C, D_R), dtype=torch.bfloat16):
    """Inputs of a batch: `sizes` drafted tokens as the last of `lens` cached
    ones, over a shuffled pool whose unused rows hold NaN."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    W = sum(width)
    need = [-(-n // page) for n in lens]
    pool = sum(need) + 2
    order = rng.permutation(pool).astype(np.int32)
    table = np.zeros((len(lens), max(max(need), 1)), np.int32)
    cache = torch.full((pool * page, W), float("nan"))
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        for k in range(need[b]):
            m = min(page, n - k * page)
            r = int(table[b, k]) * page
            cache[r:r + m] = torch.randn((m, W), generator=g)
    T = sum(sizes) + spare_rows
    mask = np.zeros(T, np.uint64)
    cu = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    for b, n in enumerate(sizes):
        for r in range(n):
            if masks == "tree":
                up = int(rng.integers(-1, r)) if r else -1
                m = (int(mask[cu[b] + up]) if up >= 0 else 0) | 1 << r
            elif masks == "chain":
                m = (2 << r) - 1
            elif masks == "none":
                m = 0
            else:  # any bits, those past the tree among them
                m = int(rng.integers(0, 2 ** 63)) * 2 + int(rng.integers(0, 2))
            mask[cu[b] + r] = np.uint64(m & (2 ** 64 - 1))
    q = torch.randn((T, n_h, W), generator=g)
    q[sum(sizes):] = float("nan")
    dev = "cuda"
    return dict(q=q.to(dtype).to(dev), cache=cache.to(dtype).to(dev), d_c=width[0],
                table=torch.from_numpy(table).to(dev), lens=torch.tensor(lens, dtype=torch.int32, device=dev),
                cu=torch.from_numpy(cu).to(dev), mask=torch.from_numpy(mask.view(np.int64)).to(dev), page=page,
                sizes=sizes, n_h=n_h)


def rows_of(inp, b, n):
    p = torch.arange(n, device="cuda")
    return inp["table"][b].long()[p // inp["page"]] * inp["page"] + p % inp["page"]


def reference(inp):
    """(u, lse) and their bounds, per token; only cache rows that a token sees
    enter its sums."""
    out = {}
    cu, lens, masks = inp["cu"].tolist(), inp["lens"].tolist(), inp["mask"].tolist()
    d_c = inp.get("d_c", D_C)
    # fp32 tensors enter the products as tf32, which may cut them: 2^-10
    cut = 2.0 ** -10 if inp["q"].dtype == torch.float32 else 0.0
    weight = 2.0 ** -11 if inp["q"].dtype == torch.float32 else 2.0 ** -8
    for b, n in enumerate(inp["sizes"]):
        if n == 0:
            continue
        kv_all = inp["cache"][rows_of(inp, b, lens[b])].double()
        for r in range(n):
            t = cu[b] + r
            seen = torch.tensor([j < lens[b] - n or bool(masks[t] >> (j - lens[b] + n) & 1)
                                 for j in range(lens[b] - n, lens[b])], device="cuda")
            keep = torch.cat([torch.ones(lens[b] - n, dtype=torch.bool, device="cuda"), seen])
            kv = kv_all[keep]
            q = inp["q"][t].double()
            if len(kv) == 0:
                z = torch.zeros((inp["n_h"], d_c), dtype=torch.float64, device="cuda")
                out[t] = (z, z[:, 0] - math.inf, z + 1e-30, z[:, 0])
                continue
            s = q @ kv.T * SCALE
            lse = torch.logsumexp(s, -1)
            a = torch.exp(s - lse[:, None])
            u, abs_c = a @ kv[:, :d_c], a @ kv[:, :d_c].abs()
            # A score is a sum of W products in fp32: off by at most W half-steps
            # of the sum of their sizes, and by what its operands are cut.  A
            # weight moves by that (relatively) and by its rounding; u, normalised
            # by the rounded weights, by (weight's) (abs_c + |u|), to first order;
            # 1.02 covers the second.  Sums over L tokens in fp32 add L
            # half-steps, exp2 and log2 a few.
            e = (q.abs() @ kv.abs().T * SCALE).amax(-1) * (q.shape[1] * 2.0 ** -24 + 2 * cut + cut * cut)
            tok = (len(kv) + 64) * 2.0 ** -24
            du = 1.02 * (weight + e + tok)[:, None] * (abs_c + u.abs()) + cut * abs_c
            dl = e + tok + 2.0 ** -22 * (lse.abs() + s.abs().amax(-1) + 1)
            out[t] = (u, lse, du, dl)
    return out


def check(inp, u, lse):
    ref = reference(inp)
    half = 2.0 ** -8 if u.dtype == torch.bfloat16 else 2.0 ** -24
    for t, (ur, lr, du, dl) in ref.items():
        got = u[t].double()
        bound = du + half * (ur.abs() + du)
        assert torch.isfinite(got).all(), t
        worst = ((got - ur).abs() / bound).max().item()
        assert worst <= 1, (t, worst)
        if lse is not None:
            empty = lr == -math.inf
            assert torch.equal(lse[t] == -math.inf, empty), t
            worst = ((lse[t].double() - lr).abs() / dl)[~empty]
            assert worst.numel() == 0 or worst.max().item() <= 1, (t, worst.max().item())


def run(inp, splits=0, u_dtype=torch.bfloat16, with_lse=True):
    d_c = inp["d_c"]
    u = torch.full((inp["q"].shape[0], inp["n_h"], d_c), -7.0, dtype=u_dtype, device="cuda")
    lse = torch.full(u.shape[:2], -7.0, device="cuda") if with_lse else None
    p = mla.tree_params(inp["q"], inp["cache"], inp["table"], inp["lens"], inp["cu"], inp["mask"], u, lse,
                        inp["page"], inp["q"].shape[2] - d_c, SCALE, splits)
    ws = torch.full((mla.mla_decode_tree_workspace_size(p),), 255, dtype=torch.uint8, device="cuda")
    mla.mla_decode_tree(p, ws)
    return u, lse


def behind_is_untouched(inp, u, lse):
    n = sum(inp["sizes"])
    assert (u[n:] == -7).all() and (lse is None or (lse[n:] == -7).all())


@pytest.mark.parametrize("splits", [0, 1, 5])
@pytest.mark.parametrize("n_h,sizes,lens", [
    (128, (1,), (1,)),                        # one token, nothing before it
    (128, (2, 0, 5), (130, 70, 1000)),        # an idle sequence between two
    (128, (3, 1), (64, 65)),                  # a tile's end and one past it
    (16, (8, 9, 1), (200, 513, 64)),          # one row block, one and a bit, a part of one
    (20, (7, 13), (333, 129)),                # rows that no 16-row group holds
    (1, (64, 3), (700, 3)),                   # one head; a tree without a context
    (127, (2, 2), (100, 900)),
])
def test_trees(n_h, sizes, lens, splits):
    inp = draw(sizes, lens, n_h, seed=n_h + len(sizes))
    u, lse = run(inp, splits)
    mla.mla_check_device_errors()
    check(inp, u, lse)
    behind_is_untouched(inp, u, lse)


@pytest.mark.parametrize("masks", ["chain", "any", "none"])
@pytest.mark.parametrize("lens", [(64, 30), (700, 127)])
def test_masks(masks, lens):
    # full trees of 64 and 30 tokens, with and without a context before them
    inp = draw((64, 30), lens, 16, masks=masks, seed=5)
    u, lse = run(inp, u_dtype=torch.float32)
    mla.mla_check_device_errors()
    check(inp, u, lse)


@pytest.mark.parametrize("n_h,splits", [(128, 0), (128, 300), (8, 0), (8, 3)])
def test_many_blocks_over_chunks(n_h, splits):
    # chunks that hold several blocks, blocks that several chunks hold
    sizes = (17, 64, 1, 33)
    inp = draw(sizes, (1500, 333, 2100, 64), n_h, page=128, seed=11)
    for dt in (torch.bfloat16, torch.float32):
        u, lse = run(inp, splits, dt)
        mla.mla_check_device_errors()
        check(inp, u, lse)
        behind_is_untouched(inp, u, lse)


@pytest.mark.parametrize("B,splits", [(700, 0), (3000, 0), (3000, 2)])
def test_many_idle_sequences(B, splits):
    # few of many sequences have drafted tokens; batches on both sides of what
    # the plan keeps on chip
    rng = np.random.default_rng(B)
    sizes = np.zeros(B, int)
    sizes[rng.choice(B, 9, replace=False)] = rng.integers(1, 20, 9)
    sizes[0], sizes[-1] = 3, 5
    inp = draw(tuple(sizes.tolist()), tuple((sizes + rng.integers(0, 200, B)).tolist()), 16, seed=B)
    u, lse = run(inp, splits)
    mla.mla_check_device_errors()
    check(inp, u, lse)
    behind_is_untouched(inp, u, lse)


def test_nothing_drafted():
    inp = draw((0, 0), (70, 5), 16)
    u, lse = run(inp)
    mla.mla_check_device_errors()
    assert (u == -7).all() and (lse == -7).all()


def test_without_lse():
    inp = draw((3, 4), (100, 200), 32, seed=3)
    u, _ = run(inp, with_lse=False)
    mla.mla_check_device_errors()
    check(inp, u, None)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("n_h", [128, 20])
def test_other_branches_may_hold_anything(value, n_h):
    # drafted token 1 of a tree is non-finite (in both CTAs' columns, in one's,
    # in the RoPE key): the rows that do not see it are as if it were not there
    sizes, lens = (6, 5), (131, 64)
    for cols in ((0, 300, 575), (130,), (40,), (560,)):
        inp = draw(sizes, lens, n_h, seed=8, masks="chain")
        mask = inp["mask"].cpu().numpy().view(np.uint64)
        for b, n in enumerate(sizes):
            c0 = int(inp["cu"][b])
            for r in range(2, n):
                mask[c0 + r] &= np.uint64(~2 & (2 ** 64 - 1))  # 0 and 2.. form a chain; 1 is a leaf
            row = rows_of(inp, b, lens[b])[lens[b] - n + 1]
            for c in cols:
                inp["cache"][row, c] = value
        inp["mask"] = torch.from_numpy(mask.view(np.int64)).cuda()
        u, lse = run(inp)
        mla.mla_check_device_errors()
        ref = reference(inp)
        for b, n in enumerate(sizes):
            c0 = int(inp["cu"][b])
            for r in range(n):
                ur, lr, du, dl = ref[c0 + r]
                if r == 1:
                    continue
                assert ((u[c0 + r].double() - ur).abs() <= du + 2.0 ** -8 * (ur.abs() + du)).all()
                assert ((lse[c0 + r].double() - lr).abs() <= dl).all()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("n_h", [128, 12])
@pytest.mark.parametrize("length", [64, 101, 159, 160])
def test_tokens_nobody_sees_may_hold_anything(value, n_h, length):
    # of 64 drafted tokens, in tiles of 64 positions, at both ends of each half
    # of a tile and across two of them; whole rows of the value
    inp = draw((64, 3), (length, 70), n_h, seed=length, masks="chain")
    hidden = {0, 7, 26, 27, 31, 32, 58, 59, 63}
    mask = inp["mask"].cpu().numpy().view(np.uint64)
    for r in range(64):
        mask[r] &= np.uint64((2 ** 64 - 1) & ~sum(1 << h for h in hidden))
    inp["mask"] = torch.from_numpy(mask.view(np.int64)).cuda()
    rows = rows_of(inp, 0, length)
    for h in hidden:
        inp["cache"][rows[length - 64 + h]] = value
    u, lse = run(inp)
    mla.mla_check_device_errors()
    check(inp, u, lse)
    behind_is_untouched(inp, u, lse)


def test_large_scores_move_the_maximum():
    # scores that climb by 2^20 ... 2^50 from tile to tile, past every decision
    # to rescale
    inp = draw((4, 2), (640, 333), 32, seed=2)
    for b, n in enumerate((640, 333)):
        rows = rows_of(inp, b, n)
        inp["cache"][rows] *= torch.linspace(0.2, 12, n, device="cuda")[:, None].to(torch.bfloat16)
    u, lse = run(inp)
    mla.mla_check_device_errors()
    check(inp, u, lse)


def test_one_token_is_the_decode():
    inp = draw((1, 1, 1), (100, 1000, 64), 128, seed=4, masks="chain", spare_rows=0)
    u, lse = run(inp, u_dtype=torch.float32)
    ud, lsed = mla.decode(inp["q"].view(3, 1, 128, W), inp["cache"], inp["table"], inp["lens"], 64, D_R, SCALE)
    mla.mla_check_device_errors()
    ref = reference(inp)
    for t in range(3):
        # both are within the bound of the exact value; the decode's partials add 2^-11
        assert ((u[t] - ud[t, 0]).abs().double() <= 2 * ref[t][2] + 2.0 ** -10 * (ref[t][2] / 2.0 ** -8)).all()
        assert ((lse[t] - lsed[t, 0]).abs().double() <= 2 * ref[t][3]).all()


def test_bad_lengths_and_prefix_sums_are_flagged():
    inp = draw((3, 4, 2), (100, 200, 90), 16, seed=6)
    inp["lens"][1] = 3  # shorter than its tree
    u, lse = run(inp)
    with pytest.raises(mla.MLAError) as e:
        mla.mla_check_device_errors()
    assert e.value.flags == mla.DEVFLAG_BAD_SEQLEN
    assert (u[3:7] == 0).all() and (lse[3:7] == -math.inf).all()
    inp["sizes"] = (3, 0, 0)
    check(inp, u, lse)
    # a longer length than the block table holds
    inp["lens"][1] = inp["table"].shape[1] * 64 + 1
    u, lse = run(inp)
    with pytest.raises(mla.MLAError) as e:
        mla.mla_check_device_errors()
    assert e.value.flags == mla.DEVFLAG_BAD_SEQLEN
    assert (u[3:7] == 0).all()
    # prefix sums out of range or order: those sequences are skipped
    for cu in ([0, 3, 500, 9], [0, 3, 2, 4], [0, 3, -4, -4], [-2, 3, 3, 3]):
        inp["lens"][1] = 200
        inp["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        u, lse = run(inp)
        with pytest.raises(mla.MLAError) as e:
            mla.mla_check_device_errors()
        assert e.value.flags & mla.DEVFLAG_BAD_TREE
        assert (u[7:] == -7).all()
        if cu[0] == 0:
            check(inp, u, lse)
    # more than 64 tokens
    inp = draw((64,), (300,), 8, seed=6, spare_rows=8)
    inp["cu"] = torch.tensor([0, 65], dtype=torch.int32, device="cuda")
    u, lse = run(inp)
    with pytest.raises(mla.MLAError) as e:
        mla.mla_check_device_errors()
    assert e.value.flags == mla.DEVFLAG_BAD_TREE and (u == -7).all() and (lse == -7).all()


def test_bad_page_is_flagged_not_read():
    inp = draw((3, 4), (100, 200), 16, seed=6)
    for bad in (-1, 10 ** 6):
        inp["table"][1, 1] = bad
        run(inp)
        with pytest.raises(mla.MLAError) as e:
            mla.mla_check_device_errors()
        assert e.value.flags == mla.DEVFLAG_BAD_PAGE


def test_captured_and_replayed_on_another_stream():
    inp = draw((5, 8), (400, 777), 128, seed=9)
    want_u, want_lse = run(inp)
    u, lse = torch.zeros_like(want_u), torch.zeros_like(want_lse)
    p = mla.tree_params(inp["q"], inp["cache"], inp["table"], inp["lens"], inp["cu"], inp["mask"], u, lse, 64, D_R, SCALE)
    ws = torch.empty(mla.mla_decode_tree_workspace_size(p), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        mla.mla_decode_tree(p, ws)
    for _ in range(3):
        u.fill_(-7)
        lse.fill_(-7)
        graph.replay()
    # new lengths and masks in the same buffers
    assert torch.equal(u, want_u) and torch.equal(lse, want_lse)
    inp["lens"].copy_(torch.tensor([300, 70], dtype=torch.int32))
    inp["cache"].nan_to_num_(0.0)
    graph.replay()
    mla.mla_check_device_errors()
    check(inp, u, lse)
    # two calls at once, each with its own workspace
    other = draw((7, 2), (900, 64), 128, seed=10)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        ra = mla.decode_tree(inp["q"], inp["cache"], inp["table"], inp["lens"], inp["cu"], inp["mask"], 64, D_R, SCALE, stream=a)
        rb = mla.decode_tree(other["q"], other["cache"], other["table"], other["lens"], other["cu"], other["mask"], 64, D_R, SCALE, stream=b)
        got.append((ra, rb))
    torch.cuda.synchronize()
    mla.mla_check_device_errors()
    for ra, rb in got:
        check(inp, *ra)
        check(other, *rb)


def test_repeats_bit_for_bit():
    inp = draw((17, 40), (1500, 1300), 128, seed=12)
    first = run(inp)
    for _ in range(3):
        again = run(inp)
        assert torch.equal(first[0][:57], again[0][:57]) and torch.equal(first[1][:57], again[1][:57])


@pytest.mark.parametrize("dtype,d_c,d_R", [(torch.bfloat16, 64, 16), (torch.bfloat16, 192, 64), (torch.bfloat16, 256, 0),
                                           (torch.float32, 64, 16), (torch.float32, 96, 32)])
@pytest.mark.parametrize("splits", [0, 3])
@pytest.mark.parametrize("n_h,sizes,lens,masks", [
    (8, (1, 0, 16, 33), (1, 50, 129, 1000), "tree"), (20, (7, 64), (64, 300), "any"), (128, (2, 1), (65, 700), "chain"),
    (5, (3, 2), (3, 64), "none"),
])
def test_small_latents(n_h, sizes, lens, masks, dtype, d_c, d_R, splits):
    inp = draw(sizes, lens, n_h, seed=n_h + d_c, masks=masks, width=(d_c, d_R), dtype=dtype)
    for u_dtype in {dtype, torch.float32}:
        u, lse = run(inp, splits, u_dtype)
        mla.mla_check_device_errors()
        check(inp, u, lse)
        behind_is_untouched(inp, u, lse)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_small_latents_other_branches_may_hold_anything(dtype, value):
    inp = draw((4, 70 - 64), (130, 66), 16, seed=3, masks="chain", width=(64, 16), dtype=dtype)
    mask = inp["mask"].cpu().numpy().view(np.uint64)
    for b, n in enumerate((4, 6)):
        c0 = int(inp["cu"][b])
        mask[c0 + 2:c0 + n] &= np.uint64(~2 & (2 ** 64 - 1))  # token 1 is a leaf
        row = rows_of(inp, b, int(inp["lens"][b]))[int(inp["lens"][b]) - n + 1]
        inp["cache"][row, [5, 63, 70]] = value
    inp["mask"] = torch.from_numpy(mask.view(np.int64)).cuda()
    u, lse = run(inp, u_dtype=dtype)
    mla.mla_check_device_errors()
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    for t, (ur, lr, du, dl) in reference(inp).items():
        if t in (1, 5):
            # the token itself: NaN, but where every product is -inf, whose
            # weight is 0 (heads with q < 0 at all three places)
            zero = (inp["q"][t][:, [5, 63, 70]] < 0).all(-1) & (value == float("inf"))
            assert torch.equal(torch.isfinite(u[t].float()).all(-1), zero)
            continue
        assert ((u[t].double() - ur).abs() <= du + half * (ur.abs() + du)).all()
        assert ((lse[t].double() - lr).abs() <= dl).all()


def test_unsupported_widths_are_refused():
    for width, dtype in (((512, 32), torch.bfloat16), ((512, 64), torch.float32), ((128, 8), torch.float32), ((72, 8), torch.bfloat16)):
        inp = draw((2,), (70,), 4, width=width, dtype=dtype)
        with pytest.raises(mla.MLAError) as e:
            run(inp, u_dtype=dtype)
        assert e.value.status == 2
