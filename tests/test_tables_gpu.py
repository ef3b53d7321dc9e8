"""Block tables and slot maps, the append through a slot map and the move of
accepted branches, against their definitions, and one whole verification step
of speculative decoding."""
import math

import numpy as np
import pytest
import torch

from gpu_pipeline import f64
from mla_latent_kv_23_b200 import mla
from oracle import mla_oracle as orc
from test_tree_gpu import D_C, D_R, SCALE, W, reference

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def flags():
    try:
        return mla.mla_check_device_errors()
    except mla.MLAError as e:
        return e.flags


class Tables:
    """One call's buffers, filled with a mark where nothing is to be written."""

    def __init__(self, ctx, new, page=64, max_pages=None, free=None, used=0, room=None, parents=None,
                 held=None, table=None, num_pages=None):
        B = len(ctx)
        need = [max(0, -(-(c + n) // page)) for c, n in zip(ctx, new)]
        self.page, self.B = page, B
        self.max_pages = max_pages or max(need + [1]) + 1
        self.free = free if free is not None else list(range(1000, 1000 + sum(need) + 3))[::-1]
        self.num_pages = num_pages or 1000 + len(self.free)
        self.room = room if room is not None else sum(n for n in new if n > 0) + 5
        self.ctx, self.new, self.used, self.held = ctx, new, used, held
        self.table0 = np.arange(B * self.max_pages, dtype=np.int32).reshape(B, self.max_pages) % 900 if table is None else table
        self.parents = parents
        self.table = i32(self.table0)
        self.out = {k: torch.full((n,), -7, dtype=torch.int32, device="cuda")
                    for k, n in (("free_used", 1), ("seqlens", B), ("cu", B + 1), ("seq_ids", self.room),
                                 ("pos", self.room), ("slots", self.room), ("held", B))}
        self.out["tree_mask"] = torch.full((self.room,), -7, dtype=torch.int64, device="cuda")

    def params(self):
        o = self.out
        up = None
        if self.parents is not None:
            up = i32((list(self.parents) + [5] * self.room)[:self.room])
        return mla.tables_params(i32(self.ctx), i32(self.new), self.table, i32(self.free), i32([self.used]),
                                 o["free_used"], o["seqlens"], o["cu"], o["seq_ids"], o["pos"], o["slots"], self.page,
                                 self.num_pages, parents=up, tree_mask=None if up is None else o["tree_mask"],
                                 pages_held=None if self.held is None else i32(self.held),
                                 pages_held_out=None if self.held is None else o["held"])

    def expected(self):
        e = {k: v.cpu().numpy().copy() for k, v in self.out.items()}
        for k in e:
            e[k][:] = -7
        table, used, t, wrong = self.table0.copy(), self.used, 0, 0
        for b, (c, n) in enumerate(zip(self.ctx, self.new)):
            have = -(-c // self.page)
            if self.held is not None:
                have_c, have = have, self.held[b]
            bad = c < 0 or n < 0 or c + n > self.max_pages * self.page
            if self.held is not None:
                bad = bad or have < have_c or have > self.max_pages
            if bad:
                wrong |= mla.DEVFLAG_BAD_SEQLEN
                c = n = have = 0
            want = max(have, -(-(c + n) // self.page))
            for k in range(have, want):
                if used < len(self.free):
                    table[b, k] = self.free[used]
                else:
                    table[b, k] = -1
                    wrong |= mla.DEVFLAG_NO_PAGES
                used += 1
                if k < want and not 0 <= table[b, k] < self.num_pages:
                    if table[b, k] != -1:
                        wrong |= mla.DEVFLAG_BAD_PAGE
                    table[b, k] = -1
            e["cu"][b], e["seqlens"][b], e["held"][b] = t, c + n, want
            branch = []
            for i in range(n):
                p = c + i
                m, depth = 0, i
                if self.parents is not None and n <= 64:
                    up = self.parents[t] if t < len(self.parents) else -1
                    if not -1 <= up < i:
                        wrong |= mla.DEVFLAG_BAD_TREE
                        up = -1
                    m = (branch[up] if up >= 0 else 0) | 1 << i
                    branch.append(m)
                    depth = bin(m).count("1") - 1
                if t < self.room:
                    page = table[b, p // self.page]
                    if not 0 <= page < self.num_pages:
                        if p // self.page < have:
                            wrong |= mla.DEVFLAG_BAD_PAGE
                        page = -1
                    e["seq_ids"][t], e["pos"][t] = b, c + depth
                    e["slots"][t] = -1 if page < 0 else page * self.page + p % self.page
                    e["tree_mask"][t] = m - (1 << 64) * (m >> 63)
                t += 1
        e["cu"][self.B] = t
        e["free_used"][0] = min(used, len(self.free))
        if t > self.room:
            wrong |= mla.DEVFLAG_NO_ROOM
        if self.parents is None:
            e["tree_mask"][:] = -7
        if self.held is None:
            e["held"][:] = -7
        return table, e, wrong

    def check(self):
        mla.mla_build_tables(self.params())
        got_flags = flags()
        table, e, wrong = self.expected()
        assert got_flags == wrong
        assert np.array_equal(self.table.cpu().numpy(), table)
        for k, v in e.items():
            assert np.array_equal(self.out[k].cpu().numpy(), v), k


def random_parents(new, rng):
    up = []
    for n in new:
        up += [int(rng.integers(-1, i)) if i else -1 for i in range(n)]
    return up


@pytest.mark.parametrize("page", [64, 1, 100])
@pytest.mark.parametrize("ctx,new", [
    ((0,), (1,)), ((63, 64, 65), (1, 1, 1)), ((10, 0, 500, 7), (0, 64, 65, 3)), ((128,), (0,)),
    ((5, 5, 5, 5, 5), (1, 2, 3, 127, 130)),
])
@pytest.mark.parametrize("trees", [False, True])
def test_tables(ctx, new, page, trees):
    rng = np.random.default_rng(1)
    Tables(ctx, new, page, parents=random_parents(new, rng) if trees else None).check()


@pytest.mark.parametrize("B,most", [(1, 70000), (700, 200), (3000, 9), (16384, 3)])
def test_tables_of_many(B, most):
    rng = np.random.default_rng(B)
    ctx, new = rng.integers(0, 500, B).tolist(), rng.integers(0, most + 1, B).tolist()
    Tables(ctx, new, parents=random_parents(new, rng)).check()


def test_a_wide_block_table():
    # so many columns that sums over the requests might pass 32 bits
    rng = np.random.default_rng(5)
    ctx, new = rng.integers(0, 500, 600).tolist(), rng.integers(0, 200, 600).tolist()
    Tables(ctx, new, max_pages=60000, parents=random_parents(new, rng)).check()


def test_chains_and_stars_of_64():
    for up in (list(range(-1, 63)), [-1] * 64, [-1] + [0] * 63, [-1, 0] + [i // 2 for i in range(2, 64)]):
        Tables((77,), (64,), parents=up).check()


def test_pages_held():
    # pages kept from rejected tokens; one request has too few, one too many
    Tables((64, 64, 100, 0), (1, 1, 200, 0), held=(1, 3, 2, 2), max_pages=6).check()
    Tables((64, 64, 100), (1, 1, 1), held=(0, 7, 2), max_pages=6).check()


def test_what_runs_out():
    Tables((0, 60, 0), (100, 10, 300), free=[5, 6, 7]).check()                # no pages for the last request
    Tables((0, 60), (100, 10), free=[5, 6, 7], used=9).check()                # nothing free at all
    Tables((0, 60), (100, 10), room=50, parents=[-1] * 110).check()           # outputs too small
    Tables((0, 60), (100, 10), room=0).check()
    Tables((0,), (0,), free=[]).check()
    Tables((-1, 60, 5), (100, -3, 10)).check()
    Tables((60, 2 ** 31 - 1, 5), (100, 2 ** 31 - 1, 10), max_pages=4, free=[3] * 9, room=200).check()
    Tables((0, 60), (100, 10), free=[5, 1006, -3, 8], num_pages=1000).check()  # ids out of range
    Tables((90,), (10,), table=np.full((1, 3), -1, np.int32)).check()
    Tables((5,), (6,), parents=[-1, 1, 0, -2, 3, 64]).check()                 # not earlier tokens


def test_empty_batch():
    t = Tables((), (), max_pages=2, free=[4], used=1)
    t.table = torch.zeros((0, 2), dtype=torch.int32, device="cuda")
    mla.mla_build_tables(t.params())
    mla.mla_check_device_errors()
    assert t.out["cu"].tolist() == [0] and t.out["free_used"].tolist() == [1]


# ------------------------------------------------------------------ append
def append_reference(h, wd, wk, pos):
    """The rows and how far each value may be off: a product is K products
    summed in fp32 in some order, at most K half-steps of the sum of their
    sizes; a rotated value adds both of its pair, and 2^-20 of them for the
    angle; then one rounding to the cache's type."""
    h64, w64, d_c = f64(h), np.concatenate([f64(wd), f64(wk)]), wd.shape[0]
    e = h.shape[1] * 2.0 ** -24 * (np.abs(h64) @ np.abs(w64).T)
    ref = np.concatenate([orc.latent(f64(wd), h64), np.zeros((len(h64), len(wk)))], 1)
    if len(wk):
        ref[:, d_c:] = orc.rope_key(f64(wk), h64, pos.cpu().numpy(), 10000.0)
        pair = e[:, d_c:].reshape(len(ref), -1, 2).sum(-1).repeat(2, 1)
        size = np.abs(ref[:, d_c:]).reshape(len(ref), -1, 2).sum(-1).repeat(2, 1)
        e[:, d_c:] = 1.5 * pair + 2.0 ** -20 * size
    half = 2.0 ** -8 if h.dtype == torch.bfloat16 else 2.0 ** -24
    return ref, e + half * (np.abs(ref) + e)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d_model,d_c,d_R", [
    (1, 64, 512, 64), (37, 7168, 512, 64), (256, 256, 512, 64), (257, 320, 512, 64), (1000, 512, 512, 64),
    (5, 1024, 64, 16), (40, 64, 136, 8), (33, 128, 512, 0),
])
def test_append_through_slots(T, d_model, d_c, d_R, dtype):
    g = torch.Generator().manual_seed(T)
    rows = 2 * T + 3
    h = torch.randn((T, d_model), generator=g).to(dtype)
    wd = (torch.randn((d_c, d_model), generator=g) / math.sqrt(d_model)).to(dtype)
    wk = (torch.randn((d_R, d_model), generator=g) / math.sqrt(d_model)).to(dtype)
    slots = torch.randperm(rows, generator=g)[:T].to(torch.int32)
    pos = torch.randint(0, 131072, (T,), generator=g).to(torch.int32)
    if T > 3:
        slots[2] = -1  # a token without a row
    before = torch.randn((rows, d_c + d_R), generator=g).to(dtype).cuda()
    cache = before.clone()
    mla.mla_append_latent_slots(h.cuda(), wd.cuda(), wk.cuda(), slots.cuda(), pos.cuda(), cache, rope_base=10000.0)
    mla.mla_check_device_errors()
    live = (slots >= 0).numpy()
    got = f64(cache)[slots[live].long().numpy()]
    ref, e = append_reference(h, wd, wk, pos)
    assert (np.abs(got - ref[live]) <= e[live]).all()
    rest = torch.ones(rows, dtype=torch.bool)
    rest[slots[live].long()] = False
    assert torch.equal(cache[rest.cuda()], before[rest.cuda()])


def test_append_slot_out_of_range():
    h = torch.randn((4, 64), device="cuda").to(torch.bfloat16)
    wd, wk = torch.randn((64, 64), device="cuda").to(torch.bfloat16), torch.randn((16, 64), device="cuda").to(torch.bfloat16)
    for dtype in (torch.bfloat16, torch.float32):
        cache = torch.full((8, 80), 3.0, device="cuda", dtype=dtype)
        mla.mla_append_latent_slots(h.to(dtype), wd.to(dtype), wk.to(dtype), i32([1, 8, -1, 2 ** 31 - 1]), i32([0, 1, 2, 3]), cache)
        assert flags() == mla.DEVFLAG_BAD_PAGE
        assert (cache[[0, 2, 3, 4, 5, 6, 7]] == 3).all() and not (cache[1] == 3).all()


# ------------------------------------------------------------------ accept
@pytest.mark.parametrize("width,dtype", [(576, torch.bfloat16), (80, torch.float32), (576, torch.float32), (8, torch.bfloat16)])
def test_accept(width, dtype):
    rng = np.random.default_rng(width)
    page = 64
    sizes, lens = [64, 0, 7, 1, 30, 64, 5], [64, 10, 70, 200, 130, 191, 5]
    accepted = [63, -1, 4, 0, -1, 40, 4]
    B, T = len(sizes), sum(sizes) + 4
    cu = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    mask = rng.integers(0, 2 ** 63, T).astype(np.uint64) * np.uint64(2) + rng.integers(0, 2, T).astype(np.uint64)
    mask[cu[3]] = 1
    mask[cu[6] + 4] = 0b11111  # the whole chain: nothing moves
    table = rng.permutation(B * 4).astype(np.int32).reshape(B, 4)
    before = torch.from_numpy(rng.standard_normal((B * 4 * page, width)).astype(np.float32)).to(dtype).cuda()
    want, want_path, want_len = before.clone(), np.full(T, -7), list(lens)
    for b, n in enumerate(sizes):
        m = int(mask[cu[b] + accepted[b]]) if accepted[b] >= 0 else 0
        path = [i for i in range(n) if m >> i & 1]
        row = [int(table[b, p // page]) * page + p % page for p in range(lens[b] - n, lens[b])]
        for i, k in enumerate(path):
            want[row[i]] = before[row[k]]
        want_path[cu[b]:cu[b + 1]] = path + [-1] * (n - len(path))
        want_len[b] = lens[b] - n + len(path)
    for in_place in (False, True):
        cache, lens_in, path = before.clone(), i32(lens), i32([-7] * T)
        out = lens_in if in_place else i32([-7] * B)
        p = mla.accept_params(cache, i32(table), lens_in, i32(cu), torch.from_numpy(mask.view(np.int64)).cuda(), i32(accepted), out, path, page)
        mla.mla_accept_tree(p)
        mla.mla_check_device_errors()
        assert torch.equal(cache, want) and out.tolist() == want_len and np.array_equal(path.cpu().numpy(), want_path)


def test_accept_flags():
    before = torch.randn((256, 576), device="cuda").to(torch.bfloat16)
    mask = torch.full((8,), 0b11010, dtype=torch.int64, device="cuda")

    def call(cu, lens, accepted, table=((0, 1), (2, 3))):
        cache, out, path = before.clone(), i32([-7, -7]), i32([-7] * 8)
        mla.mla_accept_tree(mla.accept_params(cache, i32(table), i32(lens), i32(cu), mask, i32(accepted), out, path, 64))
        return cache, out.tolist(), path.tolist(), flags()

    cache, out, path, f = call([0, 5, 8], [100, 50], [5, -1])  # no such token
    assert f == mla.DEVFLAG_BAD_TREE and out == [95, 47] and path == [-1] * 8 and torch.equal(cache, before)
    cache, out, path, f = call([0, 5, 8], [100, 50], [4, -2])
    assert f == mla.DEVFLAG_BAD_TREE and out == [98, 47] and path == [1, 3, 4, -1, -1, -1, -1, -1]
    for cu in ([0, 9, 8], [-1, 4, 8], [0, 5, 4]):
        cache, out, path, f = call(cu, [100, 50], [-1, -1])
        assert f == mla.DEVFLAG_BAD_TREE and torch.equal(cache, before)
    cache, out, path, f = call([0, 5, 8], [129, 2], [4, 1])  # past the block table, shorter than the tree
    assert f == mla.DEVFLAG_BAD_SEQLEN and out == [129, 2] and torch.equal(cache, before)
    cache, out, path, f = call([0, 5, 8], [100, 50], [4, -1], table=((0, 4), (2, 3)))
    assert f == mla.DEVFLAG_BAD_PAGE and torch.equal(cache, before)


# ------------------------------------------------------------------ a whole step
def test_a_verification_step_and_the_next():
    """Prompts, a drafted tree, the accepted branch, and one more token: the
    cache that is left equals one that only ever held the kept tokens, and the
    attention over it, in a captured step, equals the definition."""
    g = torch.Generator().manual_seed(3)
    rng = np.random.default_rng(3)
    page, d_model, n_h, B = 64, 256, 16, 3
    dev = "cuda"
    wd = (torch.randn((D_C, d_model), generator=g) / 16).to(torch.bfloat16).to(dev)
    wk = (torch.randn((D_R, d_model), generator=g) / 16).to(torch.bfloat16).to(dev)
    ctx, tree = [60, 130, 1], [9, 30, 64]
    max_pages, n_free = 4, 20
    num_pages = 24
    cache = torch.full((num_pages * page, W), float("nan"), device=dev, dtype=torch.bfloat16)
    free = i32(rng.permutation(num_pages)[:n_free])
    table = torch.zeros((B, max_pages), dtype=torch.int32, device=dev)

    def step(state, new, h, parents):
        """Tables and append; the outputs are the next step's inputs."""
        T = h.shape[0]
        o = {k: torch.zeros(n, dtype=torch.int32, device=dev) for k, n in
             (("used", 1), ("lens", B), ("cu", B + 1), ("seq", T), ("pos", T), ("slots", T), ("held", B))}
        o["mask"] = torch.zeros(T, dtype=torch.int64, device=dev)
        mla.mla_build_tables(mla.tables_params(state["lens"], i32(new), table, free, state["used"], o["used"], o["lens"], o["cu"], o["seq"], o["pos"],
                                               o["slots"], page, num_pages, parents=parents, tree_mask=o["mask"], pages_held=state["held"],
                                               pages_held_out=o["held"]))
        mla.mla_append_latent_slots(h, wd, wk, o["slots"], o["pos"], cache)
        return o

    state = {"lens": i32([0] * B), "used": i32([0]), "held": i32([0] * B)}
    h_ctx = torch.randn((sum(ctx), d_model), generator=g).to(torch.bfloat16).to(dev)
    chain = i32(sum(([-1] + list(range(n - 1)) for n in ctx), []))
    s1 = step(state, ctx, h_ctx, chain)
    h_tree = torch.randn((sum(tree), d_model), generator=g).to(torch.bfloat16).to(dev)
    parents = random_parents(tree, rng)
    s2 = step(s1, tree, h_tree, i32(parents))
    q = torch.randn((sum(tree), n_h, W), generator=g).to(torch.bfloat16).to(dev)
    inp = dict(q=q, cache=cache, table=table, lens=s2["lens"], cu=s2["cu"], mask=s2["mask"], page=page, sizes=tree, n_h=n_h)
    u, lse = mla.decode_tree(q, cache, table, s2["lens"], s2["cu"], s2["mask"], page, D_R, SCALE)
    mla.mla_check_device_errors()
    for t, (ur, lr, du, dl) in reference(inp).items():
        assert ((u[t].double() - ur).abs() <= du + 2.0 ** -24 * ur.abs()).all() and ((lse[t].double() - lr).abs() <= dl).all()
    # keep a branch
    accepted = [8, -1, 63]
    lens, path = torch.zeros_like(s2["lens"]), torch.zeros_like(s2["slots"])
    mla.mla_accept_tree(mla.accept_params(cache, table, s2["lens"], s2["cu"], s2["mask"], i32(accepted), lens, path, page))
    # the definition: contexts and kept tokens in order at consecutive positions
    at = np.concatenate([[0], np.cumsum(ctx)])
    cut = np.concatenate([[0], np.cumsum(tree)])
    for b in range(B):
        keep, k = [], accepted[b]
        while k >= 0:
            keep.append(k)
            k = parents[cut[b] + k]
        keep = keep[::-1]
        assert path[cut[b]:cut[b + 1]].tolist() == keep + [-1] * (tree[b] - len(keep))
        assert lens[b].item() == ctx[b] + len(keep)
        hs = torch.cat([h_ctx[at[b]:at[b + 1]], h_tree[cut[b]:cut[b + 1]][keep]])
        # (against the definition, not a second append: the sum over d_model is
        # split by the number of tokens, so two appends differ by rounding)
        want, e = append_reference(hs, wd, wk, torch.arange(len(hs)))
        p = torch.arange(len(hs), device=dev)
        assert (np.abs(f64(cache[table[b].long()[p // page] * page + p % page]) - want) <= e).all()
    # one more token each, captured; the pages of rejected tokens are used again
    h_next = torch.randn((B, d_model), generator=g).to(torch.bfloat16).to(dev)
    state = {"lens": lens, "used": s2["used"], "held": s2["held"]}
    new, none = i32([1] * B), i32([-1] * B)
    o = {k: torch.zeros(n, dtype=torch.int32, device=dev) for k, n in
         (("used", 1), ("lens", B), ("cu", B + 1), ("seq", B), ("pos", B), ("slots", B), ("held", B))}
    o["mask"] = torch.zeros(B, dtype=torch.int64, device=dev)
    q1 = torch.randn((B, n_h, W), generator=g).to(torch.bfloat16).to(dev)
    u1 = torch.zeros((B, n_h, D_C), dtype=torch.bfloat16, device=dev)
    l1 = torch.zeros((B, n_h), device=dev)
    pt = mla.tables_params(state["lens"], new, table, free, state["used"], o["used"], o["lens"], o["cu"], o["seq"], o["pos"], o["slots"], page, num_pages,
                           parents=none, tree_mask=o["mask"], pages_held=state["held"], pages_held_out=o["held"])
    pd = mla.tree_params(q1, cache, table, o["lens"], o["cu"], o["mask"], u1, l1, page, D_R, SCALE)
    ws = torch.empty(mla.mla_decode_tree_workspace_size(pd), dtype=torch.uint8, device=dev)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        mla.mla_build_tables(pt)
        mla.mla_append_latent_slots(h_next, wd, wk, o["slots"], o["pos"], cache)
        mla.mla_decode_tree(pd, ws)
    for _ in range(2):
        graph.replay()
    mla.mla_check_device_errors()
    assert o["pos"].tolist() == lens.tolist() and o["used"].tolist() == s2["used"].tolist()
    inp = dict(q=q1, cache=cache, table=table, lens=o["lens"], cu=o["cu"], mask=o["mask"], page=page, sizes=[1] * B, n_h=n_h)
    for t, (ur, lr, du, dl) in reference(inp).items():
        assert ((u1[t].double() - ur).abs() <= du + 2.0 ** -8 * (ur.abs() + du)).all() and ((l1[t].double() - lr).abs() <= dl).all()
