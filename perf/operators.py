"""Cases of the speculative-decoding operators over the paged latent cache.

One step of a server that verifies drafted tokens runs four operators in turn:

* ``tables``: block tables and slot maps built on the GPU from the requests' lengths (new pages from a free list, a
  cache row and a position for every new token, an ancestor mask for every token of a drafted tree);
* ``append``: the new tokens' latent and RoPE key, written to the cache rows of the slot map;
* ``tree``: attention of the drafted trees' tokens over the paged latent cache;
* ``accept``: the accepted branch of every tree moved to the front of its tree's rows.

``own`` chooses between their plain form in elementary torch operations and the framework's calls.  Lengths and tree
sizes are spread over a case's range by a rule of the case alone; the seed chooses their order and every value.
"""
import math

import numpy as np
import torch

own = False

D_C, D_R, D_MODEL = 512, 64, 7168  # the latent, RoPE and hidden widths of the DeepSeek-V3 shape
WIDTH = D_C + D_R
SCALE = 1.0 / math.sqrt(192.0)
ROPE_BASE = 10000.0
DEV = "cuda"


# ---------------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one request, one new token, a short context: the call's latency is all there is
        {"name": "tree 1x1x70", "op": "tree", "B": 1, "heads": 128, "t_min": 1, "t_max": 1, "l_min": 70, "l_max": 70, "page": 64},
        # the v3 decode batch with chains of eight drafted tokens
        {"name": "tree 16x8x4096", "op": "tree", "B": 16, "heads": 128, "t_min": 8, "t_max": 8, "l_min": 4096, "l_max": 4096, "page": 64},
        # the v3 batch with full trees of 64 tokens: as many scores as one call can hold, tensor-bound
        {"name": "tree 16x64x4096", "op": "tree", "B": 16, "heads": 128, "t_min": 64, "t_max": 64, "l_min": 3900, "l_max": 4200, "page": 64},
        # one of eight head shards (16 heads) on the ragged batch, trees of odd sizes, larger pages
        {"name": "tree 64 shard ragged", "op": "tree", "B": 64, "heads": 16, "t_min": 5, "t_max": 21, "l_min": 512, "l_max": 32768, "page": 128},
        # four requests of the longest context
        {"name": "tree 4x6x131072", "op": "tree", "B": 4, "heads": 128, "t_min": 6, "t_max": 6, "l_min": 131072, "l_max": 131072, "page": 64},
        # a step of a small server: eight drafted tokens per request
        {"name": "tables 16 drafts", "op": "tables", "B": 16, "t_min": 8, "t_max": 8, "l_min": 900, "l_max": 4096, "page": 64, "trees": True},
        # a full scheduler step: 512 requests, drafted trees and whole prompts mixed
        {"name": "tables 512 mixed", "op": "tables", "B": 512, "t_min": 1, "t_max": 8192, "l_min": 0, "l_max": 20000, "page": 64, "trees": True},
        # the new tokens of a few requests
        {"name": "append 37", "op": "append", "T": 37, "page": 64},
        # the new tokens of the v3 batch with full trees
        {"name": "append 1024", "op": "append", "T": 1024, "page": 64},
        # a small server's accepted branches
        {"name": "accept 16x8", "op": "accept", "B": 16, "t_min": 8, "t_max": 8, "page": 64},
        # many requests with trees of up to 64 tokens and long accepted branches
        {"name": "accept 256x64", "op": "accept", "B": 256, "t_min": 33, "t_max": 64, "page": 64},
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "tables", "append", "accept"])
    page = rng.choice([64, 64, 128, 256])
    if op == "append":
        return {"op": op, "T": _log(rng, 1, 1024), "page": page}
    if op == "accept":
        t = _log(rng, 1, 64)
        return {"op": op, "B": _log(rng, 1, 256), "t_min": rng.randint(0, t), "t_max": t, "page": page}
    if op == "tables":
        trees = rng.random() < 0.5
        t = _log(rng, 1, 8192)
        b = max(1, min(_log(rng, 1, 512), 512 * 2048 // t))
        l_max = _log(rng, 1, 20000)
        return {"op": op, "B": b, "t_min": rng.randint(0, min(t, 64)), "t_max": t, "l_min": rng.randint(0, l_max), "l_max": l_max, "page": page, "trees": trees}
    heads = rng.choice([128, 128, 64, 32, 16, 8, rng.randint(1, 128)])
    t = _log(rng, 1, 64)
    l_max = _log(rng, max(65, t + 1), 65536)
    # no more scores than the listed trees have, and no larger caches
    b = max(1, min(_log(rng, 1, 64), 2000000 // l_max, 500000000 // (l_max * heads * t)))
    return {"op": op, "B": b, "heads": heads, "t_min": rng.randint(0, t), "t_max": t, "l_min": rng.randint(t, l_max), "l_max": l_max, "page": page}


def _spread(lo, hi, n, step):
    """n whole numbers from lo to hi, evenly over the logarithm of their distance from 0, in the order of `step`."""
    if n == 1:
        return [hi]
    a, b = math.log1p(lo), math.log1p(hi)
    v = [min(hi, max(lo, int(round(math.expm1(a + (b - a) * i / (n - 1)))))) for i in range(n)]
    while math.gcd(step, n) != 1:
        step += 1
    return [v[i * step % n] for i in range(n)]


def _sizes(case):
    """(tokens in the cache with the new ones, new tokens) of every request, before the seed orders them."""
    n = case["B"]
    t = _spread(case["t_min"], case["t_max"], n, 7)
    if case["op"] == "accept":
        return [(k + 100, k) for k in t]
    ctx = _spread(case["l_min"], case["l_max"], n, 1)
    return [(c, k) for c, k in zip(ctx, t)] if case["op"] == "tree" else [(c + k, k) for c, k in zip(ctx, t)]


def work(case):
    if case["op"] == "append":
        t = case["T"]
        return {"bytes": 2 * t * D_MODEL + 2 * WIDTH * D_MODEL + 2 * t * WIDTH + 8 * t, "flops": 2 * t * WIDTH * D_MODEL}
    s = _sizes(case)
    rows = sum(t for _, t in s)
    if case["op"] == "tables":
        pages = sum(-(-n // case["page"]) - -(-(n - t) // case["page"]) for n, t in s)
        # lengths in and out, prefix sums, new pages in and out, three numbers a token, a parent and a mask where it is a tree's
        tree = sum(t for _, t in s if t <= 64) if case["trees"] else 0
        return {"bytes": 4 * (4 * len(s) + 3) + 8 * pages + 12 * rows + 4 * tree + 8 * rows * case["trees"], "flops": 0}
    if case["op"] == "accept":
        # the mask of the accepted token and one row in and out for each token of an accepted branch, about a quarter of a tree
        return {"bytes": sum(24 + 8 * t + max(1, t // 4) * 4 * WIDTH for _, t in s if t), "flops": 0}
    h = case["heads"]
    seen = sum(t * (n - t + 1) for n, t in s)
    read = sum(n for n, t in s if t)
    return {"bytes": 2 * WIDTH * read + rows * h * (2 * WIDTH + 2 * D_C + 4) + 8 * rows + 8 * len(s), "flops": 2 * h * (WIDTH + D_C) * seen}


# --------------------------------------------------------------------------------------------------------- the inputs
def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _normal(shape, g, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(torch.bfloat16)


def _tree_masks(parents, n):
    """Ancestor masks [B, 64] (bit i: token i is on the token's branch) and depths, from parents [B, 64] (-1: a root)."""
    i = torch.arange(64, device=DEV)
    up = (parents.long()[:, :, None] == i) & (i[:, None] < n.long()[:, None, None])
    seen = (up | torch.eye(64, dtype=torch.bool, device=DEV)).float()
    for _ in range(6):  # branches of 1, 2, 4 ... 64 tokens
        seen = (torch.matmul(seen, seen) > 0).float()
    on = (seen > 0) & (i[:, None] < n.long()[:, None, None])
    masks = (on.long() << i).sum(-1)  # bit 63 is the sign
    return masks, on.sum(-1) - 1


def _random_parents(n, g):
    """Drafted trees: a token follows one of the four before it, or starts a branch at the root."""
    i = torch.arange(64, device=DEV).expand(len(n), 64)
    back = torch.randint(1, 5, i.shape, generator=g, device=DEV)
    return (i - back).clamp(min=-1).to(torch.int32)


def _pages(case, lens, g):
    """A block table over a shuffled pool that holds the requests' pages and a few more."""
    page = case["page"]
    need = [-(-n // page) for n in lens]
    pool = sum(need) + 8
    order = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    first = np.cumsum([0] + need)
    at = torch.from_numpy(first[:-1]).to(DEV)[:, None] + torch.arange(max(max(need), 1), device=DEV)
    table = order[at.clamp(max=pool - 1)]
    held = torch.arange(table.shape[1], device=DEV) < torch.tensor(need, device=DEV)[:, None]
    return torch.where(held, table, torch.zeros_like(table)).contiguous(), pool, order[int(first[-1]):].contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = {"op": case["op"], "page": case["page"]}
    if case["op"] == "append":
        t = case["T"]
        pool = -(-2 * t // case["page"]) * case["page"]
        st["h"] = _normal((t, D_MODEL), g)
        st["w_dkv"] = _normal((D_C, D_MODEL), g, D_MODEL ** -0.5)
        st["w_kr"] = _normal((D_R, D_MODEL), g, D_MODEL ** -0.5)
        st["slots"] = torch.randperm(pool, generator=g, device=DEV)[:t].to(torch.int32)
        st["pos"] = torch.randint(0, 131072, (t,), generator=g, device=DEV).to(torch.int32)
        st["cache"] = _normal((pool, WIDTH), g)
        return st
    sizes = _sizes(case)
    order = torch.randperm(len(sizes), generator=g, device=DEV).tolist()
    lens, news = [sizes[i][0] for i in order], [sizes[i][1] for i in order]
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    total = int(cu[-1])
    st["cu"] = torch.from_numpy(cu).to(DEV)
    n64 = _i32([min(t, 64) for t in news])
    parents = _random_parents(news, g)
    tok = torch.arange(total, device=DEV)
    seq = torch.bucketize(tok, st["cu"].long()[1:], right=True)
    local = tok - st["cu"].long()[seq]
    packed_parents = parents[seq, local.clamp(max=63)].contiguous()
    if case["op"] == "tables":
        table, pool, free = _pages(case, [n - t for n, t in zip(lens, news)], g)
        more = sum(-(-n // case["page"]) - -(-(n - t) // case["page"]) for n, t in zip(lens, news))
        width = max(1, -(-max(lens) // case["page"]))
        st["table"] = torch.zeros((len(lens), max(width, table.shape[1])), dtype=torch.int32, device=DEV)
        st["table"][:, : table.shape[1]] = table
        used = table.numel()  # the pool's other pages: ids behind those in use
        st["num_pages"] = used + more + 16
        st["free"] = torch.randperm(more + 11, generator=g, device=DEV).to(torch.int32) + used
        st["free_used"] = _i32([5])
        st["ctx"] = _i32([n - t for n, t in zip(lens, news)])
        st["new"] = _i32(news)
        st["parents"] = packed_parents if case["trees"] else None
        st["out"] = {"free_used": _i32([0]), "seqlens": _i32([0] * len(lens)), "cu": _i32([0] * (len(lens) + 1))}
        for k in ("seq_ids", "pos", "slots"):
            st["out"][k] = torch.full((max(total, 1),), -7, dtype=torch.int32, device=DEV)
        if case["trees"]:
            st["out"]["tree_mask"] = torch.full((max(total, 1),), -7, dtype=torch.int64, device=DEV)
        if own:
            from mla_latent_kv_23_b200 import mla
            o = st["out"]
            st["p"] = mla.tables_params(st["ctx"], st["new"], st["table"], st["free"], st["free_used"], o["free_used"], o["seqlens"], o["cu"], o["seq_ids"],
                                        o["pos"], o["slots"], case["page"], st["num_pages"], parents=st["parents"], tree_mask=o.get("tree_mask"))
        return st
    masks, _ = _tree_masks(parents, n64)
    st["mask"] = masks[seq, local].contiguous() if total else torch.zeros(1, dtype=torch.int64, device=DEV)
    st["seqlens"] = _i32(lens)
    st["table"], pool, _ = _pages(case, lens, g)
    st["cache"] = _normal((pool * case["page"], WIDTH), g)
    if case["op"] == "accept":
        # the accepted token is one in the middle of its tree; every fifth request accepts none
        st["accepted"] = _i32([t // 2 if t and i % 5 else -1 for i, t in enumerate(news)])
        st["out"] = {"seqlens": _i32([0] * len(lens)), "path": torch.full((max(total, 1),), -7, dtype=torch.int32, device=DEV)}
        if own:
            from mla_latent_kv_23_b200 import mla
            st["p"] = mla.accept_params(st["cache"], st["table"], st["seqlens"], st["cu"], st["mask"], st["accepted"], st["out"]["seqlens"], st["out"]["path"], case["page"])
        return st
    st["q"] = _normal((max(total, 1), case["heads"], WIDTH), g)
    st["u"] = torch.zeros((max(total, 1), case["heads"], D_C), dtype=torch.bfloat16, device=DEV)
    st["lse"] = torch.zeros((max(total, 1), case["heads"]), dtype=torch.float32, device=DEV)
    st["total"], st["max_q"], st["max_len"] = total, max(max(news), 1), max(lens)
    if own:
        from mla_latent_kv_23_b200 import mla
        st["p"] = mla.tree_params(st["q"], st["cache"], st["table"], st["seqlens"], st["cu"], st["mask"], st["u"], st["lse"], case["page"], D_R, SCALE)
        st["ws"] = torch.empty(mla.mla_decode_tree_workspace_size(st["p"]), dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------------------------------------------------ the plain form
def _plain_append(st):
    x = st["h"].float()
    c = torch.matmul(x, st["w_dkv"].float().T)
    k = torch.matmul(x, st["w_kr"].float().T)
    ang = st["pos"].double()[:, None] * ROPE_BASE ** (-torch.arange(0, D_R, 2, device=DEV, dtype=torch.float64) / D_R)
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    even, odd = k[:, 0::2], k[:, 1::2]
    k = torch.stack([even * cos - odd * sin, even * sin + odd * cos], -1).flatten(1)
    st["cache"][st["slots"].long()] = torch.cat([c, k], 1).to(torch.bfloat16)
    return {"cache": st["cache"]}


def _plain_tables(st):
    page, o = st["page"], st["out"]
    ctx, new = st["ctx"].long(), st["new"].long()
    have, want = (ctx + page - 1) // page, (ctx + new + page - 1) // page
    start = torch.cumsum(want - have, 0) - (want - have) + st["free_used"].long()
    col = torch.arange(st["table"].shape[1], device=DEV)
    taken = (col >= have[:, None]) & (col < want[:, None])
    at = (start[:, None] + col - have[:, None]).clamp(0, len(st["free"]) - 1)
    st["table"].copy_(torch.where(taken, st["free"][at], st["table"]))
    o["free_used"].copy_(st["free_used"] + (want - have).sum())
    o["seqlens"].copy_(ctx + new)
    o["cu"][1:] = torch.cumsum(new, 0)
    cu = o["cu"].long()
    tok = torch.arange(len(o["slots"]), device=DEV)
    seq = torch.bucketize(tok, cu[1:], right=True)
    live = seq < len(ctx)
    seq = seq.clamp(max=len(ctx) - 1)
    local = tok - cu[seq]
    pos = ctx[seq] + local
    row = st["table"].long()[seq, (pos // page).clamp(max=st["table"].shape[1] - 1)] * page + pos % page
    o["slots"].copy_(torch.where(live, row.to(torch.int32), o["slots"]))
    o["seq_ids"].copy_(torch.where(live, seq.to(torch.int32), o["seq_ids"]))
    if st["parents"] is not None:
        n = torch.where(new <= 64, new, 0)
        last = len(st["parents"]) - 1
        i = torch.arange(64, device=DEV)
        if last >= 0:
            masks, depth = _tree_masks(torch.where(i < n[:, None], st["parents"][(cu[:-1, None] + i).clamp(max=last)], -1), n)
            tree = new[seq] <= 64
            low = local.clamp(max=63)
            pos = torch.where(tree, ctx[seq] + depth[seq, low], pos)
            o["tree_mask"].copy_(torch.where(live, torch.where(tree, masks[seq, low], 0), o["tree_mask"]))
    o["pos"].copy_(torch.where(live, pos.to(torch.int32), o["pos"]))
    return {"table": st["table"], **o}


def _plain_tree(st):
    page, cu, lens = st["page"], st["cu"].long(), st["seqlens"].long()
    n = cu[1:] - cu[:-1]
    j = torch.arange(st["max_len"], device=DEV)
    rows = st["table"].long()[:, j // page] * page + j % page
    kv = st["cache"][rows].float()
    kv = torch.where((j < lens[:, None])[..., None], kv, torch.zeros((), device=DEV))
    r = torch.arange(st["max_q"], device=DEV)
    at = (cu[:-1, None] + r).clamp(max=len(st["q"]) - 1)
    q = st["q"][at].float()
    b, t, h, _ = q.shape
    s = torch.matmul(q.reshape(b, t * h, WIDTH), kv.transpose(1, 2)).view(b, t, h, -1) * SCALE
    rel = j - (lens - n)[:, None]
    bit = (st["mask"][at][:, :, None] >> rel.clamp(0, 63)[:, None, :]) & 1
    seen = (j < lens[:, None])[:, None] & ((rel < 0)[:, None] | (bit == 1))
    s = s.masked_fill_(~seen[:, :, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    u = torch.matmul(p.view(b, t * h, -1), kv[..., :D_C]).view(b, t, h, D_C) / torch.where(z > 0, z, torch.ones_like(z))
    lse = (m + z.log()).squeeze(-1)
    tok = torch.arange(st["total"], device=DEV)
    seq = torch.bucketize(tok, cu[1:], right=True)
    local = tok - cu[seq]
    st["u"][: st["total"]] = u[seq, local].to(torch.bfloat16)
    st["lse"][: st["total"]] = lse[seq, local]
    return {"u": st["u"], "lse": st["lse"]}


def _plain_accept(st):
    page, o, cu, lens = st["page"], st["out"], st["cu"].long(), st["seqlens"].long()
    n, node = cu[1:] - cu[:-1], st["accepted"].long()
    i = torch.arange(64, device=DEV)
    mask = st["mask"][(cu[:-1] + node.clamp(min=0)).clamp(max=len(st["mask"]) - 1)]
    on = (((mask[:, None] >> i) & 1) == 1) & (i < n[:, None]) & (node >= 0)[:, None]
    kept = on.sum(1)
    to = torch.cumsum(on, 1) - 1

    def row(p):
        p = p.clamp(min=0)
        return torch.gather(st["table"].long(), 1, (p // page).clamp(max=st["table"].shape[1] - 1)) * page + p % page

    base = (lens - n)[:, None]
    path = torch.full((len(n), 65), -1, dtype=torch.int64, device=DEV)
    path.scatter_(1, torch.where(on, to, 64), i.expand_as(on))
    path = path[:, :64]
    # a place without a token to move repeats its tree's first move, or leaves one of the request's own rows as it is
    some = torch.where((kept > 0)[:, None], path[:, :1], 0)
    base = torch.minimum(base, lens[:, None] - 1)
    moved = i < kept[:, None]
    src, dst = row(base + torch.where(moved, path, some)), row(base + torch.where(moved, i, 0))
    st["cache"][dst] = st["cache"][src]
    o["seqlens"].copy_(lens - n + kept)
    tok = torch.arange(len(o["path"]), device=DEV)
    seq = torch.bucketize(tok, cu[1:], right=True)
    live, seq = seq < len(n), seq.clamp(max=len(n) - 1)
    o["path"].copy_(torch.where(live, path[seq, (tok - cu[seq]).clamp(0, 63)].to(torch.int32), o["path"]))
    return {"cache": st["cache"], **o}


def run(st):
    if own:
        from mla_latent_kv_23_b200 import mla
        if st["op"] == "append":
            mla.mla_append_latent_slots(st["h"], st["w_dkv"], st["w_kr"], st["slots"], st["pos"], st["cache"], rope_base=ROPE_BASE)
            return {"cache": st["cache"]}
        if st["op"] == "tables":
            mla.mla_build_tables(st["p"])
            return {"table": st["table"], **st["out"]}
        if st["op"] == "accept":
            mla.mla_accept_tree(st["p"])
            return {"cache": st["cache"], **st["out"]}
        mla.mla_decode_tree(st["p"], st["ws"])
        return {"u": st["u"], "lse": st["lse"]}
    return {"append": _plain_append, "tables": _plain_tables, "tree": _plain_tree, "accept": _plain_accept}[st["op"]](st)


# -------------------------------------------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    """The operators' definitions, request by request and token by token."""
    st = prepare(case, seed)
    if case["op"] == "append":
        cache, x, pos = st["cache"].double(), st["h"].double(), st["pos"].tolist()
        new = torch.cat([x @ st["w_dkv"].double().T, x @ st["w_kr"].double().T], 1)
        turn = torch.tensor([[p / ROPE_BASE ** (2 * k / D_R) for k in range(D_R // 2)] for p in pos], dtype=torch.float64, device=DEV)
        z = torch.complex(new[:, D_C::2], new[:, D_C + 1 :: 2]) * torch.polar(torch.ones_like(turn), turn)
        new[:, D_C:] = torch.view_as_real(z).flatten(1)
        for t, r in enumerate(st["slots"].tolist()):
            cache[r] = new[t]
        return {"cache": cache}
    cu = st["cu"].tolist()
    page = case["page"]
    if case["op"] == "tables":
        out = {k: v.cpu().numpy().copy() for k, v in st["out"].items()}
        table, free, used = st["table"].cpu().numpy().copy(), st["free"].tolist(), st["free_used"].item()
        parents = None if st["parents"] is None else st["parents"].tolist()
        for b, (ctx, new) in enumerate(zip(st["ctx"].tolist(), st["new"].tolist())):
            for k in range(-(-ctx // page), -(-(ctx + new) // page)):
                table[b, k] = free[used]
                used += 1
            out["seqlens"][b], out["cu"][b + 1] = ctx + new, cu[b + 1]
            at = slice(cu[b], cu[b + 1])
            p = ctx + np.arange(new)
            out["seq_ids"][at], out["slots"][at], out["pos"][at] = b, table[b, p // page] * page + p % page, p
            if parents is not None:
                out["tree_mask"][at] = 0
                branch, depth = [], []
                for i in range(new if new <= 64 else 0):
                    up = parents[cu[b] + i]
                    branch.append((branch[up] if up >= 0 else 0) | 1 << i)
                    depth.append(depth[up] + 1 if up >= 0 else 0)
                    out["tree_mask"][cu[b] + i] = branch[-1] - (1 << 64 if branch[-1] >> 63 else 0)
                    out["pos"][cu[b] + i] = ctx + depth[-1]
        out["free_used"][0] = used
        return {"table": table, **out}
    lens, table, masks = st["seqlens"].tolist(), st["table"], st["mask"].tolist()

    def row(b, p):
        return table[b].long()[p // page] * page + p % page

    if case["op"] == "accept":
        out = {k: v.cpu().numpy().copy() for k, v in st["out"].items()}
        cache = st["cache"].double()
        for b, node in enumerate(st["accepted"].tolist()):
            n = cu[b + 1] - cu[b]
            path = [i for i in range(n) if node >= 0 and masks[cu[b] + node] >> i & 1]
            out["path"][cu[b] : cu[b + 1]] = path + [-1] * (n - len(path))
            out["seqlens"][b] = lens[b] - n + len(path)
            if path:
                base = lens[b] - n
                cache[row(b, torch.arange(base, base + len(path), device=DEV))] = cache[row(b, base + torch.tensor(path, device=DEV))]
        return {"cache": cache, **out}
    u, lse = st["u"].double(), st["lse"].double()
    for b, n in enumerate(lens):
        t = cu[b + 1] - cu[b]
        if not t:
            continue
        kv = st["cache"][row(b, torch.arange(n, device=DEV))].double()
        i = torch.arange(t, device=DEV)
        seen = torch.ones((t, n), dtype=torch.bool, device=DEV)
        seen[:, n - t :] = ((st["mask"][cu[b] : cu[b + 1], None] >> i) & 1) == 1
        # eight heads at a time bound the scores' memory
        for h in range(0, case["heads"], 8):
            q = st["q"][cu[b] : cu[b + 1], h : h + 8].double()
            s = torch.einsum("thw,nw->thn", q, kv) * SCALE
            s = torch.where(seen[:, None], s, -math.inf)
            lse[cu[b] : cu[b + 1], h : h + 8] = torch.logsumexp(s, -1)
            u[cu[b] : cu[b + 1], h : h + 8] = torch.einsum("thn,nd->thd", torch.nan_to_num(torch.softmax(s, -1)), kv[:, :D_C])
    return {"u": u, "lse": lse}
