"""The state that a speculative-decoding step hands to the next one (lengths,
pages held, entries of the free list in use), through steps that refuse a
request as well."""
import numpy as np
import pytest
import torch

from mla_latent_kv_23_b200 import mla

pytestmark = pytest.mark.gpu

PAGE, MAX_PAGES = 64, 4
ROOM = 2048


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def flags():
    try:
        return mla.mla_check_device_errors()
    except mla.MLAError as e:
        return e.flags


def tables(table, free, ctx, new, held, used, num_pages=256):
    """One step from the given state: (state after it, slots, cu_new, flags)."""
    B = len(ctx)
    o = {k: torch.full((n,), -7, dtype=torch.int32, device="cuda")
         for k, n in (("used", 1), ("lens", B), ("cu", B + 1), ("seq", ROOM), ("pos", ROOM), ("slots", ROOM), ("held", B))}
    mla.mla_build_tables(mla.tables_params(
        i32(ctx), i32(new), table, i32(free), i32([used]), o["used"], o["lens"], o["cu"], o["seq"], o["pos"],
        o["slots"], PAGE, num_pages, pages_held=i32(held), pages_held_out=o["held"]))
    f = flags()
    state = dict(lens=o["lens"].tolist(), held=o["held"].tolist(), used=o["used"].item())
    return state, o["slots"].tolist(), o["cu"].tolist(), f


def held_pages(table, held):
    t = table.tolist()
    return [p for b, n in enumerate(held) for p in t[b][:n]]


def rows(table, b, first, n):
    t = table.tolist()[b]
    return [t[p // PAGE] * PAGE + p % PAGE for p in range(first, first + n)]


def test_a_refused_request_keeps_its_length_and_pages():
    table = torch.full((3, MAX_PAGES), -1, dtype=torch.int32, device="cuda")
    free = np.random.default_rng(0).permutation(40)
    s, _, _, f = tables(table, free, [0, 0, 0], [100, 200, 130], [0, 0, 0], 0)
    assert f == 0 and s == dict(lens=[100, 200, 130], held=[2, 4, 3], used=9)
    before = table.tolist()[1]
    # 300 tokens do not fit four pages; a negative number of new ones
    for new, end in (([10, 100, 5], [110, 200, 135]), ([0, -1, 1], [110, 200, 136])):
        s, slots, cu, f = tables(table, free, s["lens"], new, s["held"], s["used"])
        assert f == mla.DEVFLAG_BAD_SEQLEN
        assert s == dict(lens=end, held=[2, 4, 3], used=9) and table.tolist()[1] == before
        assert cu == [0, new[0], new[0], new[0] + new[2]]
        assert slots[:cu[3]] == rows(table, 0, end[0] - new[0], new[0]) + rows(table, 2, end[2] - new[2], new[2])
    s, slots, cu, f = tables(table, free, s["lens"], [60, 20, 70], s["held"], s["used"])
    assert f == 0 and s == dict(lens=[170, 220, 206], held=[3, 4, 4], used=11)
    assert table.tolist()[1] == before and sorted(held_pages(table, s["held"])) == sorted(free[:11].tolist())
    assert slots[:150] == rows(table, 0, 110, 60) + rows(table, 1, 200, 20) + rows(table, 2, 136, 70)


def test_a_wrong_length_keeps_the_pages():
    # the length itself is wrong (negative, past the block table, past what the
    # request holds): it cannot be carried on, the pages can
    table = i32(np.arange(16).reshape(4, MAX_PAGES))
    s, _, cu, f = tables(table, [20, 21], [-3, 300, 200, 64], [1, 1, 1, 1], [2, 4, 3, 1], 0)
    assert f == mla.DEVFLAG_BAD_SEQLEN and cu == [0, 0, 0, 0, 1]
    assert s == dict(lens=[0, 0, 0, 65], held=[2, 4, 3, 2], used=1)
    assert table.tolist() == [[0, 1, 2, 3], [4, 5, 6, 7], [8, 9, 10, 11], [12, 20, 14, 15]]
    # a number of pages that no block table row has is none
    s, _, _, f = tables(table[:2], [20, 21], [5, 5], [1, 1], [-1, 5], 0)
    assert f == mla.DEVFLAG_BAD_SEQLEN and s == dict(lens=[0, 0], held=[0, 0], used=0)


def test_any_steps_lose_no_page():
    # requests grow, are refused, lose rejected tokens; whatever happens, the
    # pages taken from the list are the pages held
    rng = np.random.default_rng(7)
    B = 50
    table = torch.full((B, MAX_PAGES), -1, dtype=torch.int32, device="cuda")
    free = rng.permutation(256)[:B * MAX_PAGES]
    lens, held, used = [0] * B, [0] * B, 0
    refused = 0
    for _ in range(30):
        new = rng.integers(-1, 40, B)
        new[rng.random(B) < 0.1] = 300
        before = table.tolist()
        s, _, _, f = tables(table, free, lens, new, held, used)
        want = []
        for b in range(B):
            bad = new[b] < 0 or lens[b] + new[b] > MAX_PAGES * PAGE
            refused += bad
            want.append(lens[b] if bad else lens[b] + int(new[b]))
            assert s["held"][b] == max(held[b], -(-want[b] // PAGE))
            assert table.tolist()[b][:held[b]] == before[b][:held[b]]
        assert s["lens"] == want and f & ~mla.DEVFLAG_BAD_SEQLEN == 0
        assert sorted(held_pages(table, s["held"])) == sorted(free[:s["used"]].tolist())
        lens = [max(0, n - int(rng.integers(0, 30))) for n in want]
        held, used = s["held"], s["used"]
    assert refused > 100 and max(held) == MAX_PAGES


def test_pages_that_ran_out_are_not_held():
    # five of eight pages: the last request gets two of its five
    table = torch.full((3, 5), -1, dtype=torch.int32, device="cuda")
    s, slots, cu, f = tables(table, [9, 3, 7, 5, 1], [0, 0, 0], [100, 10, 300], [0, 0, 0], 0)
    assert f == mla.DEVFLAG_NO_PAGES
    assert s == dict(lens=[100, 10, 300], held=[2, 1, 2], used=5)
    assert table.tolist() == [[9, 3, -1, -1, -1], [7, -1, -1, -1, -1], [5, 1, -1, -1, -1]]
    assert slots[110:410] == rows(table, 2, 0, 128) + [-1] * 172
    # again with a longer list, from the lengths before: it keeps the two and gets three more
    s, slots, _, f = tables(table, [9, 3, 7, 5, 1, 8, 6, 4, 2], [100, 10, 0], [0, 0, 300], s["held"], s["used"])
    assert f == 0 and s == dict(lens=[100, 10, 300], held=[2, 1, 5], used=8)
    assert table.tolist()[2] == [5, 1, 8, 6, 4] and slots[:300] == rows(table, 2, 0, 300)


def test_nothing_free_adds_no_page():
    for used in (2, 5, -1):  # the list is used up, or its count is out of range
        table = torch.full((2, 5), -1, dtype=torch.int32, device="cuda")
        table[:, 0] = i32([11, 12])
        s, _, _, f = tables(table, [9, 3], [64, 60], [200, 4], [1, 1], used)
        assert f == mla.DEVFLAG_NO_PAGES and s == dict(lens=[264, 64], held=[1, 1], used=2)
        assert table.tolist() == [[11, -1, -1, -1, -1], [12, -1, -1, -1, -1]]


def test_accept_of_wrong_input():
    before = torch.randn((256, 576), device="cuda").to(torch.bfloat16)
    mask = torch.full((8,), 0b11010, dtype=torch.int64, device="cuda")

    def accept(cu, lens, accepted):
        cache, out, path = before.clone(), i32([-7, -7]), i32([-7] * 8)
        mla.mla_accept_tree(mla.accept_params(cache, i32([[0, 1], [2, 3]]), i32(lens), i32(cu), mask, i32(accepted), out, path, PAGE))
        f = flags()
        assert torch.equal(cache, before)
        return out.tolist(), path.tolist(), f

    # which rows are a tree's is not known: nothing is done for it
    for cu, accepted in (([0, 9, 8], [3, 1]), ([-1, 4, 2], [3, 1]), ([0, 9, 9], [-1, -1]), ([3, 2, 9], [0, 0])):
        out, path, f = accept(cu, [100, 50], accepted)
        assert f == mla.DEVFLAG_BAD_TREE and out == [100, 50] and path == [-7] * 8
    # its rows in the cache are not known: nothing is kept on the path, the length stays
    out, path, f = accept([0, 5, 8], [129, 2], [4, 1])
    assert f == mla.DEVFLAG_BAD_SEQLEN and out == [129, 2] and path == [-1] * 8
    # only the accepted token is wrong: the tree is dropped
    out, path, f = accept([0, 5, 8], [100, 50], [5, -2])
    assert f == mla.DEVFLAG_BAD_TREE and out == [95, 47] and path == [-1] * 8


def test_accept_of_a_prompt():
    # 65 rows are no tree: flagged, and the cache, the path and the length stay
    cache = torch.randn((256, 576), device="cuda").to(torch.bfloat16)
    before, mask = cache.clone(), torch.full((68,), 0b110, dtype=torch.int64, device="cuda")
    out, path = i32([-7, -7]), i32([-7] * 68)
    mla.mla_accept_tree(mla.accept_params(cache, i32([[0, 1], [2, 3]]), i32([70, 80]), i32([0, 65, 68]), mask,
                                          i32([-1, 2]), out, path, PAGE))
    assert flags() == mla.DEVFLAG_BAD_TREE
    assert out.tolist() == [70, 79] and path.tolist() == [-7] * 65 + [1, 2, -1]
    want = before.clone()
    want[128 + 77], want[128 + 78] = before[128 + 78], before[128 + 79]
    assert torch.equal(cache, want)
