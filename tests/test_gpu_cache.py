"""The paged cache's lengths, pages and slots against a cache kept sequence
by sequence (decode_model.CacheModel), the moves of a tree's accepted path,
and a run of all of them around the verify step as a decode loop uses them."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from decode_model import CacheModel
from workload import WORKLOADS, make_inputs, make_tree_inputs

pytestmark = pytest.mark.gpu

_SKIP = not torch.cuda.is_available()


@pytest.fixture(scope="module")
def sv():
    if _SKIP:
        pytest.skip("no GPU")
    import draft_token_verification_03_amd as sv
    sv.load_library()
    return sv


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def setup(rng, B, page, blocks, spare, lengths):
    """Tables for these lengths in random pages, and the free list."""
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    tables, at = np.full((B, blocks), -1, dtype=np.int32), 0
    for b, n in enumerate(need):
        tables[b, :n] = order[at:at + n]
        at += n
    free = np.full(max(pages, 1), -5, dtype=np.int32)
    free[:spare] = order[at:]
    return tables, free, spare, pages


EXTEND = [(1, 1, 4, 4, 100), (5, 16, 8, 6, 100), (64, 16, 32, 7, 100), (300, 8, 20, 33, 100), (1500, 4, 12, 5, 100),
          (7, 64, 40, 2000, 100), (40, 16, 100, 900, 100), (20, 16, 30, 40, 30), (50, 1, 60, 8, 50), (3, 5, 7, 0, 0), (1024, 8, 9, 12, 90),
          (1025, 8, 9, 12, 100), (5000, 4, 12, 5, 100), (2, 128, 200, 20000, 100)]


@pytest.mark.parametrize("B,page,blocks,most,share", EXTEND)
def test_extend_matches_the_model(sv, B, page, blocks, most, share):
    """share: how many of a hundred needed pages the free list holds."""
    rng = np.random.default_rng(B + most)
    new = rng.integers(0, most + 1, B)
    length = rng.integers(0, blocks * page - most + 1, B)
    need = sum(-(-(s + n) // page) - -(-s // page) for s, n in zip(length, new))
    tables, free, spare, pages = setup(rng, B, page, blocks, need * share // 100 + (2 if share == 100 else 0), length)
    total = int(new.sum()) + 3
    model = CacheModel(length, tables, free[:spare], page, blocks, pages)
    slots, pos, ids, start, granted, bad, lack = model.extend(new, total)
    table, count = i32(tables), i32([spare])
    out = torch.empty(1, dtype=torch.int32, device="cuda")
    call = sv.CacheExtend(i32(length), table, i32(free), count, page, total, new_len=i32(new), free_count_out=out)
    for _ in range(2):  # not in place: the same again
        got = [x.cpu().numpy().tolist() for x in call()]
        assert got == [slots, pos, ids, start, granted]
        assert table.cpu().numpy().tolist() == model.tables
        assert int(out) == len(model.free) and int(count) == spare
    assert int(call.error_word) == (sv.SV_ERR_LENGTH if bad else 0) | (sv.SV_ERR_PAGES if lack else 0)
    assert lack == (share < 100 and need > 0)


def test_extend_extra_and_refused_sequences(sv):
    """new_len + extra, lengths that do not fit, too few token slots."""
    page, blocks = 4, 3
    length, new = [3, -1, 11, 0, 5, 12], [1, 2, 1, -3, -2, -2]
    rng = np.random.default_rng(0)
    tables, free, spare, pages = setup(rng, 6, page, blocks, 9, [3, 0, 11, 0, 5, 12])
    for total in (12, 2):
        model = CacheModel(length, tables, free[:spare], page, blocks, pages)
        want = model.extend([n + 2 for n in new], total)
        table, count = i32(tables), i32([spare])
        call = sv.CacheExtend(i32(length), table, i32(free), count, page, total, new_len=i32(new), extra=2)
        got = [x.cpu().numpy().tolist() for x in call()]
        assert got == list(want[:5])
        assert table.cpu().numpy().tolist() == model.tables
        assert int(count) == len(model.free)  # in place
        assert int(call.error_word) == sv.SV_ERR_LENGTH


def test_extend_bad_pages_and_counts(sv):
    """A page outside the pool, in the free list or the table, gives no slot;
    a count outside the list is held within it."""
    page = 4
    table = i32([[99, -1], [2, -1]])
    free = i32([7, -3, 1])
    call = sv.CacheExtend(i32([3, 4]), table, free, i32([2]), page, 4, new_len=i32([1, 3]))
    slots = call()[0].cpu().tolist()
    assert slots == [-1, -1, -1, -1] and int(call.error_word) == sv.SV_ERR_PAGE
    for count, want in ((50, [4, 5]), (-2, [-1, -1])):
        call = sv.CacheExtend(i32([0]), i32([[-1]]), free, i32([count]), page, 2, extra=2)
        assert call()[0].cpu().tolist() == want
        assert int(call.error_word) & sv.SV_ERR_PAGES


COMMIT = [(1, 1, 4, 4, 0.0), (5, 16, 8, 6, 0.0), (64, 16, 32, 7, 0.3), (300, 8, 20, 33, 0.1), (1500, 4, 50, 9, 0.2),
          (2000, 16, 40, 8, 0.05), (3, 64, 9, 500, 1.0), (1024, 8, 100, 20, 0.4), (1025, 8, 9, 12, 0.5), (5000, 4, 20, 5, 0.1)]


@pytest.mark.parametrize("B,page,blocks,most,ended", COMMIT)
def test_commit_matches_the_model(sv, B, page, blocks, most, ended):
    rng = np.random.default_rng(B + most)
    reserved = rng.integers(0, most + 1, B)
    length = rng.integers(0, blocks * page - most + 1, B)
    accepted = np.array([rng.integers(-1, r) if r else -1 for r in reserved])
    fin = (rng.random(B) < ended).astype(np.int32)
    held = length + reserved
    tables, free, spare, pages = setup(rng, B, page, blocks, 5, held)
    for finished in (None, fin):
        model = CacheModel(length, tables, free[:spare], page, blocks, pages)
        model.commit(reserved, accepted, finished=finished)
        lens, flist, count = i32(length), i32(free), i32([spare])
        out_len, out_count = torch.empty_like(lens), torch.empty_like(count)
        f = None if finished is None else i32(finished)
        call = sv.CacheCommit(lens, i32(reserved), i32(accepted), i32(tables), flist, count, page, finished=f,
                              seq_len_out=out_len, free_count_out=out_count)
        for _ in range(2):
            call()
            n = int(out_count)
            assert out_len.cpu().tolist() == model.seq_len
            assert n == len(model.free) and flist.cpu().tolist()[:n] == model.free
            assert flist.cpu().tolist()[n:] == free.tolist()[n:]  # behind the list: as it was
        assert int(call.error_word) == 0
        # in place
        call = sv.CacheCommit(lens, i32(reserved), i32(accepted), i32(tables), flist, count, page, finished=f)
        call()
        assert lens.cpu().tolist() == model.seq_len and int(count) == n


def test_commit_clamps_and_reports(sv):
    page, blocks = 4, 3
    length, reserved, accepted = [4, 4, 4, -1, 10], [3, 3, 0, 2, 9], [7, -5, 0, 1, 1]
    tables = [[0, 1, -1], [2, 3, -1], [4, -1, -1], [5, -1, -1], [6, 7, 8]]
    free = [9] + [-5] * 9
    model = CacheModel(length, tables, free[:1], page, blocks, 10)
    assert model.commit(reserved, accepted)
    lens, flist, count = i32(length), i32(free), i32([1])
    call = sv.CacheCommit(lens, i32(reserved), i32(accepted), i32(tables), flist, count, page)
    call()
    assert int(call.error_word) == sv.SV_ERR_LENGTH
    assert lens.cpu().tolist() == model.seq_len == [7, 4, 4, -1, 10]
    assert flist.cpu().tolist()[:int(count)] == model.free == [9, 3]
    # a bad page goes back as -1; a full list takes no more
    for tab, cnt, want, bits in (([[0, 77]], 0, [-1, -5], sv.SV_ERR_PAGE), ([[0, 1]], 2, [-5, -5], sv.SV_ERR_PAGES)):
        flist, count = i32([-5, -5]), i32([cnt])
        call = sv.CacheCommit(i32([4]), i32([2]), i32([-1]), i32(tab), flist, count, page)
        call()
        assert flist.cpu().tolist() == want and int(call.error_word) == bits
        assert int(count) == (1 if cnt == 0 else 2)


def test_extend_then_giving_all_back_restores_the_list(sv):
    rng = np.random.default_rng(4)
    B, page, blocks = 70, 8, 30
    length, new = rng.integers(0, 100, B), rng.integers(0, 60, B)
    tables, free, spare, pages = setup(rng, B, page, blocks, 900, length)
    lens, table, flist, count = i32(length), i32(tables), i32(free), i32([spare])
    ext = sv.CacheExtend(lens, table, flist, count, page, 70 * 60, new_len=i32(new))
    granted = ext()[4]
    assert int(count) < spare
    sv.cache_commit(lens, granted, i32([-1] * B), table, flist, count, page)
    assert int(count) == spare and flist.cpu().tolist() == free.tolist() and lens.cpu().tolist() == length.tolist()


COMPACT = [(1, 2, 5, 1, 16, 64, torch.bfloat16), (3, 4, 20, 2, 8, 40, torch.float32), (130, 2, 9, 1, 4, 16, torch.float32),
           (2, 3, 128, 1, 16, 24, torch.float16), (1, 5, 12, 3, 5, 3, torch.uint8), (2, 64, 60, 4, 16, 136, torch.bfloat16)]


@pytest.mark.parametrize("L,B,N,G,page,D,dtype", COMPACT)
def test_compact_moves_the_path(sv, L, B, N, G, page, D, dtype):
    rng = np.random.default_rng(L + N)
    blocks = -(-(N + 40) // page)
    length = rng.integers(0, blocks * page - N, B)
    tables, _, _, pages = setup(rng, B, page, blocks, 2, length + N + 1)
    d = rng.integers(0, N + 1, B)
    path = np.full((B, N), -1, dtype=np.int32)
    for b in range(B):
        path[b, :d[b]] = np.sort(rng.permutation(N)[:d[b]])
    x = torch.randint(0, 255, (L, pages, G, page, D), device="cuda").to(dtype)
    y, want = x.clone(), x.clone()
    call = sv.CacheCompact(y, i32(tables), i32(length), i32(path), i32(d))
    call()
    for b in range(B):
        for i in range(d[b]):
            s, t = length[b] + 1 + path[b, i], length[b] + 1 + i
            want[:, tables[b, t // page], :, t % page] = x[:, tables[b, s // page], :, s % page]
    assert int(call.error_word) == 0 and torch.equal(y, want)


def test_compact_refuses_bad_paths_lengths_and_pages(sv):
    page, blocks = 4, 3
    tables = np.arange(6 * blocks, dtype=np.int32).reshape(6, blocks)
    x = torch.randn(18, 1, page, 8, device="cuda")
    path = [[1, 1, -1], [2, 1, -1], [0, 3, -1], [0, 2, -1], [1, 2, -1], [0, 2, -1]]
    length = [0, 0, 0, 9, -1, 0]
    acc = [2, 2, 2, 2, 2, 4]
    y = x.clone()
    call = sv.CacheCompact(y, i32(tables), i32(length), i32(path), i32(acc))
    call()
    assert int(call.error_word) == sv.SV_ERR_TREE | sv.SV_ERR_LENGTH and torch.equal(x, y)
    bad = i32([[0, 77, 2]])  # positions 4..7 in no page
    call = sv.CacheCompact(y, bad, i32([0]), i32([[2, 3, 4, 7, -1, -1, -1, -1]]), i32([4]))
    call()
    want = x.clone()
    want[0, :, 1] = x[0, :, 3]  # node 2: position 3 -> 1; 4 and 5 stay away; node 7: 8 -> page 77
    assert int(call.error_word) == sv.SV_ERR_PAGE and torch.equal(y, want)


def write_tokens(pool, slots, marks):
    """What a forward pass does: each token's row into its slot."""
    ok = slots >= 0
    flat = pool.view(-1, pool.shape[-1])
    flat[slots[ok]] = marks[ok].unsqueeze(1).expand(-1, pool.shape[-1])


def rows_of(cache, pool, b):
    n, page = int(cache.seq_len[b]), cache.page_size
    t = cache.block_table[b].long()
    s = torch.arange(n, device="cuda")
    return pool.view(-1, pool.shape[-1])[t[s // page] * page + s % page, 0].cpu().tolist()


@pytest.mark.parametrize("name,beta", [("C2", 1.0), ("C5", 0.5)])
def test_decode_rounds_with_a_cache(sv, name, beta):
    """Rounds of extend, forward pass (marks in slots), verify and commit: the
    cache holds exactly the kept tokens' marks, in order, and no page is lost."""
    w = WORKLOADS[name].sized(B=9, V=1009, beta=beta)
    cache = sv.PagedCache(w.B, 20, 9 * 20 + 1, 4)
    pool = torch.full((cache.num_pages, 1, 4, 8), -1.0, device="cuda")
    draft_len = torch.zeros(w.B, dtype=torch.int32, device="cuda")
    ext = cache.extender(w.B * (w.K + 1), new_len=draft_len, extra=1)
    held = [[] for _ in range(w.B)]
    for r in range(8):
        inp = make_inputs(w, seed=50 + r, device="cuda")
        draft_len.copy_(torch.randint(0, w.K + 1, (w.B,), device="cuda"))
        slots, pos, ids, start, granted = ext()
        marks = torch.arange(slots.numel(), device="cuda", dtype=torch.float32) + 1000 * (r + 1)
        write_tokens(pool, slots, marks)
        v = sv.Verifier(inp["target"], inp["draft"], inp["tokens"], inp["temperature"], inp["beta"],
                        draft_len=draft_len, cache=cache)
        acc, _ = v(r)
        acc, start = acc.cpu().tolist(), start.cpu().tolist()
        for b in range(w.B):
            held[b] += marks[start[b]:start[b] + acc[b] + 1].cpu().tolist()
            assert rows_of(cache, pool, b) == held[b]
    assert int(cache.error_word) == 0
    used = sum(-(-len(h) // 4) for h in held)
    assert int(cache.free_count) == cache.num_pages - used
    # the end of every sequence gives all pages back
    fin = torch.ones(w.B, dtype=torch.int32, device="cuda")
    cache.reserved.zero_()
    cache.committer(i32([-1] * w.B), finished=fin)()
    assert int(cache.free_count) == cache.num_pages and cache.seq_len.cpu().tolist() == [0] * w.B
    assert sorted(cache.free_list.cpu().tolist()) == list(range(cache.num_pages))


def test_rounds_when_pages_run_out(sv):
    """Sequences without their pages keep nothing and lose nothing; once others
    have ended they go on."""
    w = WORKLOADS["C2"].sized(B=6, V=509)
    cache = sv.PagedCache(w.B, 10, 13, 4)
    inp = make_inputs(w, seed=3, device="cuda")
    ext = cache.extender(w.B * (w.K + 1), extra=w.K + 1)
    v = sv.Verifier(inp["target"], inp["draft"], inp["tokens"], inp["temperature"], cache=cache)
    lens, lacked = [0] * w.B, False
    for r in range(5):
        slots, _, _, start, granted = ext()
        granted, start, slots = granted.cpu().tolist(), start.cpu().tolist(), slots.cpu().tolist()
        lacked |= 0 in granted
        held = [s for s in slots if s >= 0]
        assert len(set(held)) == len(held)
        for b in range(w.B):
            mine = slots[start[b]:start[b + 1]]
            assert (min(mine) >= 0) if granted[b] else (max(mine) == -1)
        acc = v(r)[0].cpu().tolist()
        for b in range(w.B):
            lens[b] += acc[b] + 1 if granted[b] else 0
        assert cache.seq_len.cpu().tolist() == lens
        assert int(cache.free_count) == 13 - sum(-(-n // 4) for n in lens)
    assert lacked and int(cache.error_word) == sv.SV_ERR_PAGES
    done = i32([1, 1, 1, 0, 0, 0])
    cache.reserved.zero_()
    cache.committer(i32([-1] * w.B), finished=done)()
    # (the ended ones get no tokens: 13 pages hold three sequences of up to 16)
    assert max(lens[3:]) + w.K + 1 <= 16
    more = cache.extender(w.B * (w.K + 1), new_len=i32([-w.K - 1] * 3 + [0] * 3), extra=w.K + 1)
    assert more()[4].cpu().tolist() == [0] * 3 + [w.K + 1] * 3


def test_tree_rounds_with_a_cache(sv):
    """The same for trees: the accepted path's rows follow the root's."""
    w = WORKLOADS["C4"].sized(B=6, V=503)
    shape = (3, 2, 1)
    cache = sv.PagedCache(w.B, 24, 6 * 24, 4)
    pools = torch.full((3, cache.num_pages, 1, 4, 8), -1.0, device="cuda")
    inp = make_tree_inputs(w, shape, seed=1, device="cuda")
    N = inp["parent"].shape[1]
    ext = cache.extender(w.B * (N + 1), extra=N + 1)
    held = [[] for _ in range(w.B)]
    for r in range(5):
        inp = make_tree_inputs(w, shape, seed=60 + r, device="cuda")
        slots, *_ = ext()
        marks = torch.arange(slots.numel(), device="cuda", dtype=torch.float32) + 1000 * (r + 1)
        for k in range(3):
            write_tokens(pools[k], slots, marks + k * 100000)
        v = sv.TreeVerifier(inp["target"], inp["draft"], inp["parent"], inp["tokens"], inp["temperature"], cache=cache,
                            pools=pools)
        acc, _, path, err = v(r)
        acc, path = acc.cpu().tolist(), path.cpu().tolist()
        assert int(err) == 0
        for b in range(w.B):
            at = b * (N + 1)
            held[b] += [1000 * (r + 1) + at] + [1000 * (r + 1) + at + 1 + p for p in path[b][:acc[b]]]
            for k in range(3):
                assert rows_of(cache, pools[k], b) == [x + k * 100000 for x in held[b]]
    assert int(cache.error_word) == 0


def test_cache_calls_captured(sv):
    """extend, compact and commit in one graph, replayed as rounds."""
    B, N, page = 5, 6, 4
    st = torch.cuda.Stream()
    cache = sv.PagedCache(B, 40, 5 * 40, page)
    ref = sv.PagedCache(B, 40, 5 * 40, page)
    pool = torch.zeros(2, cache.num_pages, 1, page, 8, device="cuda")
    pool_ref = pool.clone()
    path, acc = torch.full((B, N), -1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    calls = [cache.extender(B * (N + 1), extra=N + 1, stream=st), cache.compactor(pool, path, acc, stream=st),
             cache.committer(acc, stream=st)]
    calls_ref = [ref.extender(B * (N + 1), extra=N + 1), ref.compactor(pool_ref, path, acc), ref.committer(acc)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        for c in calls:
            c()
    for r in range(6):
        rng = np.random.default_rng(r)
        d = rng.integers(0, N + 1, B)
        p = np.full((B, N), -1)
        for b in range(B):
            p[b, :d[b]] = np.sort(rng.permutation(N)[:d[b]])
        path.copy_(i32(p))
        acc.copy_(i32(d))
        pool.normal_()
        pool_ref.copy_(pool)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for c in calls_ref:
            c()
        torch.cuda.synchronize()
        for x, y in ((cache.seq_len, ref.seq_len), (cache.block_table, ref.block_table), (cache.free_list, ref.free_list),
                     (cache.free_count, ref.free_count), (calls[0].slots, calls_ref[0].slots), (pool, pool_ref)):
            assert torch.equal(x, y), r
    assert int(cache.error_word) == int(ref.error_word) == 0


def test_empty_batch_and_slots_beyond_32_bits(sv):
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    slots, pos, ids, start, granted = sv.cache_extend(none, torch.zeros((0, 4), dtype=torch.int32, device="cuda"),
                                                      i32([0]), i32([1]), 4, 3, extra=1)
    assert slots.tolist() == [-1] * 3 and pos.tolist() == [0] * 3 and ids.tolist() == [-1] * 3 and start.tolist() == [0]
    assert granted.numel() == 0
    pages = (1 << 27) + 2
    free = torch.zeros(pages, dtype=torch.int32, device="cuda")
    free[0] = 1 << 27
    table = torch.full((1, 2), -1, dtype=torch.int32, device="cuda")
    call = sv.CacheExtend(i32([0]), table, free, i32([1]), 64, 3, extra=3)
    assert call()[0].tolist() == [(1 << 33) + k for k in range(3)] and int(call.error_word) == 0
    assert table.tolist() == [[1 << 27, -1]]
