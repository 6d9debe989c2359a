"""The latent cache's calls where they can go wrong: pages smaller than a load, runs of consecutive rows, pools beyond
4 GiB, rows that no sequence holds, tiles of very different scales, operands that are not finite."""
import math

import pytest
import torch

import sparse_attention_decode_lightning_b200 as dsa
from tests._latent import D, DV, Cache, attend_reference, check_attend, codes_to_double
from tests.test_gpu_attend import DEV, SCALE, check_sinks, ints, queries, run_sinks, run_sparse
from tests.test_gpu_latent_append import check, inputs, inv_freq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [128, 64])
@pytest.mark.parametrize("e4m3,page,block", [(False, 1, 1), (False, 2, 1), (False, 8, 1), (True, 1, 1), (True, 8, 4),
                                             (True, 8, 8)])
def test_pages_smaller_than_a_load(heads, e4m3, page, block):
    vis = [1, 7, 9, 130, 517]
    cache = Cache(vis, page, e4m3, block, seed=page + heads)
    check_sinks(cache, queries(cache, len(vis), heads), cache.offsets([1] * len(vis)), ints(vis), 3, 222)


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_pool_of_few_rows(e4m3):
    """Fewer rows in the pool than a load of a run brings."""
    for n in (1, 2, 5):
        cache = Cache([n], 1, e4m3, 1, seed=n)
        cache.pool = cache.pool[:cache.num_pages].contiguous()
        check_sinks(cache, queries(cache, 1, 64), cache.offsets([1]), ints([n]), 0, n)


def in_order(cache):
    """The same sequences in a pool whose pages follow one another: runs go over their ends."""
    other = object.__new__(Cache)
    other.__dict__.update(cache.__dict__)
    held = cache.table[cache.table >= 0].long()
    rest = [p for p in range(cache.num_pages) if p not in set(held.tolist())]
    order = torch.cat([held, torch.tensor(rest, dtype=torch.long, device=DEV)])
    other.pool = cache.pool[order].contiguous()
    other.scales = None if cache.scales is None else cache.scales[order].contiguous()
    other.table = cache.table.clone()
    other.table[cache.table >= 0] = torch.arange(held.numel(), dtype=torch.int32, device=DEV)
    return other


@pytest.mark.parametrize("heads", [128, 64])
@pytest.mark.parametrize("e4m3,page,block", [(False, 4, 1), (False, 8, 1), (False, 16, 1), (True, 4, 4), (True, 16, 16)])
def test_order_of_the_pages_changes_no_bit(heads, e4m3, page, block):
    """Consecutive rows come by other loads than scattered ones, to the same places."""
    lens = [300, 1, 1033, 77]
    cache = Cache(lens, page, e4m3, block, seed=page)
    q = queries(cache, 4, heads)
    off = cache.offsets([1] * 4)
    for sinks, window in ((0, 1 << 30), (5, 129), (17, 31), (1, 1)):
        a = run_sinks(cache, q, off, ints(lens), sinks, window)
        b = run_sinks(in_order(cache), q, off, ints(lens), sinks, window)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("sinks", [0, 1, 15, 16, 17, 200])
def test_windows_that_begin_anywhere(e4m3, sinks):
    """Every offset of the window's first token in a group of 16, and groups that the list only partly holds."""
    vis = [400 + i for i in range(18)]
    cache = Cache([max(vis)], 64, e4m3, 64, seed=sinks)
    check_sinks(cache, queries(cache, len(vis), 64), cache.offsets([len(vis)]), ints(vis), sinks, 150)


def test_largest_sinks_and_window():
    top = (1 << 31) - 1
    cache = Cache([333], 64, True, 64, seed=50)
    q = queries(cache, 1, 128)
    want = check_sinks(cache, q, cache.offsets([1]), ints([333]), 0, 333)
    for sinks, window in ((0, top), (top, 0), (top, top), (333, 0)):
        out, lse, _ = run_sinks(cache, q, cache.offsets([1]), ints([333]), sinks, window)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_selections_of_consecutive_positions():
    """Rising, falling, broken and repeated runs, and groups of -1, at every place of a tile."""
    cache = Cache([1024], 64, True, 64, seed=51)
    cache = in_order(cache)
    up = list(range(64, 128))
    rows = [up + up[::-1], [-1] * 16 + up + [-1] * 8 + list(range(200, 240)), list(range(9, 137)),
            [5] * 128, list(range(0, 16)) + [-1] * 96 + list(range(16, 32)), [-1] * 128,
            list(range(48, 64)) + list(range(60, 76)) + [3] + list(range(100, 115)) + list(range(896, 976))]
    q = queries(cache, len(rows), 128)
    off, vis = cache.offsets([len(rows)]), ints([1024] * len(rows))
    out, lse, ws = run_sparse(cache, q, off, vis, ints(rows))
    dsa.dsa_check_error(ws)
    lists = [[s for s in r if s >= 0] for r in rows]
    check_attend(out, lse, attend_reference(q, cache.pool, cache.scales, cache.table, off, lists, SCALE), True)


@pytest.mark.parametrize("e4m3", [False, True])
def test_cache_beyond_four_gib(e4m3):
    """Rows whose byte offsets pass 32 bits: appended, attended over a window and by selection."""
    row = D if e4m3 else 2 * D
    pages = (1 << 32) // (64 * row) + 50
    cache = Cache([400], 64, e4m3, 64, seed=52)
    few = cache.pool
    cache.pool = torch.zeros(pages, 64, D, dtype=few.dtype, device=DEV)
    cache.pool[pages - cache.num_pages:] = few
    if e4m3:
        scales = torch.ones(pages, 1, device=DEV)
        scales[pages - cache.num_pages:] = cache.scales
        cache.scales = scales
    cache.table[cache.table >= 0] += pages - cache.num_pages
    cache.num_pages = pages
    q = queries(cache, 1, 128)
    off, vis = cache.offsets([1]), ints([400])
    want = check_sinks(cache, q, off, vis, 4, 390)
    if e4m3:
        pick = torch.randperm(400, device=DEV, generator=cache.g)[:77]
        out, lse, ws = run_sparse(cache, q, off, vis, pick.int()[None].contiguous())
        check_attend(out, lse, attend_reference(q, cache.pool, cache.scales, cache.table, off, [pick.tolist()], SCALE), True)
    x = torch.randn(1, D, device=DEV, generator=cache.g).to(torch.bfloat16)
    x[:, DV:] = 0                                                 # no rotation to round
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    dsa.dsa_latent_append(x[:, :DV], x[:, DV:], inv_freq(), cache.pool, cache.table, off, vis, 1, ws,
                          kv_scales=cache.scales)
    dsa.dsa_check_error(ws)
    pg = int(cache.table[0, 399 // 64])
    got = cache.pool[pg, 399 % 64]
    if e4m3:
        got = codes_to_double(got) * cache.scales[pg, 0]
        s = float(cache.scales[pg, 0])
        assert ((got - x[0].double()).abs() <= torch.maximum(x[0].double().abs() * 2.0 ** -4, torch.tensor(s * 2.0 ** -10))).all()
    else:
        assert torch.equal(got, x[0])
    again, _, _ = run_sinks(cache, q, off, vis, 4, 390)
    assert not torch.equal(again, want[0])                        # it reads the appended row


@pytest.mark.parametrize("heads", [128, 64])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("long", [False, True])
def test_rows_that_no_sequence_holds_stay_as_they_were(heads, e4m3, long):
    """Rows before the first and behind the last sequence, with any q_vis and idx: neither written nor flagged."""
    n = 20000 if long else 70
    lens = [n, 40]
    cache = Cache(lens, 64, e4m3, 64, seed=53)
    off = ints([3, 4, 6])
    vis = ints([12, 1 << 30, n, n, 39, 40, n, 1 << 30, -5])
    q = queries(cache, 9, heads)
    q[:3] = math.nan
    out, lse, ws = run_sinks(cache, q, off, vis, 1, n)
    dsa.dsa_check_error(ws)
    part = run_sinks(cache, q[3:6].contiguous(), off - 3, vis[3:6].contiguous(), 1, n)
    # tiles may be divided over other pairs: the merge rounds apart
    ref = attend_reference(q[3:6].contiguous(), cache.pool, cache.scales, cache.table, off - 3,
                           [list(range(n)), list(range(39)), list(range(40))], SCALE)
    for o, l in ((out[3:6], lse[3:6]), part[:2]):
        check_attend(o, l, ref, e4m3)
    rest = [0, 1, 2, 6, 7, 8]
    assert torch.isnan(out[rest]).all() and torch.isnan(lse[rest]).all()      # as run_sinks filled them
    if e4m3:
        topk = 2048 if long else 100
        idx = torch.full((9, topk), 1 << 30, dtype=torch.int32, device=DEV)
        idx[3:6] = torch.arange(topk, dtype=torch.int32, device=DEV) % 30
        out, lse, ws = run_sparse(cache, q, off, vis, idx)
        dsa.dsa_check_error(ws)
        lists = [[i % 30 for i in range(topk)]] * 3
        ref = attend_reference(q[3:6].contiguous(), cache.pool, cache.scales, cache.table, off - 3, lists, SCALE)
        check_attend(out[3:6], lse[3:6], ref, True)
        assert torch.isnan(out[rest]).all() and torch.isnan(lse[rest]).all()


@pytest.mark.parametrize("ratio", [2.0 ** -14, 2.0 ** -15, 2.0 ** -16, 1.3 * 2.0 ** -15, 2.0 ** -30])
@pytest.mark.parametrize("heads", [128, 64])
def test_scales_of_one_tile_apart_by(ratio, heads):
    """Around the ratio up to which a tile's tokens share one scale, the small one in one block or in all but one;
    among them tiles of the other sort."""
    for few in (False, True):
        cache = Cache([900], 64, True, 16, seed=54, scale_exp=(-3, -3))
        flat = cache.table[0].long()
        small = 2.0 ** -3 * ratio
        for b in range(8):                                         # the first tile's eight blocks, and the sixth's
            for first in (0, 640):
                p = first + 16 * b
                if (b == 3) == few:
                    cache.scales[flat[p // 64], p % 64 // 16] = small
        q = (queries(cache, 1, heads).float() * 2.0 ** -6).to(torch.bfloat16)
        check_sinks(cache, q, cache.offsets([1]), ints([900]), 0, 900)


@pytest.mark.parametrize("heads", [128, 64])
@pytest.mark.parametrize("e4m3", [False, True])
def test_heads_that_are_not_finite_spoil_no_others(heads, e4m3):
    cache = Cache([700, 50], 64, e4m3, 64, seed=55)
    off, vis = cache.offsets([1, 1]), ints([700, 50])
    q = queries(cache, 2, heads)
    clean = run_sinks(cache, q, off, vis, 0, 700)
    bad = {(0, 3): math.nan, (0, heads - 1): math.inf, (1, 32): -math.inf, (1, 0): math.nan}
    for (t, h), v in bad.items():
        q[t, h, 7 * h % D] = v
    out, lse, ws = run_sinks(cache, q, off, vis, 0, 700)
    dsa.dsa_check_error(ws)
    for t in range(2):
        for h in range(heads):
            if (t, h) in bad:
                assert torch.isnan(out[t, h]).all() and torch.isnan(lse[t, h])
            else:
                assert torch.equal(out[t, h], clean[0][t, h]) and lse[t, h] == clean[1][t, h]


@pytest.mark.parametrize("heads", [128, 64])
@pytest.mark.parametrize("e4m3", [False, True])
def test_many_short_queries_repeat_their_bits(heads, e4m3):
    """More queries than threads look for the shares, of one or two tiles each, begun and ended often."""
    cache = Cache([260] * 3, 16, e4m3, 16, seed=56)
    counts = [900, 500, 300]
    vis = ints([(31 * i) % 260 + 1 for i in range(1700)])
    q = queries(cache, 1700, heads)
    off = cache.offsets(counts)
    first = run_sinks(cache, q, off, vis, 2, 140)
    dsa.dsa_check_error(first[2])
    for _ in range(5):
        again = run_sinks(cache, q, off, vis, 2, 140, ws=first[2])
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    some = list(range(0, 1700, 97))
    off1 = [sum(1 for t in some if t < e) for e in [0, 900, 1400, 1700]]
    v = vis[some].tolist()
    lists = [[s for s in range(n) if s < 2 or s >= n - 140] for n in v]
    ref = attend_reference(q[some].contiguous(), cache.pool, cache.scales, cache.table, ints(off1), lists, SCALE)
    check_attend(first[0][some], first[1][some], ref, e4m3)


@pytest.mark.parametrize("heads", [128, 64])
def test_queries_of_one_tile_each_keep_their_own_factors(heads):
    """Scores run ahead of the values over several queries: each has a size of its own, so that another's scaling shows."""
    cache = Cache([120], 64, True, 64, seed=57)
    Q = 600
    q = queries(cache, Q, heads).float()
    q *= torch.exp2(torch.randint(-30, 4, (Q, heads, 1), device=DEV, generator=cache.g).float())
    vis = ints([(17 * i) % 120 + 1 for i in range(Q)])
    check_sinks(cache, q.to(torch.bfloat16), cache.offsets([Q]), vis, 0, 120)


def test_captured_behind_every_sort_of_node():
    """A call begins beside the end of the kernel before it: captured after a copy, a memset, a join of two streams, another
    kernel, an append and itself, with one workspace, it still reads what those wrote."""
    cache = Cache([3000, 70], 64, True, 64, seed=58)
    off, vis = cache.offsets([1, 1]), ints([3000, 70])
    f, ws = inv_freq(), dsa.attend_workspace(128)
    q, other = queries(cache, 2, 128), queries(cache, 2, 128)
    row = torch.randn(2, D, device=DEV, generator=cache.g).to(torch.bfloat16)
    host = queries(cache, 2, 128).cpu().pin_memory()
    outs = [(torch.empty(2, 128, DV, dtype=torch.bfloat16, device=DEV), torch.empty(2, 128, device=DEV)) for _ in range(6)]

    def attend(i):
        dsa.dsa_mla_decode_sinks(q, cache.pool, cache.table, off, vis, 2, 1, 2900, SCALE, *outs[i], ws, kv_scales=cache.scales)

    def steps(stream, side):
        attend(0)
        attend(1)                                                  # behind the call's own merge
        q.copy_(host, non_blocking=True)                           # a copy node
        attend(2)
        q.zero_()
        attend(3)
        side.wait_stream(stream)                                   # a join of two streams
        with torch.cuda.stream(side):
            q.copy_(other)
        row.mul_(1.5)
        stream.wait_stream(side)
        attend(4)
        dsa.dsa_latent_append(row[:, :DV], row[:, DV:], f, cache.pool, cache.table, off, vis, 2, ws, kv_scales=cache.scales)
        attend(5)

    stream, side = torch.cuda.Stream(), torch.cuda.Stream()
    kept = [t.clone() for t in (q, row, cache.pool, cache.scales)]
    results = []
    for how in ("eager", "graph"):
        for t, k in zip((q, row, cache.pool, cache.scales), kept):
            t.copy_(k)
        torch.cuda.synchronize()
        if how == "eager":
            with torch.cuda.stream(stream):
                for _ in range(2):
                    steps(stream, side)
                    stream.synchronize()
                    results.append([t.clone() for o in outs for t in o])
        else:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                steps(stream, side)
            for _ in range(2):
                graph.replay()
                torch.cuda.synchronize()
                results.append([t.clone() for o in outs for t in o])
    dsa.dsa_check_error(ws)
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(results[i], results[2 + i]))
    zero = results[0][2 * 3]
    assert torch.equal(results[0][0], results[0][2]) and not torch.equal(results[0][4], results[0][2])
    assert not torch.equal(zero, results[0][4]) and not torch.equal(results[0][8], results[0][10])


# ---------------------------------------------------------------------- append
def test_blocks_longer_than_the_registers_hold():
    """Runs of more than 64 rows are read twice; an old scale that is no power of two, and rows that are not finite."""
    for page, block in ((128, 128), (512, 256)):
        for start, old in ((0, 1.0), (30, 1.37), (30, 2.0 ** -9)):
            cache = Cache([start + 300], page, True, block, seed=start + page)
            cache.scales.fill_(old)
            kv, pe, off, vis = inputs(cache, [start], [300])
            kv[70, 9], kv[111, 511] = math.nan, -math.inf
            check(cache, kv, pe, off, vis, True)


def test_short_runs_over_an_old_scale_that_is_no_power_of_two():
    cache = Cache([60, 60], 64, True, 64, seed=60)
    cache.scales.fill_(1.37 * 2.0 ** -3)
    kv, pe, off, vis = inputs(cache, [20, 50], [3, 10])
    kv[5, 100] = math.inf
    check(cache, kv, pe, off, vis, False)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("counts", [[3, 2], [40, 30]])
def test_frequencies_that_are_no_numbers_spoil_their_pair_alone(e4m3, counts):
    cache = Cache([100, 100], 64, e4m3, 64, seed=61)
    kv, pe, off, vis = inputs(cache, [10, 20], counts)
    other = Cache([100, 100], 64, e4m3, 64, seed=61)
    f, g = inv_freq(), inv_freq()
    g[4], g[9] = math.nan, math.inf
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    for c, fr in ((cache, f), (other, g)):
        pe_c = pe.clone()
        pe_c[:, [4, 9, 36, 41]] = 0                                # the pairs in question count for no maximum
        dsa.dsa_latent_append(kv, pe_c, fr, c.pool, c.table, off, vis, 2, ws, kv_scales=c.scales)
    dsa.dsa_check_error(ws)
    a, b = ((codes_to_double(c.pool) if e4m3 else c.pool.double()).view(-1, D) for c in (cache, other))
    slot = torch.tensor([int(cache.table[s, p // 64]) * 64 + p % 64
                         for s, (st, n) in enumerate(zip((10, 20), counts)) for p in range(st, st + n)], device=DEV)
    spoilt = [DV + i for i in (4, 9, 36, 41)]
    assert torch.isnan(b[slot][:, spoilt]).all()
    keep = [i for i in range(D) if i not in spoilt]
    assert torch.equal(a[slot][:, keep].nan_to_num(), b[slot][:, keep].nan_to_num())
    if e4m3:
        assert torch.equal(cache.scales, other.scales)


def test_positions_at_the_end_of_the_type():
    """q_vis up to the largest integer lies behind every page: skipped, flagged, nothing written."""
    for e4m3 in (False, True):
        cache = Cache([64], 64, e4m3, 64, seed=62)
        kv, pe, off, vis = inputs(cache, [0], [4])
        vis = ints([(1 << 31) - 3, (1 << 31) - 2, (1 << 31) - 1, 5])
        before = cache.pool.clone().view(torch.uint8)
        ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
        dsa.dsa_latent_append(kv, pe, inv_freq(), cache.pool, cache.table, off, vis, 1, ws, kv_scales=cache.scales)
        with pytest.raises(dsa.DSAError):
            dsa.dsa_check_error(ws)
        assert torch.equal(before, cache.pool.view(torch.uint8))


def test_mixed_lengths_take_one_kernel():
    """One long prompt among single tokens: the average decides the kernel, every row is right."""
    starts, counts = [0] + [13 * i % 64 for i in range(40)], [100] + [1] * 40
    cache = Cache([s + n for s, n in zip(starts, counts)], 64, True, 64, seed=63)
    check(cache, *inputs(cache, starts, counts), False)
