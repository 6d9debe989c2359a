"""dsa_mla_decode_sinks and dsa_sparse_mla_decode_fp8_block against their definition in 64 bits."""
import math

import pytest
import torch

import sparse_attention_decode_lightning_b200 as dsa
from tests._latent import D, DV, Cache, attend_reference, check_attend, list_of

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 192 ** -0.5


def queries(cache, Q, H):
    return torch.randn(Q, H, D, device=DEV, generator=cache.g).to(torch.bfloat16)


def run_sinks(cache, q, off, vis, sinks, window, ws=None, stream=None, scale=SCALE):
    out = torch.full((*q.shape[:2], DV), math.nan, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], math.nan, dtype=torch.float32, device=DEV)
    ws = dsa.attend_workspace(q.shape[1]) if ws is None else ws
    dsa.dsa_mla_decode_sinks(q, cache.pool, cache.table, off, vis, off.numel() - 1, sinks, window, scale, out, lse, ws,
                             kv_scales=cache.scales, stream=stream)
    return out, lse, ws


def run_sparse(cache, q, off, vis, idx, ws=None, scale=SCALE):
    out = torch.full((*q.shape[:2], DV), math.nan, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], math.nan, dtype=torch.float32, device=DEV)
    ws = dsa.attend_workspace(q.shape[1]) if ws is None else ws
    dsa.dsa_sparse_mla_decode_fp8_block(q, cache.pool, cache.scales, cache.table, off, vis, idx, off.numel() - 1, scale,
                                        out, lse, ws)
    return out, lse, ws


def check_sinks(cache, q, off, vis, sinks, window, scale=SCALE):
    out, lse, ws = run_sinks(cache, q, off, vis, sinks, window, scale=scale)
    dsa.dsa_check_error(ws)
    lists = [list_of(v, sinks, window) for v in vis.tolist()]
    ref = attend_reference(q, cache.pool, cache.scales, cache.table, off, lists, scale)
    check_attend(out, lse, ref, cache.e4m3)
    return out, lse


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


KINDS = [(False, 1, 64), (False, 1, 16), (True, 64, 64), (True, 16, 64), (True, 1, 16), (True, 256, 512)]


@pytest.mark.parametrize("heads", [128, 64])
@pytest.mark.parametrize("e4m3,block,page", KINDS)
@pytest.mark.parametrize("sinks,window", [(0, 1 << 30), (4, 100), (0, 64), (70, 0), (0, 0), (65, 63)])
def test_sinks_match_definition(heads, e4m3, block, page, sinks, window):
    """Lengths from none and one to several tiles, one token off the tiles' ends."""
    vis = [0, 1, 2, 63, 64, 65, 127, 128, 129, 300, 641]
    cache = Cache(vis, page, e4m3, block, seed=heads + sinks + page)
    check_sinks(cache, queries(cache, len(vis), heads), cache.offsets([1] * len(vis)), ints(vis), sinks, window)


@pytest.mark.parametrize("heads", [128, 64])
@pytest.mark.parametrize("e4m3", [False, True])
def test_one_long_sequence_is_divided(heads, e4m3):
    """A single query on every SM pair: 74 and more tiles, partial results merged."""
    for n in (64 * 73 + 1, 64 * 74, 64 * 75, 20011):
        cache = Cache([n], 64, e4m3, 64, seed=n)
        check_sinks(cache, queries(cache, 1, heads), cache.offsets([1]), ints([n]), 0, n)


@pytest.mark.parametrize("heads", [128, 64])
@pytest.mark.parametrize("e4m3", [False, True])
def test_ragged_verify_batch(heads, e4m3):
    """Several queries a sequence, some sequences without any, queries that share pairs and cross them."""
    lens = [900, 5, 2500, 77, 0, 1300, 64, 4097]
    counts = [4, 5, 8, 1, 0, 12, 2, 3]
    cache = Cache(lens, 16, e4m3, 16, seed=11)
    vis = [n - c + 1 + i for n, c in zip(lens, counts) for i in range(c)]
    check_sinks(cache, queries(cache, len(vis), heads), cache.offsets(counts), ints(vis), 3, 1024)


def test_many_queries_on_each_pair():
    cache = Cache([700] * 300, 64, True, 64, seed=12)
    cache.table[:] = cache.table[0]                       # 300 users of one prefix
    vis = [(37 * i) % 700 + 1 for i in range(300)]
    check_sinks(cache, queries(cache, 300, 64), cache.offsets([1] * 300), ints(vis), 1, 200)


@pytest.mark.parametrize("heads", [128, 64])
@pytest.mark.parametrize("topk", [1, 63, 64, 65, 1000, 2048])
@pytest.mark.parametrize("block,page", [(64, 64), (1, 16), (16, 64)])
def test_selected_match_definition(heads, topk, block, page):
    lens = [3000, 40, 1500, 1]
    counts = [2, 1, 3, 1]
    cache = Cache(lens, page, True, block, seed=topk + block)
    vis = [n - c + 1 + i for n, c in zip(lens, counts) for i in range(c)]
    q = queries(cache, len(vis), heads)
    idx = torch.full((len(vis), topk), -1, dtype=torch.int32, device=DEV)
    lists = []
    for t, v in enumerate(vis):
        k = min(topk, v)
        pick = torch.randperm(v, device=DEV, generator=cache.g)[:k]
        if t == 1:
            pick = pick[:0]                               # a row that selects nothing
        at = torch.randperm(topk, device=DEV, generator=cache.g)[:pick.numel()]    # -1 anywhere
        idx[t, at] = pick.to(torch.int32)
        lists.append(pick.tolist())
    out, lse, ws = run_sparse(cache, q, cache.offsets(counts), ints(vis), idx)
    dsa.dsa_check_error(ws)
    check_attend(out, lse, attend_reference(q, cache.pool, cache.scales, cache.table, cache.offsets(counts), lists, SCALE),
                 True)


def test_an_index_twice_counts_twice():
    cache = Cache([500], 64, True, 64, seed=5)
    q = queries(cache, 1, 128)
    pick = [3, 3, 499, 7, 3]
    out, lse, ws = run_sparse(cache, q, cache.offsets([1]), ints([500]), ints([pick]))
    dsa.dsa_check_error(ws)
    check_attend(out, lse, attend_reference(q, cache.pool, cache.scales, cache.table, cache.offsets([1]), [pick], SCALE),
                 True)


def test_all_positions_selected_equal_the_window_form_bitwise():
    """The same tokens in the same order: both forms run the same arithmetic."""
    cache = Cache([1200], 64, True, 16, seed=21)
    q = queries(cache, 1, 128)
    off, vis = cache.offsets([1]), ints([1200])
    a = run_sinks(cache, q, off, vis, 0, 1200)
    b = run_sparse(cache, q, off, vis, torch.arange(1200, dtype=torch.int32, device=DEV)[None].contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("spread", [(-40, -30), (20, 40), (-20, 20), (-40, 40)])
def test_scales_far_apart(spread):
    """Blocks of very different magnitude; the query is scaled so that scores stay moderate."""
    cache = Cache([600], 64, True, 16, seed=7, scale_exp=spread)
    q = (queries(cache, 1, 128).float() * 2.0 ** -(spread[1] + 8)).to(torch.bfloat16)
    check_sinks(cache, q, cache.offsets([1]), ints([600]), 0, 600)


def test_scales_that_are_no_power_of_two():
    cache = Cache([600], 64, True, 16, seed=8)
    cache.scales *= 1.37
    check_sinks(cache, queries(cache, 1, 64), cache.offsets([1]), ints([600]), 5, 300)


@pytest.mark.parametrize("e4m3", [False, True])
def test_queries_of_very_different_size(e4m3):
    """Heads from 2^-60 to 2^20 times the usual size and a zero one: fp16 operands hold each after its own scaling."""
    cache = Cache([300], 64, e4m3, 64, seed=13)
    q = queries(cache, 1, 128).float()
    f = torch.exp2(torch.linspace(-60, 20, 128, device=DEV))
    f[5] = 0
    check_sinks(cache, (q * f[None, :, None]).to(torch.bfloat16), cache.offsets([1]), ints([300]), 0, 300)


@pytest.mark.parametrize("e4m3", [False, True])
def test_peaked_and_growing_scores(e4m3):
    """Scores that rise along the list make the running maximum move at every tile; one token outweighs all."""
    n = 640
    cache = Cache([n], 64, e4m3, 64, seed=14)
    q = queries(cache, 1, 128)
    row = cache.table[0].long()[torch.arange(n, device=DEV) // 64] * 64 + torch.arange(n, device=DEV) % 64
    ramp = (torch.arange(n, device=DEV) // 64 + 1).float()
    flat = cache.pool.view(-1, D)
    if e4m3:
        cache.scales.fill_(2.0 ** -6)
        flat[row, 520] = (ramp * 40).clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        flat[row, 520] = (ramp * 0.6).to(torch.bfloat16)
    q[:, :, 520] = 200.0
    check_sinks(cache, q, cache.offsets([1]), ints([n]), 0, n)


def test_values_that_are_nan_or_infinite():
    """In a listed token they reach the result, elsewhere they do not."""
    cache = Cache([200, 200], 64, False, seed=15)
    q = queries(cache, 2, 128)
    off, vis = cache.offsets([1, 1]), ints([200, 200])
    clean = run_sinks(cache, q, off, vis, 0, 200)
    page = int(cache.table[0, 1])
    cache.pool[page, 3, 17] = math.nan
    out, lse, ws = run_sinks(cache, q, off, vis, 0, 200)
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    assert torch.equal(out[1], clean[0][1]) and torch.equal(lse[1], clean[1][1])
    out, lse, ws = run_sinks(cache, q, off, vis, 64, 132)          # position 67 lies between sinks and window
    assert not torch.isnan(out).any() and not torch.isnan(lse).any()


def test_bad_pages_and_scales_are_skipped_and_flagged():
    for what in ("page", "pool", "scale", "vis", "idx"):
        cache = Cache([300], 64, True, 64, seed=16)
        q = queries(cache, 1, 128)
        off, vis = cache.offsets([1]), ints([300])
        lists = [[s for s in range(300) if what == "vis" or not 64 <= s < 128]]
        if what == "page":
            cache.table[0, 1] = -1
        elif what == "pool":
            cache.table[0, 1] = cache.num_pages
        elif what == "scale":
            cache.scales[int(cache.table[0, 1])] = 0.0
        if what == "vis":
            vis = ints([cache.max_pages * 64 + 5])                 # the pages behind token 300 do not exist
            cache.pool[int(cache.table[0, 4]), 44:] = 0x08
            lists = [list(range(320))]
            out, lse, ws = run_sinks(cache, q, off, vis, 0, 1 << 30)
        elif what == "idx":
            pick = list(range(0, 60)) + [300, 5000, -2]
            lists = [list(range(0, 60))]
            out, lse, ws = run_sparse(cache, q, off, vis, ints([pick]))
        else:
            out, lse, ws = run_sinks(cache, q, off, vis, 0, 300)
        with pytest.raises(dsa.DSAError) as e:
            dsa.dsa_check_error(ws)
        assert e.value.status == 4
        dsa.dsa_check_error(ws)
        check_attend(out, lse, attend_reference(q, cache.pool, cache.scales, cache.table, off, lists, SCALE), True)


def test_results_repeat_and_workspace_is_shared():
    """One workspace for calls of different shapes on one stream; each repeats its bits."""
    ws = dsa.attend_workspace(128)
    first = {}
    for rep in range(2):
        for key, (lens, heads, e4m3) in {"a": ([5000], 128, True), "b": ([700, 90, 3], 64, False),
                                         "c": ([20000, 31], 64, True)}.items():
            cache = Cache(lens, 64, e4m3, 64, seed=33)
            q = queries(cache, len(lens), heads)
            out, lse, _ = run_sinks(cache, q, cache.offsets([1] * len(lens)), ints(lens), 0, 1 << 30, ws=ws)
            if rep:
                assert torch.equal(first[key][0], out) and torch.equal(first[key][1], lse)
            first[key] = out, lse
    dsa.dsa_check_error(ws)


def test_captured_calls_share_a_workspace_and_read_inputs_at_replay():
    cache = Cache([4000, 600], 64, True, 64, seed=34)
    off, vis = cache.offsets([1, 1]), ints([4000, 600])
    q = queries(cache, 2, 128)
    ws = dsa.attend_workspace(128)
    outs = [(torch.empty(2, 128, DV, dtype=torch.bfloat16, device=DEV), torch.empty(2, 128, device=DEV)) for _ in range(2)]
    graphs = []
    for (o, l), window in zip(outs, (4000, 300)):
        run_sinks(cache, q, off, vis, 2, window, ws=ws)            # sets the kernel's attributes before the capture
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dsa.dsa_mla_decode_sinks(q, cache.pool, cache.table, off, vis, 2, 2, window, SCALE, o, l, ws,
                                     kv_scales=cache.scales)
        graphs.append(g)
    q.copy_(queries(cache, 2, 128))
    vis.copy_(ints([3333, 77]))
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for (o, l), window in zip(outs, (4000, 300)):
        ref_o, ref_l, _ = run_sinks(cache, q, off, vis, 2, window)
        assert torch.equal(o, ref_o) and torch.equal(l, ref_l)


def test_two_streams_with_their_own_workspaces():
    cache = Cache([9000, 3000], 64, True, 64, seed=35)
    off, vis = cache.offsets([1, 1]), ints([9000, 3000])
    q = queries(cache, 2, 128)
    want = run_sinks(cache, q, off, vis, 0, 9000)
    wss = [dsa.attend_workspace(128) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s, ws in zip(streams, wss):
            with torch.cuda.stream(s):
                got.append(run_sinks(cache, q, off, vis, 0, 9000, ws=ws, stream=s))
    torch.cuda.synchronize()
    for o, l, _ in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


@pytest.mark.parametrize("heads", [128, 64])
def test_append_then_attend(heads):
    """A decode loop as a program runs it: prompt, then single tokens, each attended densely, over a window, and
    through a selection; against the definition on the cache as it stands."""
    lens, new = [130, 61], 5
    cache = Cache([n + new for n in lens], 64, True, 64, seed=40)
    cache.pool.fill_(0x7F)                                         # nothing is in the cache yet
    f = (10000.0 ** (-torch.arange(0, 64, 2, device=DEV, dtype=torch.float64) / 64)).float()
    ws = dsa.attend_workspace(heads)

    def append(counts, starts):
        x = torch.randn(sum(counts), D, device=DEV, generator=cache.g).to(torch.bfloat16)
        vis = ints([s + i + 1 for s, n in zip(starts, counts) for i in range(n)])
        off = cache.offsets(counts)
        dsa.dsa_latent_append(x[:, :DV], x[:, DV:], f, cache.pool, cache.table, off, vis, 2, ws, kv_scales=cache.scales)
        return off, vis

    append(lens, [0, 0])
    for i in range(new):
        off, vis = append([1, 1], [n + i for n in lens])
        q = queries(cache, 2, heads)
        for sinks, window in ((0, 1 << 30), (2, 33)):
            out, lse, _ = run_sinks(cache, q, off, vis, sinks, window, ws=ws)
            lists = [list_of(v, sinks, window) for v in vis.tolist()]
            check_attend(out, lse, attend_reference(q, cache.pool, cache.scales, cache.table, off, lists, SCALE), True)
        idx = torch.stack([torch.randperm(min(vis.tolist()), device=DEV, generator=cache.g)[:50] for _ in range(2)]).int()
        out, lse, _ = run_sparse(cache, q, off, vis, idx.contiguous(), ws=ws)
        check_attend(out, lse, attend_reference(q, cache.pool, cache.scales, cache.table, off, idx.tolist(), SCALE), True)
    dsa.dsa_check_error(ws)
