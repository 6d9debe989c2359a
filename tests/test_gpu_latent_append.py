"""dsa_latent_append against its definition in 64 bits: both cache types, block sizes, ragged and padded batches,
far positions, blocks that are partly filled, values that have no place in the type."""
import math

import pytest
import torch

import sparse_attention_decode_lightning_b200 as dsa
from tests._latent import D, DR, DV, E4M3, Cache, append_reference, codes_to_double

pytestmark = pytest.mark.gpu
DEV = "cuda"


def inv_freq():
    return (10000.0 ** (-torch.arange(0, DR, 2, device=DEV, dtype=torch.float64) / DR)).float()


def inputs(cache, starts, counts, pad=0):
    """kv and k_pe as slices of one array, q_offsets, q_vis; `pad` rows behind the last sequence."""
    T = sum(counts) + pad
    x = torch.randn(T, D + 8, device=DEV, generator=cache.g)
    x = (x * torch.exp(1.5 * torch.randn(T, 1, device=DEV, generator=cache.g))).to(torch.bfloat16)
    vis = [s + i + 1 for s, n in zip(starts, counts) for i in range(n)] + [7] * pad
    return x[:, :DV], x[:, DV:D], cache.offsets(counts), torch.tensor(vis, dtype=torch.int32, device=DEV)


def check(cache, kv, pe, off, vis, interleaved):
    before = cache.pool.clone()
    want, sc, written = append_reference(kv, pe, inv_freq(), interleaved, cache.pool, cache.scales, cache.table, off, vis)
    old_scales = None if sc is None else cache.scales.clone()
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    dsa.dsa_latent_append(kv, pe, inv_freq(), cache.pool, cache.table, off, vis, off.numel() - 1, ws,
                          kv_scales=cache.scales, interleaved=interleaved)
    dsa.dsa_check_error(ws)
    got = (codes_to_double(cache.pool) if cache.e4m3 else cache.pool.double()).view(-1, D)
    same = cache.pool.view(torch.uint8 if cache.e4m3 else torch.int16).view(-1, D)
    kept = before.view(torch.uint8 if cache.e4m3 else torch.int16).view(-1, D)
    assert torch.equal(same[~written], kept[~written])            # rows of other positions stay as they were
    g, w = got[written], want[written]
    fin = torch.isfinite(w)
    if cache.e4m3:
        assert torch.equal(cache.scales.double().view(-1), sc)
        assert torch.isnan(g[~fin]).all()
        # half a step of e4m3 (2^-4 relative, 2^-10 below its normals), and the rotation's fp32 error, which is
        # within 2^-21 of the block's largest value (448 in these units)
        tol = torch.maximum(w.abs() * 2.0 ** -4, torch.full_like(w, 2.0 ** -10)) + 448 * 2.0 ** -21
        tol = torch.where(w.abs() > 448, w.abs() - 448 + tol, tol)      # saturated
    else:
        assert torch.equal(g[:, :DV].nan_to_num(), w[:, :DV].nan_to_num())   # the latents as they are
        # half a step of bf16 and the rotation's fp32 error: cos and sin within 2^-22, two products and a sum
        big = torch.where(fin, w, 0.0)[:, DV:].abs().amax(1, keepdim=True)
        tol = w.abs() * 2.0 ** -8 + big * 2.0 ** -20
    assert ((g - w).abs()[fin] <= tol[fin]).all(), float(((g - w).abs()[fin] / tol[fin]).max())
    if old_scales is not None:
        used = torch.zeros_like(sc, dtype=torch.bool)
        used[torch.unique(torch.nonzero(written).view(-1) // cache.block)] = True
        assert torch.equal(cache.scales.view(-1)[~used], old_scales.view(-1)[~used])


CASES = [
    # starts, counts
    ([0], [1]),
    ([0], [200]),                                        # from the very first position
    ([63, 64, 65, 1023], [1, 1, 1, 1]),                  # around a page's end
    ([5, 60, 700, 0, 31], [4, 7, 1, 3, 0]),              # ragged, an empty sequence
    ([100, 1], [333, 190]),                              # long runs that start inside a block
    ([17] * 40, [3] * 40),
]


@pytest.mark.parametrize("starts,counts", CASES)
@pytest.mark.parametrize("page,block,e4m3", [(64, 1, False), (16, 1, False), (64, 64, True), (64, 16, True),
                                             (16, 1, True), (1, 1, True), (1024, 512, True)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_matches_definition(starts, counts, page, block, e4m3, interleaved):
    cache = Cache([s + n for s, n in zip(starts, counts)], page, e4m3, block, seed=len(counts) + page + block)
    check(cache, *inputs(cache, starts, counts), interleaved)


def test_far_positions_keep_their_angle():
    """Positions near 2^20: fp32 angles there would be off by a sixteenth of a radian."""
    start = (1 << 20) - 40
    cache = Cache([64], 64, False, seed=3)
    page = int(cache.table[0, 0])
    cache.table = torch.full((1, 1 << 14), -1, dtype=torch.int32, device=DEV)
    cache.table[0, start // 64:start // 64 + 1] = page
    check(cache, *inputs(cache, [start], [39]), False)


@pytest.mark.parametrize("e4m3", [False, True])
def test_padding_rows_are_skipped(e4m3):
    """q_vis = 0 at a sequence's end and in a whole sequence, and rows behind the last sequence."""
    cache = Cache([70, 40, 90], 64, e4m3, 64, seed=9)
    kv, pe, off, vis = inputs(cache, [60, 36, 80], [10, 4, 10], pad=5)
    vis[7:10] = 0
    vis[10:14] = 0
    check(cache, kv, pe, off, vis, False)


def test_block_scales_grow_and_codes_follow():
    """Appending ever larger tokens one by one: the block's codes are rescaled each time the scale grows."""
    cache = Cache([64], 64, True, 64, seed=4)
    off = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    for p in range(20):
        kv = (torch.randn(1, DV, device=DEV, generator=cache.g) * 2.0 ** p).to(torch.bfloat16)
        pe = torch.zeros(1, DR, dtype=torch.bfloat16, device=DEV)
        check(cache, kv, pe, off, torch.tensor([p + 1], dtype=torch.int32, device=DEV), False)


def test_scales_at_the_borders_of_a_power_of_two():
    """amax of exactly 448 * 2^e takes that e, the next bf16 above it takes e + 1, zeros the smallest scale."""
    for amax, want in ((448.0, 1.0), (450.0, 2.0), (1.75, 2.0 ** -8), (1.7578125, 2.0 ** -7), (0.0, 2.0 ** -40),
                       (2.0 ** 60, 2.0 ** 40), (3e38, 2.0 ** 40), (1e-38, 2.0 ** -40)):
        cache = Cache([1], 16, True, 16, seed=1)
        kv = torch.zeros(1, DV, dtype=torch.bfloat16, device=DEV)
        kv[0, 100] = -amax
        check(cache, kv, torch.zeros(1, DR, dtype=torch.bfloat16, device=DEV),
              torch.tensor([0, 1], dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV), False)
        assert float(cache.scales[int(cache.table[0, 0]), 0]) == want


def test_non_finite_values():
    """NaN and infinities are stored as NaN and leave the block's scale alone; a bf16 cache keeps them."""
    for e4m3 in (True, False):
        cache = Cache([8], 16, e4m3, 16, seed=2)
        kv, pe, off, vis = inputs(cache, [0], [8])
        kv[1, 3], kv[2, 4], kv[3, 5] = math.nan, math.inf, -math.inf
        check(cache, kv, pe, off, vis, False)


def test_bad_rows_are_skipped_and_flagged():
    """A position without a page, a page outside the pool, a row out of order, an old scale that is none."""
    for what in ("page", "table", "order", "scale"):
        cache = Cache([40, 40], 16, True, 16, seed=6)
        kv, pe, off, vis = inputs(cache, [30, 10], [4, 4])
        if what == "page":
            cache.table[0, 1:] = -1
        elif what == "table":
            cache.table[0, 1] = cache.num_pages
        elif what == "order":
            vis[2] = 39
        else:
            cache.scales[int(cache.table[0, 1])] = math.nan
        ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
        clean = cache.pool.clone()
        dsa.dsa_latent_append(kv, pe, inv_freq(), cache.pool, cache.table, off, vis, 2, ws, kv_scales=cache.scales)
        with pytest.raises(dsa.DSAError) as e:
            dsa.dsa_check_error(ws)
        assert e.value.status == 4
        dsa.dsa_check_error(ws)                                   # cleared
        changed = (clean != cache.pool).flatten(2).any(2).nonzero().tolist()
        pages = {int(cache.table[1, 0])} | ({int(cache.table[0, 1]), int(cache.table[0, 2])}
                                            if what in ("order", "scale") else
                                            {int(cache.table[0, 2])} if what == "table" else set())
        assert set(p for p, _ in changed) <= pages and changed
        if what == "order":
            assert [int(cache.table[0, 38 // 16]), 38 % 16] not in changed


def test_other_stream_and_graph():
    """On a side stream, and captured: a replay reads the inputs as they are then."""
    cache = Cache([50, 90], 64, True, 64, seed=8)
    kv, pe, off, vis = inputs(cache, [46, 80], [4, 4])
    f = inv_freq()
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    pool0, sc0 = cache.pool.clone(), cache.scales.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        dsa.dsa_latent_append(kv, pe, f, cache.pool, cache.table, off, vis, 2, ws, kv_scales=cache.scales, stream=s)
    kv.mul_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    got, gsc = cache.pool.clone(), cache.scales.clone()
    cache.pool.copy_(pool0)
    cache.scales.copy_(sc0)
    check(cache, kv, pe, off, vis, False)
    assert torch.equal(got, cache.pool) and torch.equal(gsc, cache.scales)
    assert cache.pool.view(E4M3).dtype == E4M3
