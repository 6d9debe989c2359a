"""Decoding users and prompt chunks in one append: right whichever is more, and no dearer than one after the other."""
import pytest
import torch

import sparse_attention_decode_lightning_b200 as dsa
from tests._latent import D, DV, Cache
from tests.test_gpu_latent_append import check, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"

# starts and counts: mostly single tokens, and mostly prompt rows
MIXES = [
    ([7 * i for i in range(200)] + [0, 37], [1] * 200 + [130, 200]),
    ([0, 5] + [11 * i for i in range(40)], [300, 64] + [1 + i % 4 for i in range(40)]),
    ([3, 64, 60, 100] * 10, [4, 5, 6, 65] * 10),
]


@pytest.mark.parametrize("starts,counts", MIXES)
@pytest.mark.parametrize("page,block", [(64, 64), (64, 16), (16, 4), (1024, 256)])
def test_short_and_long_runs_in_one_call(starts, counts, page, block):
    cache = Cache([s + n for s, n in zip(starts, counts)], page, True, block, seed=page + len(counts))
    cache.scales[::3] *= 1.25                                     # old scales that are no power of two
    kv, pe, off, vis = inputs(cache, starts, counts, pad=3)
    long = max(range(len(counts)), key=lambda b: counts[b])
    end = int(off[long + 1])
    vis[end - 2:end] = 0                                          # padding at the longest one's end
    kv[int(off[long]) + 1, 5] = float("inf")
    check(cache, kv, pe, off, vis, False)


def replay_us(starts, counts):
    """Shortest of some replays of ten captured calls, a call."""
    cache = Cache([s + n for s, n in zip(starts, counts)], 64, True, 64, seed=1)
    cache.scales.fill_(2.0 ** 6)                                  # they do not grow from call to call
    x = torch.randn(sum(counts), D, device=DEV).to(torch.bfloat16)
    off = cache.offsets(counts)
    vis = torch.tensor([s + i + 1 for s, n in zip(starts, counts) for i in range(n)], dtype=torch.int32, device=DEV)
    freq, ws = torch.rand(32, device=DEV), torch.zeros(256, dtype=torch.uint8, device=DEV)

    def call():
        dsa.dsa_latent_append(x[:, :DV], x[:, DV:], freq, cache.pool, cache.table, off, vis, len(counts), ws,
                              kv_scales=cache.scales)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(10):
            call()
    best = float("inf")
    for _ in range(10):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 100)
    dsa.dsa_check_error(ws)
    return best


@pytest.mark.parametrize("users,chunks,tokens", [(512, 1, 1024), (64, 8, 4000)])
def test_a_chunk_beside_decoding_users_costs_no_more_than_both_alone(users, chunks, tokens):
    """0.85 of the sum is measured; with a run's warps set by the batch's average it was 2.7 and 3.3."""
    ones = [500 + i for i in range(users)], [1] * users
    long = [0] * chunks, [tokens] * chunks
    alone = replay_us(*ones) + replay_us(*long)
    together = replay_us(ones[0] + long[0], ones[1] + long[1])
    assert together <= 1.6 * alone, (together, alone)
