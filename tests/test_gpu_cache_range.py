"""The paged int8 cache at the ends of its range: running maxima that rise again and again inside a step (against fp64
with the bounds of cache_ref); workspaces that are not the device's."""
import math

import pytest
import torch

import biased_attention_video_b200 as h3
from test_gpu_cache import DEV, check_forward, i32, make_cache, make_table

pytestmark = pytest.mark.gpu


def ladder(d, levels, unit, scale=None, seed=0):
    """A cache whose key j has the score `unit` levels[j] (plus a little) in log2 units under the queries that come
    with it, and minus that for every other query head; levels are codes."""
    n = len(levels)
    pages = -(-n // 64)
    c, host = make_cache(pages, 1, d, seed=seed)
    table = make_table([n], pages, seed=seed)
    k, v, ks, vs, _ = host
    for j, code in enumerate(levels):
        k[table[0][j // 64], 0, j % 64, 0] = code
    ks.fill_(0.01)
    if scale is not None:
        vs.copy_(scale * vs)
    for mine, theirs in ((c.k, k), (c.k_scale, ks), (c.v_scale, vs)):
        mine.copy_(theirs)

    def queries(H, rows):
        q = 0.05 * torch.randn(H, rows, d, generator=torch.Generator().manual_seed(seed))
        q[:, :, 0] = unit * math.log(2.0) * math.sqrt(d) / 0.01
        q[1::2, :, 0] *= -1
        return q.to(torch.bfloat16)

    return c, host, table, queries


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [40, 300])
def test_maxima_that_rise_with_every_32_keys(d, rows):
    """V scales that keep every page on the key-by-key path of the tiles: each 32 keys lie 2^12 above the ones before,
    so what the step has stored of its probabilities and O follow the maximum up to four times a step."""
    n = 64 * 9 + 40
    levels = [-120 + 12 * (j // 32) for j in range(n)]
    c, host, table, queries = ladder(d, levels, 1.0, scale=2.0 ** -70, seed=d + rows)
    check_forward(c, host, table, [n], [rows], 2, q=queries(2, rows))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [40, 300])
def test_maxima_that_jump_between_the_pages_of_a_step(d, rows):
    """Whole pages: the second of each pair lies 2^70 above the first one, so the first one's stored probabilities
    follow; the next pair's first page stays at that level."""
    n = 64 * 14
    levels = [-120 + 35 * ((j // 64 + 1) // 2) for j in range(n)]
    c, host, table, queries = ladder(d, levels, 2.0, seed=d + rows)
    check_forward(c, host, table, [n], [rows], 2, q=queries(2, rows))


def test_calls_refuse_a_workspace_of_the_host():
    c, _ = make_cache(2, 1, 64)
    x = torch.zeros(1, 3, 64, dtype=torch.bfloat16, device=DEV)
    before = [t.clone() for t in (c.k, c.k_scale)]
    args = i32([0, 3]), i32([0]), i32([[0]])
    ws = torch.zeros(1 << 26, dtype=torch.uint8)
    for call in (lambda: h3.cache_append(c, x, x, *args, ws=ws), lambda: h3.cache_read(c, *args, T=3, ws=ws),
                 lambda: h3.cache_forward(c, x, *args, ws=ws)):
        with pytest.raises(ValueError, match="ws must be contiguous on cuda:0, not on cpu"):
            call()
    assert torch.equal(c.k, before[0]) and torch.equal(c.k_scale, before[1])
