"""The paged int8 cache at the ends of its range, against fp64 with the bounds of cache_ref: running maxima that rise
again and again inside a step, V scales from nothing to 1e30, long caches of zeros, penalties that mask;
workspaces that are not the device's; what the status word keeps; waits that run out;
thousands of sequences; calls behind one another and captured."""
import math

import pytest
import torch

import biased_attention_video_b200 as h3
from cache_ref import bounds
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


@pytest.mark.parametrize("cap", [1e9, 1e10, 3e38])
@pytest.mark.parametrize("rows,one_time", [(1, True), (12, False), (40, True), (300, True), (300, False)])
def test_penalty_as_a_mask(cap, rows, one_time):
    """Every key outside the window is masked by the cap; a row's first keys are, and what it does see has scores of
    several hundred.  With one_time pages of one guide time, else the keys of a page alternate between two."""
    n = 64 * 10 + 20
    c, host = make_cache(11, 1, 128, seed=rows, times=True)
    table = make_table([n], 11, seed=rows)
    for i, p in enumerate(table[0]):  # the queries' times are multiples of 0.17 up to 1.87, or none
        host[4][p] = 5.0 if i < 6 else 0.17 * (i % 3)
        if not one_time:
            host[4][p, ::2] = 5.0
        if i == 8:
            host[4][p] = float("nan")
    c.times.copy_(host[4])
    check_forward(c, host, table, [n], [rows], 2, pen=(cap, 2.0, 0.01, cap), q_scale=60.0, seed=rows)


@pytest.mark.parametrize("rows,one_time", [(2, True), (300, True), (300, False)])
def test_rows_whose_keys_are_all_masked_count_nothing_in_a_merge(rows, one_time):
    n = 64 * 6 + 9
    c, host = make_cache(7, 2, 128, seed=rows, times=True)
    c.times.fill_(5.0)
    if not one_time:
        c.times[:, ::2] = 7.0
    q = 60 * torch.randn(2, rows, 128, device=DEV)
    args = q.to(torch.bfloat16), i32([0, rows]), i32([n]), i32(make_table([n], 7))
    o, lse = h3.cache_forward(c, *args, pen=(1e9, 2.0, 0.01, 1e9), q_times=torch.zeros(rows, device=DEV), lse=True)
    top = 127 * float(host[3].max())
    assert torch.all(o.abs() <= top * 1.02) and torch.all((lse + 2.0 ** 26 * math.log(2.0)).abs() <= 1e4)
    p, lp = h3.cache_forward(c, *args, lse=True)
    m, lm = h3.merge([o, p], [lse, lp], lse=True)
    assert torch.equal(m, p) and torch.equal(lm, lp)


V_SCALES = {  # pages of a sequence; what lies between is ordinary
    "pages of zero": {0: 0.0, 3: 0.0, 8: 0.0},
    "all zero": dict.fromkeys(range(9), 0.0),
    "below the smallest normal": {1: 2.0 ** -140, 4: 2.0 ** -149, 8: 2.0 ** -127},
    "about the ends": {0: 2.0 ** -61, 1: 2.0 ** -60, 2: 2.0 ** -59, 3: 0.0, 8: 2.0 ** -62},
    "all tiny": dict.fromkeys(range(9), 2.0 ** -80),
    "large": {2: 2.0 ** 39, 3: 2.0 ** 41, 8: 2.0 ** 40},
    "huge": {2: 1e30, 5: 0.0},
    "huge at the end": {8: 1e30},
}


@pytest.mark.parametrize("scales", list(V_SCALES))
@pytest.mark.parametrize("d,rows,causal", [(64, 1, False), (128, 1, False), (128, 5, True), (64, 16, True), (128, 150, True),
                                           (64, 150, False)])
def test_values_of_any_scale(scales, d, rows, causal):
    """A key counts in the normaliser whatever its value's scale; causal rows see less than the last page."""
    lengths = [64 * 8 + 50]
    c, host = make_cache(9, 1, d, seed=d + rows)
    table = make_table(lengths, 9)
    for p, scale in V_SCALES[scales].items():
        host[3][table[0][p], 0] = scale
    c.v_scale.copy_(host[3])
    check_forward(c, host, table, lengths, [rows], 2, causal=causal, seed=rows)


@pytest.mark.parametrize("d,H,rows", [(64, 1, 1), (128, 2, 7), (64, 2, 40)])
def test_a_long_cache_of_zeros(d, H, rows):
    """131,072 rows of zero keys and values: O = 0 and LSE = log 131072.  The sums are powers of two and exact; the
    logarithm of the scale has a relative error of 2^-22 of at most 60, what follows a few roundings of 2^-24 of 89."""
    n = 1 << 17
    c = h3.Cache.empty(n // 64, 1, d)
    table = torch.randperm(n // 64, device=DEV).to(torch.int32)[None]
    ws = h3.cache_workspace(c, H, rows, 1)
    x = torch.zeros(1, n, d, dtype=torch.bfloat16, device=DEV)
    h3.cache_append(c, x, x, i32([0, n]), i32([0]), table, ws=ws)
    q = torch.randn(H, rows, d, device=DEV).to(torch.bfloat16)
    o, lse = h3.cache_forward(c, q, i32([0, rows]), i32([n]), table, ws=ws, lse=True)
    assert h3.check(ws) == h3.OK
    assert torch.all(o == 0) and torch.all((lse - math.log(n)).abs() <= 2.0 ** -15)


@pytest.mark.parametrize("rows", [1, 40])
def test_a_long_cache_whose_first_page_is_lower(rows):
    """116,883 rows of zero values; all but the first page lie 2^2 above it, less than what raises the few-row kernel's
    maximum, so the normaliser's terms stay four times larger than at their maximum."""
    n = 116883
    c, host, table, queries = ladder(64, [0 if j < 64 else 100 for j in range(n)], 0.02, scale=0.0)
    q = queries(1, rows)
    q[:, :, 1:] = 0
    check_forward(c, host, table, [n], [rows], 1, q=q)


@pytest.mark.parametrize("rows", [1, 5, 150])
def test_marked_values_leave_the_normaliser(rows):
    """A V scale of NaN makes the output NaN and leaves LSE as it is; a K scale of NaN makes both NaN."""
    c, _ = make_cache(3, 1, 128, seed=2)
    q = torch.randn(2, rows, 128, device=DEV).to(torch.bfloat16)
    args = q, i32([0, rows]), i32([130]), i32([[0, 1, 2]])
    _, want = h3.cache_forward(c, *args, lse=True)
    c.v_scale[1, 0] = float("nan")
    o, lse = h3.cache_forward(c, *args, lse=True)
    # the same scores and sums, in another order of roundings of 2^-24 and with the scale's logarithm (2^-22 of 60)
    assert torch.all(torch.isnan(o)) and torch.all((lse - want).abs() <= 2.0 ** -15)
    c.k_scale[1, 0] = float("nan")
    o, lse = h3.cache_forward(c, *args, lse=True)
    assert torch.all(torch.isnan(o)) and torch.all(torch.isnan(lse))


def test_a_give_up_is_not_hidden_by_bad_data():
    """A bad page id is recorded first; then a wait that runs out on the same workspace (one that nothing arrives at),
    which says more: its output is incomplete.  The other way round the give-up stays."""
    c, _ = make_cache(2, 1, 64)
    x = torch.zeros(1, 3, 64, dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    bad = i32([0, 3]), i32([0]), i32([[7]])
    h3.cache_append(c, x, x, *bad, ws=ws)
    assert h3.check(ws) == h3.EDATA
    h3.cache_append(c, x, x, *bad, ws=ws)
    h3.selftest_timeout(ws, 100)
    assert h3.check(ws) == h3.ETIMEOUT
    h3.selftest_timeout(ws, 100)
    h3.cache_append(c, x, x, *bad, ws=ws)
    assert h3.check(ws) == h3.ETIMEOUT and h3.check(ws) == h3.OK


@pytest.mark.parametrize("d,rows,length,pen", [(128, 300, 2000, False), (64, 40, 100, False), (128, 1500, 900, True),
                                               (64, 300, 4000, True)])
def test_tiles_give_up_and_recover(d, rows, length, pen):
    """Every wait of the tile kernel bounded to one poll, which does not suspend: the first wait for rows from memory runs
    out, the block's roles leave, and the word says so, also when a bad page was recorded.  With larger limits roles leave
    at other steps, or none does and the output is whole.  Each time the next call on the same workspace is right."""
    c, host = make_cache(length // 64 + 3, 2, d, seed=21, times=pen)
    table = make_table([length], length // 64 + 3, width=length // 64 + 2)
    ws = h3.cache_workspace(c, 2, rows, 1)
    q = torch.randn(2, rows, d, device=DEV).to(torch.bfloat16)
    more = dict(pen=h3.DEFAULT_PENALTY, q_times=torch.rand(rows, device=DEV)) if pen else {}
    args = q, i32([0, rows]), i32([length]), i32(table)
    want, _ = h3.cache_forward(c, *args, **more)

    def bounded(polls, page_table):
        try:
            h3.set_wait_polls(polls)
            o, _ = h3.cache_forward(c, *args[:3], page_table, ws=ws, **more)
            return o, h3.check(ws)
        finally:
            h3.set_wait_polls(0)

    bad = table.copy()
    bad[0][0] = -1
    for polls, page_table in [(1, table), (1, bad), (3, table), (10, table), (30, table), (100, table), (1000, table)]:
        o, status = bounded(polls, i32(page_table))
        assert status == h3.ETIMEOUT or (polls > 1 and status == h3.OK and torch.equal(o, want)), polls
        o, _ = h3.cache_forward(c, *args, ws=ws, **more)
        assert h3.check(ws) == h3.OK and torch.equal(o, want), polls


@pytest.mark.parametrize("B,H,max_rows", [(3000, 2, 2), (3000, 2, None), (65536, 1, 1), (65536, 1, None)])
def test_thousands_of_sequences(B, H, max_rows):
    """Sequences of at most four cached rows and one or two new ones, many of them empty: appended, read back, attended."""
    d, g = 64, torch.Generator(device=DEV).manual_seed(B + H)
    pick = lambda hi: torch.randint(0, hi, (B,), generator=g, device=DEV)
    n = torch.minimum(pick(2 if max_rows == 1 else 3), pick(3))
    length = pick(4)
    n[-1], length[-1] = 1, 3
    start = torch.cat([n.new_zeros(1), n.cumsum(0)]).to(torch.int32)
    T = int(start[-1])
    table = torch.randperm(B, generator=g, device=DEV).to(torch.int32)[:, None]
    c = h3.Cache(*(torch.randint(-127, 128, (B, 1, 64, d), generator=g, device=DEV, dtype=torch.int8) for _ in range(2)),
                 *(0.005 + 0.03 * torch.rand(B, 1, generator=g, device=DEV) for _ in range(2)))
    ws = h3.cache_workspace(c, H, T, B)
    held = length.to(torch.int32)
    now = held + n.to(torch.int32)
    x = torch.randn(2, 1, T, d, generator=g, device=DEV).to(torch.bfloat16)
    h3.cache_append(c, x[0], x[1], start, held, table, ws=ws)
    kb, vb = h3.cache_read(c, start, held, table, T=T, ws=ws)
    seq = torch.repeat_interleave(torch.arange(B, device=DEV), n)
    page = table[seq, 0].long()
    for back, new, scale in ((kb, x[0], c.k_scale), (vb, x[1], c.v_scale)):
        # half a step and its rounding in fp32, then the rounding to bf16
        step = scale[page]
        assert torch.all((back[0].float() - new[0].float()).abs() <= 0.501 * step + 2.0 ** -8 * (new[0].float().abs() + step))
    q = torch.randn(H, T, d, generator=g, device=DEV).to(torch.bfloat16)
    o, lse = h3.cache_forward(c, q, start, now, table, max_rows=max_rows, ws=ws, lse=True)
    assert h3.check(ws) == h3.OK
    k, v = ((codes[:, 0, :6].double() * scale.double()[..., None])[page] for codes, scale in ((c.k, c.k_scale), (c.v, c.v_scale)))
    s = torch.einsum("htd,tjd->htj", q.double(), k) / math.sqrt(d)
    s = s.masked_fill(torch.arange(6, device=DEV) >= now[seq].long()[:, None], -math.inf)
    ref_l = torch.logsumexp(s, -1)
    w = torch.exp(s - ref_l[..., None])
    reach = torch.einsum("htd,tjd->htj", q.double().abs(), k.abs()).amax(-1) / math.sqrt(d)
    ref_o = torch.einsum("htj,tjd->htd", w, v)
    tol_o, tol_l = bounds(ref_o, ref_l, torch.einsum("htj,tjd->htd", w, v.abs()), reach, 6, d)
    assert torch.all((o.double() - ref_o).abs() <= tol_o) and torch.all((lse.double() - ref_l).abs() <= tol_l)


def test_captured_calls_behind_copies_and_joins():
    """One graph: a copy, few rows, tiles on the same workspace, a merge, then few rows and tiles again behind work of
    another stream; each replay with new queries and lengths equals the calls one by one."""
    c, _ = make_cache(40, 2, 128, seed=9)
    table = i32(make_table([1200, 1300], 40))
    few, many = 3, 150
    g = torch.Generator(device=DEV).manual_seed(0)
    qs = torch.randn(4, 4, 2 * many, 128, generator=g, device=DEV).to(torch.bfloat16)
    lens = [i32(x) for x in ([1200, 1300], [1, 700], [0, 65], [999, 128])]
    start_few, start_many = i32([0, few, 2 * few]), i32([0, many, 2 * many])
    side = torch.cuda.Stream()

    def calls(q, x, length, ws):
        here = torch.cuda.current_stream()
        q.copy_(x)
        a, la = h3.cache_forward(c, q[:, :2 * few], start_few, length, table, max_rows=few, ws=ws, lse=True)
        b, lb = h3.cache_forward(c, q, start_many, length, table, max_rows=many, ws=ws, lse=True)
        m, lm = h3.merge([b, b], [lb, lb], lse=True)
        side.wait_stream(here)
        with torch.cuda.stream(side):
            twice = q * 2
        here.wait_stream(side)
        e, le = h3.cache_forward(c, twice[:, :2 * few], start_few, length, table, causal=True, max_rows=few, ws=ws, lse=True)
        side.wait_stream(here)
        with torch.cuda.stream(side):
            thrice = twice * 1.5
        here.wait_stream(side)
        f, lf = h3.cache_forward(c, thrice, start_many, length, table, causal=True, max_rows=many, ws=ws, lse=True)
        return a, la, b, lb, m, lm, e, le, f, lf

    ws = [h3.cache_workspace(c, 4, 2 * many, 2) for _ in range(2)]
    q = [qs[0].clone() for _ in range(2)]
    x_in, len_in = qs[0].clone(), lens[0].clone()
    calls(q[0], x_in, len_in, ws[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(q[0], x_in, len_in, ws[0])
    for _ in range(3):
        for x, length in zip(qs, lens):
            x_in.copy_(x), len_in.copy_(length)
            graph.replay()
            want = calls(q[1], x, length, ws[1])
            for i, (a, b) in enumerate(zip(got, want)):
                assert torch.equal(a.nan_to_num(), b.nan_to_num()), i
    assert h3.check(ws[0]) == h3.OK and h3.check(ws[1]) == h3.OK


def test_calls_right_behind_one_another():
    """Append, few rows and tiles in turn without a pause, one workspace, the length moving on the device: as with a
    synchronisation after every call."""
    out = []
    for pause in (False, True):
        c, _ = make_cache(30, 2, 64, seed=3)
        table = i32(make_table([600, 900], 30))
        g = torch.Generator(device=DEV).manual_seed(5)
        ws = h3.cache_workspace(c, 6, 240, 2)
        length, res = i32([3, 64]), []
        for i, n in enumerate([1, 120, 2, 1, 64, 5, 120, 1, 1, 3]):
            start = i32([0, n, 2 * n])
            x = torch.randn(10, 2 * n, 64, generator=g, device=DEV).to(torch.bfloat16)
            h3.cache_append(c, x[:2], x[2:4], start, length, table, ws=ws)
            if pause:
                torch.cuda.synchronize()
            length += n
            res += h3.cache_forward(c, x[4:], start, length, table, causal=True, max_rows=n, ws=ws, lse=True)
            if pause:
                torch.cuda.synchronize()
        res += h3.cache_read(c, i32([0, 318, 636]), i32([3, 64]), table, T=636, ws=ws)
        assert h3.check(ws) == h3.OK
        out.append(res)
    assert all(torch.equal(a, b) for a, b in zip(*out))


@pytest.mark.parametrize("rows,bad", [(4, [1, 3]), (150, [0, 77])])
def test_queries_that_are_not_finite_spoil_their_own_rows(rows, bad):
    lengths = [64 * 5 + 7]
    c, host = make_cache(6, 1, 128, seed=rows)
    table = make_table(lengths, 6)
    q = torch.randn(2, rows, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    args = i32([0, rows]), i32(lengths), i32(table)
    want, want_l = h3.cache_forward(c, q, *args, lse=True)
    q[:, bad[0], 5] = float("nan")
    q[:, bad[1], 9] = float("inf")
    o, lse = h3.cache_forward(c, q, *args, lse=True)
    rest = [i for i in range(rows) if i not in bad]
    assert torch.all(torch.isnan(o[:, bad])) and torch.all(torch.isnan(lse[:, bad]))
    # the other rows' running maximum may lie elsewhere: twice the roundings of 2^-8 of probabilities and output
    top = 127 * float(host[3].max())
    assert torch.all((o[:, rest].float() - want[:, rest].float()).abs() <= 2.0 ** -6 * top)
    assert torch.all((lse[:, rest] - want_l[:, rest]).abs() <= 2.0 ** -15)
