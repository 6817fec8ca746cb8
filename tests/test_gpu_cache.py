"""The paged int8 cache on the GPU: append (bit for bit against the fp32 rule), read, attention (against fp64 with
derived bounds), and the three together with the library's forward and merge."""
import math

import numpy as np
import pytest
import torch

import biased_attention_video_b200 as h3
import inputs
from cache_ref import HostCache, attend, bounds, rotate, values

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def offsets(counts):
    return i32(np.concatenate([[0], np.cumsum(counts)]))


def make_cache(n_pages, H, d, seed=0, times=False):
    """A cache full of arbitrary codes and scales."""
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randint(-127, 128, (n_pages, H, 64, d), generator=g, dtype=torch.int8) for _ in range(2))
    ks, vs = (0.005 + 0.03 * torch.rand(n_pages, H, generator=g) for _ in range(2))
    t = None
    if times:
        t = torch.randint(0, 12, (n_pages, 64), generator=g).float() * 0.17
        t[torch.rand(n_pages, 64, generator=g) < 0.3] = float("nan")
    c = h3.Cache(*(x.to(DEV) for x in (k, v, ks, vs)), times=None if t is None else t.to(DEV))
    return c, (k, v, ks, vs, t)


def make_table(lengths, n_pages, seed=0, width=None):
    """Disjoint pages in random order; unused entries hold an id far outside the cache."""
    ids = np.random.default_rng(seed).permutation(n_pages)
    need = [-(-n // 64) for n in lengths]
    assert sum(need) <= n_pages
    table = np.full((len(lengths), width or max(1, max(need))), 1 << 30, np.int64)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table


# --------------------------------------------------------------------- append


def host_state(c):
    return [t.cpu().numpy() for t in (c.k, c.v, c.k_scale, c.v_scale)]


def same_cache(c, ref, live):
    """Codes of the live rows [(page, rows)] and all scales, bit for bit."""
    k, v, ks, vs = host_state(c)
    for got, which in ((k, "k"), (v, "v")):
        for page, n in live:
            assert np.array_equal(got[page, :, :n], ref.codes[which][page, :, :n]), (which, page)
    assert np.array_equal(ks, ref.scale["k"], equal_nan=True)
    assert np.array_equal(vs, ref.scale["v"], equal_nan=True)


APPENDS = [  # d, H, rotation (None or interleaved, dim), rows held and new rows of each sequence, padding
    (128, 2, (False, 128), [(0, 1)], 0),
    (128, 3, (True, 128), [(0, 64), (63, 1), (64, 1), (65, 2)], 5),
    (64, 2, (False, 64), [(5, 0), (0, 200), (130, 61), (61, 3)], 1),
    (64, 1, (True, 32), [(17, 46), (100, 29)], 0),
    (128, 2, (False, 48), [(1, 127), (127, 130)], 0),
    (128, 5, None, [(n, 1) for n in range(0, 320, 7)], 2),
]


@pytest.mark.parametrize("d,H,rot,rows,pad", APPENDS)
def test_append_matches_the_rule_bit_for_bit(d, H, rot, rows, pad):
    rng = np.random.default_rng(d + H + len(rows))
    held, new = [r[0] for r in rows], [r[1] for r in rows]
    n_pages = sum(-(-(a + n) // 64) for a, n in rows) + 2
    table = make_table([a + n for a, n in rows], n_pages, seed=H)
    c, _ = make_cache(n_pages, H, d, seed=d)
    ref = HostCache(*host_state(c))
    T = sum(new) + pad
    x = torch.from_numpy(rng.normal(size=(2, H, T, d)).astype(np.float32) * rng.choice([0.2, 1, 5], size=(2, H, T, 1))
                         .astype(np.float32)).to(torch.bfloat16)
    x[:, :, sum(new):] = float("nan")  # padding rows are not read
    rope = None
    n_pos = max(a + n for a, n in rows)
    if rot is not None:
        ang = rng.uniform(-3, 3, size=(n_pos, rot[1] // 2))
        cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
        rope = h3.Rope(torch.from_numpy(cos).to(DEV), torch.from_numpy(sin).to(DEV), interleaved=rot[0])
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    h3.cache_append(c, x[0].to(DEV), x[1].to(DEV), offsets(new), i32(held), i32(table), rope=rope, ws=ws)
    assert h3.check(ws) == h3.OK
    at, live = 0, []
    for b, (a, n) in enumerate(rows):
        k, v = (x[i, :, at:at + n].float().numpy() for i in range(2))
        if rot is not None:
            k = rotate(k, cos[a:a + n], sin[a:a + n], rot[1], rot[0])
        ref.append("k", k, table[b], a)
        ref.append("v", v, table[b], a)
        live += [(table[b][p], min(64, a + n - 64 * p)) for p in range(-(-(a + n) // 64))]
        at += n
    untouched = set(range(n_pages)) - {p for p, _ in live}
    same_cache(c, ref, live + [(p, 64) for p in untouched])


def test_append_token_by_token_stays_within_its_steps():
    """130 single rows of growing size: codes as the rule gives them, and every stored value within half a step of the
    value for its own rounding and half a step for each time its page's scale grew after it."""
    rng = np.random.default_rng(3)
    H, d, n = 2, 128, 130
    c, _ = make_cache(5, H, d)
    ref = HostCache(*host_state(c))
    table = np.array([[4, 1, 2]])
    x = torch.from_numpy((rng.normal(size=(2, H, n, d)) * np.linspace(0.5, 4, n)[:, None]).astype(np.float32)).to(
        torch.bfloat16)
    grew = np.zeros((2, H, n))
    for t in range(n):
        before = [ref.scale["k"].copy(), ref.scale["v"].copy()]
        h3.cache_append(c, x[0, :, t:t + 1].to(DEV), x[1, :, t:t + 1].to(DEV), i32([0, 1]), i32([t]), i32(table))
        for i, which in enumerate("kv"):
            ref.append(which, x[i, :, t:t + 1].float().numpy(), table[0], t)
            page = table[0][t // 64]
            if t % 64:
                for h in range(H):
                    if ref.scale[which][page, h] > before[i][page, h]:
                        grew[i, h, t // 64 * 64:t] += 1
    same_cache(c, ref, [(4, 64), (1, 64), (2, 2)])
    for i, (codes, scale) in enumerate(((c.k, c.k_scale), (c.v, c.v_scale))):
        got = values(codes.cpu(), scale.cpu(), table[0], n)
        step = scale.cpu().double()[torch.as_tensor(table[0])][:, :].repeat_interleave(64, 0)[:n].t()
        allowed = (0.5 + 0.5 * torch.from_numpy(grew[i])) * step * (1 + 2.0 ** -14)
        assert torch.all((got - x[i].double()).abs() <= allowed[..., None])


def test_append_takes_strided_rows_and_table_rows_by_index():
    """K and V inside one projection's output [T, heads + extra, d]; rotation rows by index."""
    rng = np.random.default_rng(5)
    H, d, n = 4, 128, 150
    c, _ = make_cache(4, H, d)
    ref = HostCache(*host_state(c))
    table = np.array([[3, 0, 2]])
    proj = torch.from_numpy(rng.normal(size=(n, 3 * H + 1, d)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    k, v = proj[:, H:2 * H].transpose(0, 1), proj[:, 2 * H:3 * H].transpose(0, 1)
    ang = rng.uniform(-3, 3, size=(40, 64))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    index = rng.integers(0, 40, size=n)
    rope = h3.Rope(torch.from_numpy(cos).to(DEV), torch.from_numpy(sin).to(DEV), index=i32(index), interleaved=True)
    h3.cache_append(c, k, v, i32([0, n]), i32([0]), i32(table), rope=rope)
    ref.append("k", rotate(k.float().cpu().numpy(), cos[index], sin[index], 128, True), table[0], 0)
    ref.append("v", v.float().cpu().numpy(), table[0], 0)
    same_cache(c, ref, [(3, 64), (0, 64), (2, 22)])


def test_append_edge_values():
    """Zero rows, tiny rows (the smallest scale), the largest finite values, and values that are not finite, which
    mark their page and head only; appending at a smaller length starts the page over."""
    H, d = 2, 64
    c, _ = make_cache(3, H, d)
    ref = HostCache(*host_state(c))
    table = np.array([[0, 1, 2]])
    x = torch.zeros(2, H, 150, d)
    x[:, :, 64:128] = 2.0 ** -110
    x[:, :, 70, 3] = 2.0 ** -99
    x[0, 0, 130] = 3.0e38
    x = x.to(torch.bfloat16)
    h3.cache_append(c, x[0].to(DEV), x[1].to(DEV), i32([0, 150]), i32([0]), i32(table))
    for i, w in enumerate("kv"):
        ref.append(w, x[i].float().numpy(), table[0], 0)
    same_cache(c, ref, [(0, 64), (1, 64), (2, 22)])
    y = torch.ones(2, H, 3, d).to(torch.bfloat16)
    y[0, 1, 1, 5] = float("inf")
    y[1, 0, 2, 0] = float("nan")
    h3.cache_append(c, y[0].to(DEV), y[1].to(DEV), i32([0, 3]), i32([150]), i32(table))
    for i, w in enumerate("kv"):
        ref.append(w, y[i].float().numpy(), table[0], 150)
    same_cache(c, ref, [(0, 64), (1, 64)])
    assert torch.isnan(c.k_scale[2]).tolist() == [False, True]
    assert torch.isnan(c.v_scale[2]).tolist() == [True, False]
    # dropping rows: position 128 on is new, so the page's scale comes from the new rows alone
    z = torch.full((2, H, 2, d), 0.5).to(torch.bfloat16)
    h3.cache_append(c, z[0].to(DEV), z[1].to(DEV), i32([0, 2]), i32([128]), i32(table))
    for i, w in enumerate("kv"):
        ref.append(w, z[i].float().numpy(), table[0], 128)
    same_cache(c, ref, [(0, 64), (1, 64), (2, 2)])


def test_append_writes_guide_times():
    c, (_, _, _, _, t) = make_cache(3, 1, 64, times=True)
    table = i32([[2, 0]])
    x = torch.zeros(1, 70, 64, dtype=torch.bfloat16, device=DEV)
    rt = torch.arange(70, device=DEV, dtype=torch.float32)
    h3.cache_append(c, x, x, i32([0, 70]), i32([10]), table, row_times=rt)
    want = t.clone()
    want[2, 10:] = torch.arange(54.0)
    want[0, :16] = torch.arange(54.0, 70.0)
    assert torch.equal(c.times.cpu().nan_to_num(-1), want.nan_to_num(-1))
    h3.cache_append(c, x[:, :2], x[:, :2], i32([0, 2]), i32([11]), table)  # without times: no guide rows
    want[2, 11:13] = float("nan")
    assert torch.equal(c.times.cpu().nan_to_num(-1), want.nan_to_num(-1))


# ----------------------------------------------------------------------- read


@pytest.mark.parametrize("d,H", [(64, 3), (128, 1)])
def test_read_gives_the_stored_values_rounded_once(d, H):
    spans = [(0, 1), (3, 200), (64, 64), (100, 0), (63, 2)]  # first row, rows
    n_pages = 12
    table = make_table([a + n for a, n in spans], n_pages)
    c, (k, v, ks, vs, _) = make_cache(n_pages, H, d, seed=9)
    T = sum(n for _, n in spans) + 4
    args = offsets([n for _, n in spans]), i32([a for a, _ in spans]), i32(table)
    keep = torch.full((H, T, d), 7.0, dtype=torch.bfloat16, device=DEV)
    kb, vb = h3.cache_read(c, *args, k_out=keep.clone(), v_out=keep.clone())
    only, none = h3.cache_read(c, *args, v_out=keep.clone())[::-1]
    assert none is None and torch.equal(only, vb)
    at = 0
    for b, (a, n) in enumerate(spans):
        for got, codes, scale in ((kb, k, ks), (vb, v, vs)):
            want = values(codes, scale, table[b], a + n)[:, a:].float().to(torch.bfloat16)
            assert torch.equal(got[:, at:at + n].cpu(), want)
        at += n
    assert torch.all(kb[:, at:] == 7) and torch.all(vb[:, at:] == 7)
    k2, v2 = h3.cache_read(c, *args, T=T)
    assert torch.equal(k2[:, :at], kb[:, :at]) and torch.equal(v2[:, :at], vb[:, :at])


# -------------------------------------------------------------------- forward


def check_forward(c, host, table, lengths, rows, H, causal=False, pen=None, pad=0, seed=0, q=None, max_rows=None,
                  q_scale=1.0, ws=None):
    k, v, ks, vs, times = host
    d = k.shape[3]
    g = torch.Generator().manual_seed(seed)
    T = sum(rows) + pad
    if q is None:
        q = (q_scale * torch.randn(H, T, d, generator=g)).to(torch.bfloat16)
        q[:, sum(rows):] = float("nan")
    qt = None
    if pen is not None:
        qt = torch.randint(0, 12, (T,), generator=g).float() * 0.17
        qt[torch.rand(T, generator=g) < 0.3] = float("nan")
    out = torch.full((H, T, d), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((H, T), 7.0, device=DEV)
    if ws is None:
        ws = h3.cache_workspace(c, H, T, len(rows))
    h3.cache_forward(c, q.to(DEV) if not q.is_cuda else q, offsets(rows), i32(lengths), i32(table), causal=causal,
                     pen=pen, q_times=None if qt is None else qt.to(DEV), max_rows=max_rows, ws=ws, out=out, lse=lse)
    assert h3.check(ws) == h3.OK
    o, l, at = out.cpu().double(), lse.cpu().double(), 0
    for b, (L, n) in enumerate(zip(lengths, rows)):
        kk, vv = values(k, ks, table[b], L), values(v, vs, table[b], L)
        bias = None
        if pen is not None:
            tk = times[torch.as_tensor(table[b][: -(-L // 64)], dtype=torch.long)].reshape(-1)[:L].double()
            dt = (qt[at:at + n].double()[:, None] - tk).abs()
            s, w, f, cap = pen
            bias = -torch.nan_to_num((s * ((dt - w).clamp(min=0) / f) ** 2).clamp(max=cap), nan=0.0)
        ref_o, ref_l, spread, reach = attend(q[:, at:at + n].cpu().double(), kk, vv, causal, bias)
        tol_o, tol_l = bounds(ref_o, ref_l, spread, reach, max(L, 1), d)
        err = (o[:, at:at + n] - ref_o).abs()
        assert torch.all(err <= tol_o), (b, L, n, float((err / tol_o).max()))
        empty = torch.isinf(ref_l)
        assert torch.equal(torch.isinf(l[:, at:at + n]), empty) and torch.all(l[:, at:at + n][empty] < 0)
        errl = torch.where(empty, 0.0, (l[:, at:at + n] - ref_l).abs())
        assert torch.all(errl <= torch.where(empty, 1.0, tol_l)), (b, L, n, float((errl / tol_l).nan_to_num().max()))
        at += n
    assert torch.all(o[:, at:] == 7) and torch.all(l[:, at:] == 7)
    return out, lse


FORWARDS = [  # d, query heads, K/V heads, lengths, rows, causal, penalty, padding
    (128, 1, 1, [1], [1], False, None, 0),
    (128, 8, 8, [64, 65, 63, 0, 129], [1, 1, 1, 1, 1], False, None, 2),
    (128, 8, 2, [1000, 17, 333], [1, 1, 1], True, None, 0),
    (64, 7, 1, [100, 5, 700], [1, 2, 3], True, None, 1),
    (64, 6, 3, [31, 32, 33, 2000], [4, 9, 1, 17], False, h3.DEFAULT_PENALTY, 0),
    (128, 4, 4, [500], [8], True, h3.DEFAULT_PENALTY, 0),
    (128, 4, 1, [3, 70, 0], [9, 70, 5], True, None, 3),          # rows that see nothing
    (128, 2, 2, [640, 1], [33, 64], False, None, 0),
    (128, 3, 1, [900, 130], [300, 129], True, None, 0),
    (64, 2, 1, [257, 1025], [127, 260], False, None, 7),
    (64, 4, 4, [777], [513], True, h3.DEFAULT_PENALTY, 0),
    (128, 2, 1, [1500, 64, 0, 200], [400, 1, 300, 0], False, h3.DEFAULT_PENALTY, 0),
    (128, 16, 2, [2500] * 3, [1, 40, 5], True, None, 0),         # one call of short and long sequences
    (128, 56, 8, [5000], [1], False, None, 0),
    (64, 5, 5, [0], [3], False, None, 0),
]


@pytest.mark.parametrize("case", range(len(FORWARDS)))
@pytest.mark.parametrize("hint", [False, True])
def test_forward_matches_fp64(case, hint):
    d, H, kv, lengths, rows, causal, pen, pad = FORWARDS[case]
    n_pages = sum(-(-n // 64) for n in lengths) + 3
    table = make_table(lengths, n_pages, seed=case, width=max(-(-n // 64) for n in lengths) + 2)
    c, host = make_cache(n_pages, kv, d, seed=case, times=pen is not None)
    check_forward(c, host, table, lengths, rows, H, causal, pen, pad, seed=case, max_rows=max(rows) if hint else None)


@pytest.mark.parametrize("rows", [1, 40, 300])
def test_forward_with_strong_scores(rows):
    """Scores of several hundred: the running maximum moves by far more than a probability's range."""
    lengths = [700]
    c, host = make_cache(11, 2, 128, seed=4)
    check_forward(c, host, make_table(lengths, 11), lengths, [rows], 4, q_scale=60.0, seed=4)


@pytest.mark.parametrize("rows", [1, 40, 300])
def test_forward_with_scores_of_millions(rows):
    """Scores 127 2^15 (4.2 million) apart from the next by 2^15 or more: each row gets its best key's value.  The
    probability's rounding to 16 bits and the output's are 2^-8 of the value each; the score is a product of fp32
    factors with at most eight roundings of 2^-24 up to the normaliser."""
    L, d = 700, 64
    g = torch.Generator().manual_seed(8)
    k = torch.zeros(11, 1, 64, d, dtype=torch.int8)
    k[..., 0] = torch.randint(-126, 127, (11, 1, 64), generator=g, dtype=torch.int8)
    v = torch.randint(-127, 128, (11, 1, 64, d), generator=g, dtype=torch.int8)
    k[10, 0, 20, 0], k[4, 0, 7, 0] = 127, -127
    ks, vs = torch.full((11, 1), 2.0 ** -6), 0.005 + 0.03 * torch.rand(11, 1, generator=g)
    c = h3.Cache(*(x.to(DEV) for x in (k, v, ks, vs)))
    q = torch.zeros(2, rows, d, dtype=torch.bfloat16)
    q[0, :, 0], q[1, :, 0] = 2.0 ** 24, -(2.0 ** 24)
    ws = h3.cache_workspace(c, 2, rows, 1)
    o, lse = h3.cache_forward(c, q.to(DEV), i32([0, rows]), i32([L]), i32([list(range(11))]), ws=ws, lse=True)
    assert h3.check(ws) == h3.OK
    for h, (page, row) in enumerate([(10, 20), (4, 7)]):
        ref = (v[page, 0, row].double() * vs[page, 0].double()).expand(rows, d)
        assert torch.all((o[h].cpu().double() - ref).abs() <= (2.0 ** -7 + 2.0 ** -16) * ref.abs())
        assert torch.all((lse[h].cpu().double() - 127 * 2.0 ** 15).abs() <= 2.0 ** -21 * 127 * 2.0 ** 15)


@pytest.mark.parametrize("rows", [1, 40, 300])
def test_forward_scales_far_apart(rows):
    """Pages whose scales differ by many orders of magnitude, a page of zeros with the smallest scale among them."""
    lengths = [64 * 9]
    c, host = make_cache(9, 1, 128, seed=6)
    host[2][:, 0] = torch.tensor([2.0 ** -100, 1e-20, 1e-8, 1e-4, 1e-2, 0.02, 0.01, 3e-3, 1e-3])
    host[3][:, 0] = torch.tensor([1e-3, 2.0 ** -100, 50.0, 1e-12, 1e-2, 1e3, 0.01, 3e-3, 1e-20])
    host[0][0] = 0
    c.k_scale.copy_(host[2])
    c.v_scale.copy_(host[3])
    c.k.copy_(host[0])
    check_forward(c, host, make_table(lengths, 9), lengths, [rows], 2, seed=6)


@pytest.mark.parametrize("rows", [2, 200])
def test_forward_strided_queries_and_shared_pages(rows):
    """Two sequences over the same pages (a shared prefix), queries inside a projection's output."""
    table = np.array([[2, 0, 1, 4], [2, 0, 1, 3]])
    lengths = [250, 200]
    c, host = make_cache(5, 2, 128, seed=8)
    g = torch.Generator().manual_seed(1)
    proj = torch.randn(2 * rows, 9, 128, generator=g).to(torch.bfloat16).to(DEV)
    check_forward(c, host, table, lengths, [rows, rows], 6, q=proj[:, 1:7].transpose(0, 1), seed=2)


@pytest.mark.parametrize("rows", [1, 150])
def test_forward_ignores_what_lies_behind_the_length(rows):
    """Stale scales in unused pages, NaN times behind the end: none of it may reach a row."""
    lengths = [130]
    c, host = make_cache(4, 1, 64, seed=2, times=True)
    table = make_table(lengths, 4, width=4)
    unused = [p for p in range(4) if p not in table[0][:3]]
    c.k_scale[unused] = float("nan")
    c.v_scale[unused] = float("inf")
    table[0][3] = unused[0]
    check_forward(c, host, table, lengths, [rows], 2, pen=h3.DEFAULT_PENALTY, seed=3)


@pytest.mark.parametrize("rows", [1, 150])
def test_forward_of_a_marked_page_is_nan(rows):
    c, host = make_cache(3, 2, 128, seed=2)
    c.v_scale[1, 0] = float("nan")
    q = torch.randn(2, 2 * rows, 128, device=DEV).to(torch.bfloat16)
    o, _ = h3.cache_forward(c, q, offsets([rows, rows]), i32([130, 60]), i32([[0, 1, 2], [2, 0, 0]]))
    assert torch.all(torch.isnan(o[0, :rows])) and not torch.any(torch.isnan(o[1]))
    assert not torch.any(torch.isnan(o[:, rows:]))


@pytest.mark.parametrize("rows", [1, 150])
def test_forward_skips_and_reports_bad_pages(rows):
    c, host = make_cache(4, 1, 128, seed=5)
    q = torch.randn(1, rows, 128, device=DEV).to(torch.bfloat16)
    ws = h3.cache_workspace(c, 1, rows, 1)
    o, l = h3.cache_forward(c, q, i32([0, rows]), i32([192]), i32([[0, 4, 2]]), ws=ws, lse=True)
    assert h3.check(ws) == h3.EDATA and h3.check(ws) == h3.OK
    k, v = (torch.cat([values(a, s, [0], 64), values(a, s, [2], 64)], 1) for a, s in ((host[0], host[2]),
                                                                                     (host[1], host[3])))
    ref_o, ref_l, spread, reach = attend(q.cpu().double(), k, v)
    tol_o, tol_l = bounds(ref_o, ref_l, spread, reach, 128, 128)
    assert torch.all((o.cpu().double() - ref_o).abs() <= tol_o)
    assert torch.all((l.cpu().double() - ref_l).abs() <= tol_l)


def test_bad_rows_are_forced_into_range_and_reported():
    c, _ = make_cache(4, 1, 64)
    x = torch.ones(1, 8, 64, device=DEV).to(torch.bfloat16)
    ws = h3.cache_workspace(c, 1, 8, 2)
    before = [t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale)]
    for start, length, table in (([0, 9, 12], [0, 0], [[0], [1]]), ([-3, 2, 1], [0, 0], [[0], [1]]),
                                 ([0, 4, 8], [62, -5], [[0], [1]]), ([0, 4, 8], [0, 0], [[-1], [4]])):
        args = i32(start), i32(length), i32(table)
        h3.cache_append(c, x, x, *args, ws=ws)
        assert h3.check(ws) == h3.EDATA
        h3.cache_read(c, *args, T=8, ws=ws)
        assert h3.check(ws) == h3.EDATA
        h3.cache_forward(c, x, *args, ws=ws)
        assert h3.check(ws) == (h3.EDATA if start != [0, 4, 8] or length != [0, 0] else h3.OK)
    for t, b in zip((c.k, c.v, c.k_scale, c.v_scale), before):
        assert torch.equal(t[2:], b[2:])  # pages that no table names


def test_far_pages():
    """Codes past 2^31 bytes."""
    H, d = 8, 128
    n = (1 << 31) // (H * 64 * d) + 40
    c = h3.Cache(*(torch.zeros(n, H, 64, d, dtype=torch.int8, device=DEV) for _ in range(2)),
                 *(torch.ones(n, H, device=DEV) for _ in range(2)))
    table = np.array([[n - 1, n - 2, n - 3]])
    x = torch.randn(2, H, 150, d, device=DEV).to(torch.bfloat16)
    h3.cache_append(c, x[0], x[1], i32([0, 150]), i32([0]), i32(table))
    k, v = h3.cache_read(c, i32([0, 150]), i32([0]), i32(table), T=150)
    # half a step of a page's scale (its largest value / 127), and the rounding to bf16
    step = x.abs().amax().float() / 127
    for got, want in ((k, x[0]), (v, x[1])):
        assert torch.all((got.float() - want.float()).abs() <= 0.5 * step * 1.01 + 2.0 ** -8 * want.float().abs() + step * 2.0 ** -8)
    host = tuple(t[[n - 1, n - 2, n - 3]].cpu() for t in (c.k, c.v, c.k_scale, c.v_scale)) + (None,)
    for rows in (1, 100):
        q = torch.randn(H, rows, d, device=DEV).to(torch.bfloat16)
        o, l = h3.cache_forward(c, q, i32([0, rows]), i32([150]), i32(table), lse=True)
        ref_o, ref_l, spread, reach = attend(q.cpu().double(), values(host[0], host[2], [0, 1, 2], 150),
                                             values(host[1], host[3], [0, 1, 2], 150))
        tol_o, tol_l = bounds(ref_o, ref_l, spread, reach, 150, d)
        assert torch.all((o.cpu().double() - ref_o).abs() <= tol_o)
        assert torch.all((l.cpu().double() - ref_l).abs() <= tol_l)


# ------------------------------------------------------------------- together


def test_captured_append_and_attention_follow_the_lengths():
    """A decode loop as a captured graph: each replay appends one row and attends to all rows so far; the lengths move
    on the device.  Every step equals the same calls made one by one on a second cache."""
    H, kv, d, B, steps = 4, 2, 128, 2, 70
    cs = [make_cache(8, kv, d, seed=1)[0] for _ in range(2)]
    table = i32(make_table([128, 128], 8))
    g = torch.Generator(device=DEV).manual_seed(0)
    xs = torch.randn(steps, 2 * kv + H, B, d, generator=g, device=DEV).to(torch.bfloat16)
    start = i32([0, 1, 2])

    def step(c, x, length, ws):
        h3.cache_append(c, x[:kv], x[kv:2 * kv], start, length, table, ws=ws)
        length += 1
        return h3.cache_forward(c, x[2 * kv:], start, length, table, causal=True, max_rows=1, ws=ws, lse=True)

    ws = [h3.cache_workspace(cs[0], H, B, B) for _ in range(2)]
    lens = [i32([0, 3]) for _ in range(2)]
    x_in = xs[0].clone()
    step(cs[0], x_in, lens[0], ws[0])  # warm-up; what it wrote is replaced
    lens[0].copy_(i32([0, 3]))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o_g, l_g = step(cs[0], x_in, lens[0], ws[0])
    cs[0].k.copy_(cs[1].k), cs[0].v.copy_(cs[1].v)
    cs[0].k_scale.copy_(cs[1].k_scale), cs[0].v_scale.copy_(cs[1].v_scale)
    for t in range(steps):
        x_in.copy_(xs[t])
        graph.replay()
        o, l = step(cs[1], xs[t], lens[1], ws[1])
        assert torch.equal(o, o_g) and torch.equal(l, l_g), t
    assert torch.equal(cs[0].k, cs[1].k) and torch.equal(cs[0].k_scale, cs[1].k_scale)
    assert h3.check(ws[0]) == h3.OK and h3.check(ws[1]) == h3.OK


def test_cached_prefix_merges_with_the_forward_of_the_rest():
    """Guide rows from the cache, output rows through the library's dense forward, merged: the attention over both,
    against fp64 on the stored guide values; and the same with the guide rows read back into one bf16 call."""
    cfg = inputs.custom(2, 128, [inputs.Segment(inputs.SEG_GUIDE, 3 * 100, 3), inputs.Segment(inputs.SEG_OUTPUT, 3 * 90, 3)],
                        seed=41)
    seg, times, _ = cfg.layout()
    q, k, v = (torch.from_numpy(inputs.tensor(cfg, t).view(np.int16)).view(torch.bfloat16) for t in range(3))
    n, m = 300, 270
    c = h3.Cache.empty(6, 2, 128, times=True)
    table = i32([[5, 3, 0, 1, 2]])
    h3.cache_append(c, k[:, :n].to(DEV), v[:, :n].to(DEV), i32([0, n]), i32([0]), table,
                    row_times=torch.from_numpy(times[:n]).to(DEV))
    o1, l1 = h3.cache_forward(c, q[:, n:].to(DEV), i32([0, m]), i32([n]), table, pen=inputs.DEFAULT_PENALTY,
                              q_times=torch.from_numpy(times[n:]).to(DEV), lse=True)
    rest = [x[:, n:].contiguous().to(DEV) for x in (q, k, v)]
    o2, l2 = h3.dense_biased(*rest, torch.from_numpy(seg[n:]).to(DEV), torch.from_numpy(times[n:]).to(DEV), lse=True)
    o, l = h3.merge([o1, o2], [l1, l2], lse=True)
    # fp64 over the stored guide rows and the output rows
    host = [t.cpu() for t in (c.k, c.v, c.k_scale, c.v_scale)]
    kk = torch.cat([values(host[0], host[2], [5, 3, 0, 1, 2], n), k[:, n:].double()], 1)
    vv = torch.cat([values(host[1], host[3], [5, 3, 0, 1, 2], n), v[:, n:].double()], 1)
    t64 = torch.from_numpy(times).double()
    s, w, f, cap = inputs.DEFAULT_PENALTY
    bias = torch.zeros(m, n + m, dtype=torch.float64)
    bias[:, :n] = -(s * (((t64[n:, None] - t64[:n]).abs() - w).clamp(min=0) / f) ** 2).clamp(max=cap)
    ref_o, ref_l, spread, reach = attend(q[:, n:].double(), kk, vv, bias=bias)
    tol_o, tol_l = bounds(ref_o, ref_l, spread, reach, n + m, 128)
    # each partition's output is rounded to bf16 before the merge rounds once more
    assert torch.all((o.cpu().double() - ref_o).abs() <= tol_o + 2.0 ** -8 * spread)
    assert torch.all((l.cpu().double() - ref_l).abs() <= 2 * tol_l)
    kb, vb = h3.cache_read(c, i32([0, n]), i32([0]), table, T=n)
    full = [q.to(DEV), torch.cat([kb, rest[1]], 1), torch.cat([vb, rest[2]], 1)]
    o3, l3 = h3.dense_biased(*full, torch.from_numpy(seg).to(DEV), torch.from_numpy(times).to(DEV), lse=True)
    # reading back rounds every stored value to bf16: 2^-8 of each score's terms and of each value
    loose = 2.0 ** -8 * (1 + 2 * reach[..., None]) * spread
    assert torch.all((o3[:, n:].cpu().double() - ref_o).abs() <= tol_o + loose)


def test_calls_on_another_stream_and_device_order():
    """Calls on a side stream, workspace and outputs allocated by the call."""
    c, host = make_cache(6, 2, 128, seed=3)
    table = make_table([300], 6)
    s = torch.cuda.Stream()
    q = torch.randn(2, 5, 128, device=DEV).to(torch.bfloat16)
    s.wait_stream(torch.cuda.current_stream())
    o, l = h3.cache_forward(c, q, i32([0, 5]), i32([300]), i32(table), lse=True, stream=s)
    s.synchronize()
    torch.cuda.current_stream().wait_stream(s)
    o2, l2 = h3.cache_forward(c, q, i32([0, 5]), i32([300]), i32(table), lse=True)
    assert torch.equal(o, o2) and torch.equal(l, l2)
    with pytest.raises(ValueError, match="page_table"):
        h3.cache_forward(c, q, i32([0, 5]), i32([300]), torch.from_numpy(table), lse=True)
    with pytest.raises(ValueError, match="q must be"):
        h3.cache_forward(c, q.float(), i32([0, 5]), i32([300]), i32(table))
    with pytest.raises(h3.H3Error):
        h3.cache_forward(c, torch.randn(3, 5, 128, device=DEV).to(torch.bfloat16), i32([0, 5]), i32([300]), i32(table))


@pytest.mark.parametrize("rows", [6, 150])
def test_a_marked_page_stays_away_from_rows_that_do_not_see_it(rows):
    """Causal rows: the ones whose last key lies before the marked page are as they would be without it."""
    c, host = make_cache(4, 1, 128, seed=12)
    n = 128 + rows // 2                       # rows i < rows - n % 64 ... end before position 128
    q = torch.randn(1, rows, 128, device=DEV).to(torch.bfloat16)
    args = q, i32([0, rows]), i32([n]), i32([[0, 1, 2, 3]])
    want, want_l = h3.cache_forward(c, *args, causal=True, lse=True)
    for scale in (c.k_scale, c.v_scale):
        scale[2, 0] = float("nan")
    o, l = h3.cache_forward(c, *args, causal=True, lse=True)
    clean = 128 - (n - rows)                  # row i sees keys up to n - rows + i
    assert 0 < clean < rows
    assert torch.equal(o[:, :clean], want[:, :clean]) and torch.equal(l[:, :clean], want_l[:, :clean])
    assert torch.all(torch.isnan(o[:, clean:])) and torch.all(torch.isnan(l[:, clean:]))


@pytest.mark.parametrize("rows,H,kv,B,longest", [(2, 4, 2, 500, 300), (1, 2, 2, 193, 700), (40, 2, 1, 70, 260)])
def test_forward_of_many_sequences(rows, H, kv, B, longest):
    """More sequences than a block has threads; lengths from nothing on, rows from none on."""
    rng = np.random.default_rng(B)
    lengths = [int(x) for x in rng.integers(0, longest, size=B)]
    n = [int(x) for x in rng.integers(0, rows + 1, size=B)]
    n[-1] = rows
    n_pages = sum(-(-x // 64) for x in lengths) + 1
    c, host = make_cache(n_pages, kv, 64, seed=B)
    check_forward(c, host, make_table(lengths, n_pages), lengths, n, H, causal=True, seed=B, max_rows=rows)


@pytest.mark.parametrize("H,kv,rows", [(300, 1, 3), (40, 1, 1), (33, 1, 9), (64, 2, 1)])
def test_forward_of_wide_groups(H, kv, rows):
    """Query heads of one K/V head that fill no whole number of tiles."""
    lengths = [321, 90]
    c, host = make_cache(9, kv, 64, seed=H)
    check_forward(c, host, make_table(lengths, 9), lengths, [rows, 1], H, causal=True, seed=H)


def test_forward_of_no_rows():
    c, _ = make_cache(2, 1, 64)
    for T in (1, 100):
        out = torch.full((2, T, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        q = torch.randn(2, T, 64, device=DEV).to(torch.bfloat16)
        h3.cache_forward(c, q, i32([0, 0, 0]), i32([5, 0]), i32([[0], [1]]), out=out)
        assert torch.all(out == 7)
    o, _ = h3.cache_forward(c, q[:, :0], i32([0, 0]), i32([5]), i32([[0]]))
    assert o.shape == (2, 0, 64)


@pytest.mark.parametrize("rows,hint", [(1, 1), (150, 150), (150, 1)])
def test_forward_repeats_itself(rows, hint):
    """The same call gives the same bits, also with a hint that is too small."""
    lengths = [3000, 100, 900]
    c, host = make_cache(70, 2, 128, seed=15)
    table = make_table(lengths, 70)
    first = check_forward(c, host, table, lengths, [rows] * 3, 4, seed=15, max_rows=hint)
    for _ in range(3):
        again = check_forward(c, host, table, lengths, [rows] * 3, 4, seed=15, max_rows=hint)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_two_streams_and_two_workspaces():
    """Calls that overlap, each with a workspace of its own."""
    lengths = [5000]
    cs = [make_cache(80, 2, 128, seed=s) for s in (1, 2)]
    table = make_table(lengths, 80)
    qs = [torch.randn(8, n, 128, device=DEV).to(torch.bfloat16) for n in (1, 200)]
    args = [(c, q, i32([0, q.shape[1]]), i32(lengths), i32(table)) for (c, _), q in zip(cs, qs)]
    want = [h3.cache_forward(*a, lse=True) for a in args]
    ws = [h3.cache_workspace(a[0], 8, a[1].shape[1], 1) for a in args]
    streams = [torch.cuda.Stream() for _ in args]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [h3.cache_forward(*a, ws=w, lse=True, stream=s) for a, w, s in zip(args, ws, streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    assert all(h3.check(w) == h3.OK for w in ws)


def test_forward_with_short_waits_ends_and_recovers():
    """Every wait of the tile kernel bounded to one poll.  One poll may itself block for a time that the hardware sets,
    so a wait may still come through: the call ends either complete or with the status word set; then, with the bound
    gone and the word cleared, a call on the same workspace is right."""
    lengths = [2000]
    c, host = make_cache(40, 2, 128, seed=21)
    table = make_table(lengths, 40)
    ws = h3.cache_workspace(c, 2, 300, 1)
    q = torch.randn(2, 300, 128, device=DEV).to(torch.bfloat16)
    args = q, i32([0, 300]), i32(lengths), i32(table)
    want, _ = h3.cache_forward(c, *args)
    for _ in range(20):
        try:
            h3.set_wait_polls(1)
            o, _ = h3.cache_forward(c, *args, ws=ws)
            status = h3.check(ws)
        finally:
            h3.set_wait_polls(0)
        assert status in (h3.OK, h3.ETIMEOUT)
        assert status == h3.ETIMEOUT or torch.equal(o, want)
        assert h3.check(ws) == h3.OK
    check_forward(c, host, table, lengths, [300], 2, seed=21, ws=ws)


@pytest.mark.parametrize("seed", range(6))
def test_forward_of_random_batches(seed):
    rng = np.random.default_rng(100 + seed)
    d, kv, g = int(rng.choice([64, 128])), int(rng.choice([1, 2, 3])), int(rng.choice([1, 2, 3, 5, 8]))
    B = int(rng.integers(1, 9))
    lengths = [int(x) for x in np.exp(rng.uniform(0, np.log(3000), size=B))]
    rows = [int(x) for x in np.exp(rng.uniform(0, np.log(400), size=B))]
    n_pages = sum(-(-x // 64) for x in lengths) + 2
    pen = h3.DEFAULT_PENALTY if seed % 2 else None
    c, host = make_cache(n_pages, kv, d, seed=seed, times=pen is not None)
    check_forward(c, host, make_table(lengths, n_pages, seed=seed), lengths, rows, kv * g, causal=bool(seed % 3), pen=pen,
                  pad=seed, seed=seed, max_rows=max(rows))


def test_forward_over_pages_of_one_guide_time():
    """Pages whose keys share a guide time, pages with two, a page without: the tile kernel's three ways."""
    lengths, rows = [64 * 6 + 10], [200]
    c, host = make_cache(7, 1, 128, seed=33, times=True)
    t = host[4]
    table = make_table(lengths, 7)
    for i, p in enumerate(table[0]):
        t[p] = 0.17 * i
    t[table[0][2], 20:] = 1.7
    t[table[0][4]] = float("nan")
    c.times.copy_(t)
    check_forward(c, host, table, lengths, rows, 2, pen=h3.DEFAULT_PENALTY, seed=33)
