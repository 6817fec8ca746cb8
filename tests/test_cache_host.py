"""What the cache calls refuse, before any device work: through the C ABI with addresses that are never read, and
through the Python binding with tensors of the wrong kind."""
import ctypes

import pytest
import torch

import biased_attention_video_b200 as h3

FAKE = 1 << 40


def cache(**more):
    f = dict(n_pages=8, H=2, d=128, block=64, k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, times=None)
    f.update(more)
    return h3._CacheStruct(**f)


def batch(**more):
    f = dict(B=3, T=10, max_pages=4, row_start=FAKE, length=FAKE, page_table=FAKE)
    f.update(more)
    return h3._BatchStruct(**f)


def append(c=None, b=None, k=FAKE, ks=(1280, 128), v=FAKE, vs=(1280, 128), rope=None, times=None, ws=FAKE, n=256):
    return h3.lib().h3attn_cache_append(c or cache(), b or batch(), k, *ks, v, *vs, rope, times, ws, n, None)


def read(c=None, b=None, k=FAKE, v=FAKE, ws=FAKE, n=256):
    return h3.lib().h3attn_cache_read(c or cache(), b or batch(), k, v, ws, n, None)


def forward(c=None, b=None, H=4, max_rows=0, q=FAKE, qs=(1280, 128), pen=None, q_times=None, o=FAKE, lse=None, ws=FAKE,
            n=1 << 40):
    return h3.lib().h3attn_cache_forward(c or cache(), b or batch(), H, max_rows, q, *qs, 0, pen, q_times, o, lse, ws,
                                         n, None)


BAD_CACHE = [(dict(n_pages=0), h3.EINVAL), (dict(H=0), h3.EINVAL), (dict(d=96), h3.EUNSUPPORTED),
             (dict(block=128), h3.EUNSUPPORTED), (dict(k=None), h3.EINVAL), (dict(v_scale=None), h3.EINVAL),
             (dict(k=FAKE + 8), h3.EALIGN), (dict(k_scale=FAKE + 2), h3.EALIGN), (dict(times=FAKE + 4), h3.EALIGN)]
BAD_BATCH = [(dict(B=0), h3.EINVAL), (dict(T=-1), h3.EINVAL), (dict(max_pages=0), h3.EINVAL),
             (dict(row_start=None), h3.EINVAL), (dict(page_table=None), h3.EINVAL), (dict(length=FAKE + 2), h3.EALIGN),
             (dict(T=(1 << 30) + 1), h3.EUNSUPPORTED)]


@pytest.mark.parametrize("call", [append, read, forward])
def test_cache_and_batch_are_checked_by_every_call(call):
    for bad, code in BAD_CACHE:
        assert call(c=cache(**bad)) == code, bad
    for bad, code in BAD_BATCH:
        assert call(b=batch(**bad)) == code, bad
    assert call(ws=None) == h3.EWORKSPACE
    assert call(n=255) == h3.EWORKSPACE
    assert call(ws=FAKE + 8) == h3.EALIGN
    assert call(b=batch(T=0)) == h3.OK  # nothing to do, nothing launched


def test_append_refusals():
    assert append(k=None) == h3.EINVAL and append(v=None) == h3.EINVAL
    assert append(k=FAKE + 2) == h3.EALIGN and append(vs=(1280, 132)) == h3.EALIGN
    assert append(ks=(-1280, 128)) == h3.EINVAL
    assert append(times=FAKE) == h3.EINVAL  # the cache holds no times
    assert append(c=cache(times=FAKE), times=FAKE + 2) == h3.EALIGN
    ok = dict(cos=FAKE, sin=FAKE, index=None, n_pos=8, dim=128, interleaved=0)
    for bad, code in [(dict(cos=None), h3.EINVAL), (dict(n_pos=0), h3.EINVAL), (dict(dim=24), h3.EINVAL),
                      (dict(dim=144), h3.EINVAL), (dict(dim=0), h3.EINVAL), (dict(sin=FAKE + 4), h3.EALIGN),
                      (dict(index=FAKE + 1), h3.EALIGN)]:
        assert append(rope=h3._RopeStruct(**{**ok, **bad})) == code, bad


def test_read_refusals():
    assert read(k=None, v=None) == h3.EINVAL
    assert read(k=FAKE + 2) == h3.EALIGN and read(v=FAKE + 8) == h3.EALIGN


def test_forward_refusals():
    assert forward(H=3) == h3.EINVAL and forward(H=0) == h3.EINVAL and forward(max_rows=-1) == h3.EINVAL
    assert forward(q=None) == h3.EINVAL and forward(o=None) == h3.EINVAL
    assert forward(q=FAKE + 2) == h3.EALIGN and forward(qs=(1284, 128)) == h3.EALIGN
    assert forward(o=FAKE + 8) == h3.EALIGN and forward(lse=FAKE + 2) == h3.EALIGN
    need = h3.lib().h3attn_cache_workspace_bytes(cache(), 4, 10, 3)
    assert need >= 256 and forward(n=need - 1) == h3.EWORKSPACE
    pen = h3.Penalty(*h3.DEFAULT_PENALTY)
    assert forward(pen=pen) == h3.EINVAL and forward(pen=pen, q_times=FAKE) == h3.EINVAL  # no times
    timed = cache(times=FAKE)
    assert forward(c=timed, pen=pen, q_times=FAKE + 2) == h3.EALIGN
    for bad in ((2.0, 0.2, 0.0, 6.0), (float("nan"), 0.2, 0.25, 6.0), (2.0, -1.0, 0.25, 6.0),
                (2.0, 0.2, float("inf"), 6.0)):
        assert forward(c=timed, pen=h3.Penalty(*bad), q_times=FAKE) == h3.EINVAL, bad


def test_workspace_bytes_of_bad_sizes():
    L = h3.lib()
    assert L.h3attn_cache_workspace_bytes(cache(), 3, 10, 1) == 0   # heads no multiple
    assert L.h3attn_cache_workspace_bytes(cache(d=80), 4, 10, 1) == 0
    assert L.h3attn_cache_workspace_bytes(cache(), 4, -1, 1) == 0
    assert L.h3attn_cache_workspace_bytes(cache(), 4, 10, 0) == 0
    assert L.h3attn_cache_workspace_bytes(None, 4, 10, 1) == 0


def test_binding_refuses_wrong_tensors():
    k = torch.zeros(4, 2, 64, 128, dtype=torch.int8)
    s = torch.zeros(4, 2)
    with pytest.raises(ValueError, match="k must be contiguous CUDA int8"):
        h3.Cache(k, k, s, s)
    with pytest.raises(ValueError, match="cos"):
        h3.Rope(torch.zeros(4, 32, dtype=torch.float64), torch.zeros(4, 32))
    with pytest.raises(ValueError, match="sin"):
        h3.Rope(torch.zeros(4, 32), torch.zeros(4, 16))
    with pytest.raises(ValueError, match="index"):
        h3.Rope(torch.zeros(4, 32), torch.zeros(4, 32), index=torch.zeros(3))


def test_structs_match_the_header():
    """Sizes of the C structs as a C compiler lays them out (LP64)."""
    assert ctypes.sizeof(h3._CacheStruct) == 56
    assert ctypes.sizeof(h3._BatchStruct) == 40
    assert ctypes.sizeof(h3._RopeStruct) == 40
