"""More of what the cache calls refuse before any device work: batches too long to search, workspaces and streams of
other devices."""
import types

import pytest
import torch

import biased_attention_video_b200 as h3
from test_cache_host import append, batch, forward, read


@pytest.mark.parametrize("call", [append, read, forward])
def test_more_sequences_than_a_call_searches(call):
    assert call(b=batch(B=(1 << 16) + 1)) == h3.EUNSUPPORTED
    assert call(b=batch(B=1 << 16, T=0)) == h3.OK


def test_binding_refuses_workspaces_and_streams_of_other_devices():
    """The kernels would take a foreign address, or run on another device's stream."""
    ws = torch.zeros(256, dtype=torch.uint8)
    for dev in (0, 1):
        with pytest.raises(ValueError, match=f"ws must be contiguous on cuda:{dev}, not on cpu"):
            h3._space(ws, dev)
    with pytest.raises(ValueError, match="ws must be contiguous"):
        h3._space(ws[:1].expand(1 << 20), ws.get_device())
    assert h3._space(ws, ws.get_device()) is ws
    with pytest.raises(ValueError, match="stream must be one of cuda:0, not of cuda:1"):
        h3._on(0, types.SimpleNamespace(device_index=1))
