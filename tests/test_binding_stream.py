"""The handle of the current stream, with and without PyTorch's name for it
alone (no device work)."""
import types

import torch


def test_the_current_stream_without_the_raw_name(monkeypatch):
    import bit_kv_cache_centroid_b200 as kv2
    seen = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=0x1230))
    monkeypatch.setattr(kv2, "_raw_stream", lambda d: seen.append(d) or 0x4560)
    assert kv2._stream().value == 0x4560 and seen == [3]
    monkeypatch.setattr(kv2, "_raw_stream", None)
    assert kv2._stream().value == 0x1230
    assert kv2._stream(types.SimpleNamespace(cuda_stream=0x7890)).value == 0x7890
