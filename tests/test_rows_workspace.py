"""The binding's check of a workspace that the caller passes: on the cache's
device, contiguous (no device work)."""
import numpy as np
import pytest
import torch


@pytest.mark.parametrize("ws", [torch.empty(1 << 24, dtype=torch.uint8, device="meta"),
                                torch.zeros(1, dtype=torch.uint8).expand(1 << 24),
                                torch.zeros(1 << 20, 16, dtype=torch.uint8)[:, :8]], ids=["device", "expanded", "strided"])
def test_workspaces_elsewhere_or_in_pieces_are_refused(ws):
    import bit_kv_cache_centroid_b200 as kv2
    c = kv2.Cache(2, 2, 64, 16, 8, 256, np.zeros((2, 16, 64), np.int16), device="cpu")
    Q = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16)
    K, pos, start = Q[:, :, :2].contiguous(), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    rot = kv2.Rotary(torch.zeros(10, 64))
    for call in (lambda: kv2.kv2_attention_cross(c, None, Q, 1.0, ws=ws),
                 lambda: kv2.kv2_attention_shared(c, None, c, None, Q[:, 0].contiguous(), 1.0, ws=ws),
                 lambda: kv2.kv2_rotary_append(c, rot, K, K, pos, start, 4, ws=ws)):
        with pytest.raises(ValueError, match="ws"):
            call()
