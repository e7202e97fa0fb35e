"""A query that holds a NaN gives NaN in its own output rows of the decode
calls, and the group's other heads are numbers."""
import pytest
import torch

from test_gpu_rows import device_cache, packed, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 1000, 20000])
def test_a_nan_query_gives_nan(T):
    import bit_kv_cache_centroid_b200 as kv2
    pc, P = packed(1, 2, 128, 64, 8, (T + 15) // 16 * 16, seed=95)
    c = device_cache(pc, P)
    Q = queries((1, 8, 128), 96)
    Q[0, 2, 7] = float("nan")
    bad = torch.arange(8) == 2
    for got in (kv2.kv2_attention_decode(c, T, Q.cuda(), 0.09).cpu()[0],
                kv2.kv2_attention_cross(c, None, Q.unsqueeze(1).cuda(), 0.09, max_len=T).cpu()[0, 0]):
        assert torch.isnan(got[bad]).all() and torch.isfinite(got[~bad]).all()
