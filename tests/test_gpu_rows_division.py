"""Row attention with tens of thousands of query heads a KV head."""
import pytest
import torch

import rows_plain as plain
from test_gpu_rows import device_cache, ints, packed, queries

pytestmark = pytest.mark.gpu


def parts(pc, b, h, n):
    return [(plain.tokens(pc, b, h, n), pc.psac_fmt == 1)]


@pytest.mark.parametrize("B,Nq", [(2, 0), (1, 2)])
def test_a_group_of_many_query_heads(B, Nq):
    """65,535 query heads a KV head: the rows of one unit list pass 2^32 / 65,535. Two sequences behind one prefix (Nq = 0),
    and one sequence of two queries."""
    import bit_kv_cache_centroid_b200 as kv2
    H, G, d = 2, 65535, 64
    pc, P = packed(B, H, d, 16, 8, 32, seed=12)
    pre, _ = packed(1, H, d, 16, 8, 48, seed=13)
    c, cp = device_cache(pc, P), device_cache(pre, P)
    Q = queries((2, H * G, d), 14)                                   # (sequence or query, head)
    if Nq:
        out = kv2.kv2_attention_cross(c, ints([30]), Q.unsqueeze(0).cuda(), 0.125)[0].cpu()
    else:
        out = kv2.kv2_attention_shared(cp, ints([41]), c, ints([30, 7]), Q.cuda(), 0.125).cpu()
    for i in range(2):
        for h in range(H):
            own = parts(pc, 0, h, 30) if Nq else parts(pre, 0, h, 41) + parts(pc, i, h, (30, 7)[i])
            o, s = plain.attend(Q[i, h * G:(h + 1) * G].double(), own, P[h], 0.125)
            plain.check(out[i, h * G:(h + 1) * G], o, s, torch.float32, f"{i}, head {h}")
