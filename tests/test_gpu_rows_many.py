"""Batches of many short sequences: more (sequence, KV head) pairs than one
dimension of a grid takes."""
import pytest
import torch

import rows_plain as plain
from test_gpu_rows import device_cache, ints, packed, queries

pytestmark = pytest.mark.gpu


def parts(pc, b, h, n):
    return [(plain.tokens(pc, b, h, n), pc.psac_fmt == 1)]


# 65,536 pairs: one above a grid's y dimension; 65,536 sequences: one above its z dimension too
@pytest.mark.parametrize("B,H", [(8192, 8), (65536, 1)])
def test_one_query_of_many_sequences(B, H):
    import bit_kv_cache_centroid_b200 as kv2
    pc, P = packed(B, H, 64, 16, 8, 16, seed=5)
    c = device_cache(pc, P)
    lens = torch.arange(B, dtype=torch.int32) % 17
    Q = queries((B, 1, 2 * H, 64), 6)
    got = kv2.kv2_attention_cross(c, lens.cuda(), Q.cuda(), 0.125).cpu()
    for b in [0, 1, B // 2, B - 2, B - 1] + list(range(7, B, B // 23)):
        for h in (0, H - 1):
            o, s = plain.attend(Q[b, 0, 2 * h:2 * h + 2].double(), parts(pc, b, h, int(lens[b])), P[h], 0.125)
            plain.check(got[b, 0, 2 * h:2 * h + 2], o, s, torch.float32, f"sequence {b}")


@pytest.mark.parametrize("B,H", [(8192, 8), (65536, 1)])
def test_shared_prefix_of_many_sequences(B, H):
    import bit_kv_cache_centroid_b200 as kv2
    pc, P = packed(B, H, 64, 16, 8, 16, seed=7)
    pre, _ = packed(4, H, 64, 16, 8, 144, seed=8)
    c, cp = device_cache(pc, P), device_cache(pre, P)
    lens = torch.arange(B, dtype=torch.int32) % 17
    plens = [140, 0, 1, 17]
    Q = queries((B, H, 64), 9)
    got = kv2.kv2_attention_shared(cp, ints(plens), c, lens.cuda(), Q.cuda(), 0.125).cpu()
    for b in [0, 1, B // 2, B - 2, B - 1] + list(range(7, B, B // 23)):
        for h in (0, H - 1):
            g = b // (B // 4)
            o, s = plain.attend(Q[b, h:h + 1].double(), parts(pre, g, h, plens[g]) + parts(pc, b, h, int(lens[b])), P[h], 0.125)
            plain.check(got[b, h:h + 1], o, s, torch.float32, f"sequence {b}")


def test_plain_decode_of_many_sequences():
    import bit_kv_cache_centroid_b200 as kv2
    B, H = 8192, 8
    pc, P = packed(B, H, 64, 16, 8, 16, seed=10)
    c = device_cache(pc, P)
    Q = queries((B, H, 64), 11)
    got = kv2.kv2_attention_decode(c, 13, Q.cuda(), 0.125).cpu()
    for b in range(0, B, B // 23):
        o, s = plain.attend(Q[b, H - 1:].double(), parts(pc, b, H - 1, 13), P[H - 1], 0.125)
        plain.check(got[b, H - 1:], o, s, torch.float32, f"sequence {b}")
