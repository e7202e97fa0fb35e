"""Rows of cross attention and shared-prefix decode do not reach one another:
a NaN, an infinite or a huge query in one head of a group leaves the group's
other heads as they were, on the one-query kernel too."""
import pytest
import torch

import rows_plain as plain
from test_gpu_rows import cross_plain, device_cache, ints, packed, queries, shared_plain

pytestmark = pytest.mark.gpu


def spoil(Q, G, H):
    """Q [B][H * G][d]: in every sequence b and KV head h one head of the group is bad, by turns with a NaN, an infinity,
    a negative infinity, and numbers of 1e30 (finite: its scores are, and it stands alone too). Returns the bad queries,
    and masks [B][H * G] of the rows that must be NaN and of those that must be as without the bad ones."""
    bad = Q.clone()
    nan, good = torch.zeros(Q.shape[:2], dtype=torch.bool), torch.ones(Q.shape[:2], dtype=torch.bool)
    for b in range(Q.shape[0]):
        for h in range(H):
            kind, row = (b + h) % 4, h * G + (3 * b + h) % G
            good[b, row] = False
            nan[b, row] = kind < 3
            if kind == 3:
                bad[b, row] = 1e30 * torch.sign(Q[b, row].float()).to(torch.bfloat16)
            else:
                bad[b, row, (5 * b + h) % Q.shape[2]] = (float("nan"), float("inf"), -float("inf"))[kind]
    return bad, nan, good


@pytest.mark.parametrize("G", [2, 4, 8])
@pytest.mark.parametrize("d,fmt,r", [(128, 0, 8), (64, 1, 16), (128, 0, 0)])
def test_a_bad_head_of_one_query_stays_alone(G, d, fmt, r):
    import bit_kv_cache_centroid_b200 as kv2
    B, H = 8, 2
    pc, P = packed(B, H, d, 64, r, 640, fmt=fmt, seed=80 + G)
    c = device_cache(pc, P)
    lens = [640, 1, 129, 300, 77, 128, 500, 16]
    Q = queries((B, H * G, d), 81 + G)
    bad, nan, good = spoil(Q, G, H)
    want, sigma = cross_plain(pc, P, Q.unsqueeze(1), lens, [1] * B, 0.09)
    got = kv2.kv2_attention_cross(c, ints(lens), bad.unsqueeze(1).cuda(), 0.09).cpu()[:, 0]
    plain.check(got[good], want[:, 0][good], sigma[:, 0][good], torch.float32, "the other heads")
    assert torch.isnan(got[nan]).all()
    assert torch.isfinite(got[~nan]).all()


@pytest.mark.parametrize("G", [1, 4])
def test_a_bad_head_beside_many_own_caches_stays_alone(G):
    """More own caches than SMs: their part by the split decode kernel, the prefix's by the row kernel."""
    import bit_kv_cache_centroid_b200 as kv2
    B, H, d = 80, 2, 128
    pre, P0 = packed(2, H, d, 64, 8, 512, seed=90)
    pc, P = packed(B, H, d, 64, 8, 272, seed=91)
    cp, c = device_cache(pre, P0), device_cache(pc, P)
    plens, lens = [500, 0], [(13 * k) % 260 + 1 for k in range(B)]
    Q = queries((B, H * G, d), 92)
    bad, nan, good = spoil(Q, G, H)
    want, sigma = shared_plain(pre, pc, P0, P, Q, plens, lens, 0.09)
    got = kv2.kv2_attention_shared(cp, ints(plens), c, ints(lens), bad.cuda(), 0.09).cpu()
    plain.check(got[good], want[good], sigma[good], torch.float32, "the other heads")
    assert torch.isnan(got[nan]).all()
    assert torch.isfinite(got[~nan]).all()


@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e10])
def test_tiny_and_large_queries_of_one_head(size):
    """A head of another size than its siblings, down to the smallest numbers: each as the definition has it."""
    import bit_kv_cache_centroid_b200 as kv2
    pc, P = packed(2, 2, 128, 64, 8, 640, seed=97)
    c = device_cache(pc, P)
    Q = queries((2, 8, 128), 98, 0.5)
    Q[:, 1::4] *= size
    if size > 1:
        Q[:, 1::4] = torch.where(torch.arange(128) == 3, Q[:, 1::4], torch.zeros((), dtype=Q.dtype))
    want, sigma = cross_plain(pc, P, Q.unsqueeze(1), [640, 300], [1, 1], 0.09)
    got = kv2.kv2_attention_cross(c, ints([640, 300]), Q.unsqueeze(1).cuda(), 0.09).cpu()
    keep = torch.ones(8, dtype=torch.bool)
    keep[1::4] = size < 1                                  # (beyond fp32's resolution of the scores: finite is all that holds)
    plain.check(got[:, :, keep], want[:, :, keep], sigma[:, :, keep], torch.float32)
    assert torch.isfinite(got).all()
