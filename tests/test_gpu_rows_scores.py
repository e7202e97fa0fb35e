"""Scores far beyond what a softmax meets: they choose the token that the
definition chooses, and beyond fp32's range the row is NaN, not a plain mean."""
import pytest
import torch

import rows_plain as plain
from test_gpu_rows import device_cache, packed, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [1e4, 1e6, 1e9, 1e20, 1e30])
@pytest.mark.parametrize("Nq", [40, 200])
def test_huge_scores_choose_the_largest(size, Nq):
    import bit_kv_cache_centroid_b200 as kv2
    pc, P = packed(1, 1, 128, 64, 8, 512, seed=71)
    c = device_cache(pc, P)
    Q = (queries((1, Nq, 1, 128), 72).float() * size).to(torch.bfloat16)
    got = kv2.kv2_attention_cross(c, None, Q.cuda(), 0.09).cpu()[0, :, 0].double()
    zmu, k, a, v = plain.tokens(pc, 0, 0, 512)
    q = Q[0, :, 0].double()
    s = 0.09 * (q @ k.T + (q @ P[0].double()) @ a.T)
    top = s.topk(2, -1)
    # two tokens are told apart where their scores differ by more than the keys' and coefficients' roundings: each of the
    # 2 x 136 products by 2^-11 of itself in each of two roundings, summed as magnitudes
    mags = 0.09 * (q.abs() @ (k.abs() + zmu.abs()).T + (q @ P[0].double()).abs() @ a.abs().T) * 2.0 ** -10
    clear = top.values[:, 0] - top.values[:, 1] > 2 * mags.amax(-1) + 64
    assert torch.isfinite(got).all() and clear.any()
    want = v[top.indices[clear, 0]]
    # two roundings to fp16, half a step of 2^-11 each: the value's, and that of its weight p in P . V, which the sum of
    # weights that divides it takes unrounded: (1 + 2^-11)^2 - 1 < 2.01 2^-11. All other weights are below 512 2^-64;
    # fp32 sums and the division are far below.
    assert ((got[clear] - want).abs() <= want.abs() * 2.0 ** -11 * 2.02 + 2.0 ** -24).all()


@pytest.mark.parametrize("Nq", [3, 40, 200])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_beyond_fp32_are_nan(Nq, sign):
    import bit_kv_cache_centroid_b200 as kv2
    pc, P = packed(1, 1, 128, 64, 0, 300, seed=73)
    pc.k_sz[:] = 0x51003800                                        # scales of 0.5, zeros of 40: every key positive
    c = device_cache(pc, P)
    Q = torch.full((1, Nq, 1, 128), sign * 1e38, dtype=torch.bfloat16)
    Q[0, 1] = 0.01                                                  # beside a row of ordinary scores
    got = kv2.kv2_attention_cross(c, None, Q.cuda(), 1e5, max_len=300).cpu()[0, :, 0]
    others = torch.arange(Nq) != 1
    assert torch.isnan(got[others]).all() and torch.isfinite(got[1]).all()
