"""The same call many times over: every result is the first one's, bit for
bit, and the first is right. Short units, several a CTA, so that packed tiles
are read while the rows of the unit before them are written."""
import pytest
import torch

import rows_plain as plain
from test_gpu_rows import device_cache, ints, packed, queries, shared_plain

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,H,G,Nq,length,d,r,fmt", [
    (60, 8, 2, 60, 500, 64, 8, 0),
    (40, 8, 2, 30, 1000, 128, 8, 0),
    (40, 8, 2, 30, 1000, 128, 16, 1),
    (64, 8, 4, 32, 400, 128, 8, 0),          # 128 rows
    (60, 8, 4, 40, 300, 128, 8, 0),          # 160 rows: units of 256
    (30, 8, 2, 300, 600, 64, 16, 0),
])
def test_cross_repeats_itself(B, H, G, Nq, length, d, r, fmt):
    import bit_kv_cache_centroid_b200 as kv2
    pc, P = packed(B, H, d, 64, r, (length + 15) // 16 * 16, fmt=fmt, seed=31)
    c = device_cache(pc, P)
    Q = queries((B, Nq, H * G, d), 32, 0.5)
    ws = torch.zeros(kv2.kv2_attention_cross_workspace_size(c, H * G, Nq, length), dtype=torch.uint8, device="cuda")
    out, Qd = torch.empty(Q.shape, device="cuda"), Q.cuda()
    call = lambda: kv2.kv2_attention_cross(c, None, Qd, 0.09, max_len=length, ws=ws, out=out)
    first = call().clone()
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(600):
        differ += (call() != first).any()
    assert differ.item() == 0, f"{differ.item()} of 600 calls differ from the first"
    for b in (0, B // 2, B - 1):
        for h in (0, H - 1):
            q = Q[b, :, h * G:(h + 1) * G].double().reshape(Nq * G, d)
            o, s = plain.attend(q, [(plain.tokens(pc, b, h, length), fmt == 1)], P[h], 0.09)
            plain.check(first[b, :, h * G:(h + 1) * G].cpu().reshape(Nq * G, d), o, s, torch.float32, f"sequence {b}")


@pytest.mark.parametrize("N,S,H,G", [(12, 4, 8, 4), (40, 2, 12, 1)])
def test_shared_repeats_itself(N, S, H, G):
    import bit_kv_cache_centroid_b200 as kv2
    pre, P0 = packed(N, H, 128, 64, 8, 1008, seed=33)
    pc, P = packed(N * S, H, 128, 64, 8, 272, seed=34)
    cp, c = device_cache(pre, P0), device_cache(pc, P)
    plens, lens = [1000 - 31 * k % 700 for k in range(N)], [(37 * k) % 260 for k in range(N * S)]
    Q = queries((N * S, H * G, 128), 35)
    Qd, pl, ln = Q.cuda(), ints(plens), ints(lens)
    ws = torch.zeros(kv2.kv2_attention_shared_workspace_size(cp, c, H * G, 1008, 272), dtype=torch.uint8, device="cuda")
    out = torch.empty(Q.shape, device="cuda")
    call = lambda: kv2.kv2_attention_shared(cp, pl, c, ln, Qd, 0.09, ws=ws, out=out)
    first = call().clone()
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(600):
        differ += (call() != first).any()
    assert differ.item() == 0, f"{differ.item()} of 600 calls differ from the first"
    want, sigma = shared_plain(pre, pc, P0, P, Q, plens, lens, 0.09)
    plain.check(first.cpu(), want, sigma, torch.float32, "shared")
