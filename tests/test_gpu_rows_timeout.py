"""A wait that runs out in one CTA of the row attention kernel, beside CTAs
that finish: every row is what it would be without, or NaN, and the rows of the
part that was given up are NaN."""
import pytest
import torch

from test_gpu_rows import device_cache, packed, queries

pytestmark = pytest.mark.gpu

LEAD, KEYS, GIVEN_UP = 2, 128, 4      # the kernel's list positions before a unit, keys a tile, the tile that is given up


def parts_of_cta(c, B, Nq, G, H, length):
    """Per unit that CTA c has tiles of: (sequence, KV head, first row, rows, whether a tile at or after the given-up one)."""
    N = 128 if Nq * G <= 128 else 256
    blocks, tiles = -(-Nq * G // N), max(1, -(-length // KEYS))
    units = [(b, h, r) for b in range(B) for h in range(H) for r in range(blocks)]
    T = len(units) * (tiles + LEAD)
    C = min(torch.cuda.get_device_properties(0).multi_processor_count, len(units) * tiles)
    t, out = 0, []
    for at in range(T * c // C, T * (c + 1) // C):
        u, j = divmod(at, tiles + LEAD)
        if j < LEAD:
            continue
        b, h, r = units[u]
        unit = (b, h, r * N, min(N, Nq * G - r * N))
        if not out or out[-1][0] != unit:
            out.append([unit, False])
        out[-1][1] |= t >= GIVEN_UP
        t += 1
    return out


@pytest.mark.parametrize("B,H,G,Nq,length,d", [
    (2, 3, 2, 300, 6000, 128),       # several row blocks of 256, cut units
    (60, 8, 2, 100, 250, 128),       # short units: several a CTA
    (40, 8, 2, 30, 1000, 128),       # one block of 128 rows, both groups
    (3, 4, 4, 11, 20000, 64),
])
def test_one_cta_gives_up(monkeypatch, B, H, G, Nq, length, d):
    import bit_kv_cache_centroid_b200 as kv2
    pc, P = packed(B, H, d, 64, 8, (length + 15) // 16 * 16, seed=31)
    c = device_cache(pc, P)
    Q = queries((B, Nq, H * G, d), 32, 0.5).cuda()
    ws = torch.zeros(kv2.kv2_attention_cross_workspace_size(c, H * G, Nq, length), dtype=torch.uint8, device="cuda")
    call = lambda: kv2.kv2_attention_cross(c, None, Q, 0.09, max_len=length, ws=ws).cpu()
    good = call()
    assert torch.isfinite(good).all() and ws[:4].view(torch.int32).item() == 0
    reached = 0
    for cta in (0, 1, 40, 77, 147):
        lost = parts_of_cta(cta, B, Nq, G, H, length)
        must, may = torch.zeros(B, Nq, H * G, dtype=torch.bool), torch.zeros(B, Nq, H * G, dtype=torch.bool)
        for (b, h, r0, n), nan in lost:
            for r in range(r0, r0 + n):
                may[b, r // G, h * G + r % G] = True
                must[b, r // G, h * G + r % G] |= nan
        reached += int(must.any())
        for _ in range(4):
            monkeypatch.setenv("KV2_FORCE_WAIT_TIMEOUT_CTA", str(cta))
            got = call()
            monkeypatch.delenv("KV2_FORCE_WAIT_TIMEOUT_CTA")
            assert ws[:4].view(torch.int32).item() == int(must.any())
            ws[:4].zero_()
            bad = torch.isnan(got).any(-1)
            assert torch.equal(bad, torch.isnan(got).all(-1))
            assert not (bad & ~may).any(), "rows of other CTAs are NaN"
            assert not (must & ~bad).any(), "rows of the part that was given up are numbers"
            assert torch.equal(got[~bad], good[~bad]), "rows that were finished differ"
            assert torch.equal(call(), good)
    assert reached
