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


def err(ws):
    return ws[:4].view(torch.int32).item()


@pytest.mark.parametrize("Nq", [1, 20, 300])
def test_a_lost_piece_is_not_outweighed(monkeypatch, Nq):
    """One unit in pieces over all CTAs, scores of some hundred: the piece that was given up makes its rows NaN, however
    large the other pieces' maxima."""
    import bit_kv_cache_centroid_b200 as kv2
    length = 128 * 1000
    pc, P = packed(1, 1, 128, 64, 8, length, seed=35)
    c = device_cache(pc, P)
    G = 3 if Nq == 1 else 1                                        # (three heads: the row kernel)
    Q = queries((1, Nq, G, 128), 36, 30.0).cuda()
    ws = torch.zeros(kv2.kv2_attention_cross_workspace_size(c, G, Nq, length), dtype=torch.uint8, device="cuda")
    assert torch.isfinite(kv2.kv2_attention_cross(c, None, Q, 0.09, ws=ws)).all() and err(ws) == 0
    for cta in (0, 70, 147):
        if not any(nan for _, nan in parts_of_cta(cta, 1, Nq, G, 1, length)):
            continue
        monkeypatch.setenv("KV2_FORCE_WAIT_TIMEOUT_CTA", str(cta))
        got = kv2.kv2_attention_cross(c, None, Q, 0.09, ws=ws)
        monkeypatch.delenv("KV2_FORCE_WAIT_TIMEOUT_CTA")
        assert err(ws) == 1
        ws[:4].zero_()
        lost = {r for (_, _, r0, n), nan in parts_of_cta(cta, 1, Nq, G, 1, length) if nan for r in range(r0, r0 + n)}
        for r in lost:
            assert torch.isnan(got[0, r // G, r % G]).all(), (cta, r)


def test_a_lost_split_of_an_own_cache_is_not_outweighed(monkeypatch):
    """More own caches than SMs, one CTA of the split decode kernel gives up: its pair's rows are NaN beside a prefix of
    far larger scores, all other rows as they are without."""
    import bit_kv_cache_centroid_b200 as kv2
    B, H, G, d = 100, 2, 2, 128
    pre, P0 = packed(1, H, d, 64, 8, 128, seed=37)
    pc, P = packed(B, H, d, 64, 8, 400, seed=38)
    pre.k_sz[:] = pre.k_sz & 0xFFFF0000 | 0x5640                   # scales of 100: scores far above the own caches'
    cp, c = device_cache(pre, P0), device_cache(pc, P)
    Q = queries((B, H * G, d), 39, 8.0).cuda()
    ws = torch.zeros(kv2.kv2_attention_shared_workspace_size(cp, c, H * G, 128, 400), dtype=torch.uint8, device="cuda")
    call = lambda: kv2.kv2_attention_shared(cp, None, c, None, Q, 0.09, ws=ws)
    good = call()
    assert torch.isfinite(good).all() and err(ws) == 0
    for cta in (0, 61, 199):
        monkeypatch.setenv("KV2_FORCE_WAIT_TIMEOUT_CTA", str(cta))
        got = call()
        monkeypatch.delenv("KV2_FORCE_WAIT_TIMEOUT_CTA")
        assert err(ws) == 1
        ws[:4].zero_()
        bad = torch.isnan(got).all(-1)
        assert torch.equal(bad, torch.isnan(got).any(-1))
        hit = bad.nonzero()
        assert len(hit) == G and len({(b, h // G) for b, h in hit.tolist()}) == 1, hit
        assert torch.equal(got[~bad], good[~bad])


def test_a_lost_split_of_one_query(monkeypatch):
    import bit_kv_cache_centroid_b200 as kv2
    pc, P = packed(2, 2, 128, 64, 8, 20000, seed=40)
    c = device_cache(pc, P)
    Q = queries((2, 1, 8, 128), 41, 30.0).cuda()
    ws = torch.zeros(kv2.kv2_attention_cross_workspace_size(c, 8, 1, 20000), dtype=torch.uint8, device="cuda")
    good = kv2.kv2_attention_cross(c, None, Q, 0.09, ws=ws)
    assert torch.isfinite(good).all() and err(ws) == 0
    monkeypatch.setenv("KV2_FORCE_WAIT_TIMEOUT_CTA", "1")
    got = kv2.kv2_attention_cross(c, None, Q, 0.09, ws=ws)
    monkeypatch.delenv("KV2_FORCE_WAIT_TIMEOUT_CTA")
    assert err(ws) == 1 and torch.isnan(got[0, 0, :4]).all()
    assert torch.equal(got[0, 0, 4:], good[0, 0, 4:]) and torch.equal(got[1], good[1])
