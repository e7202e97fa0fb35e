"""Cross attention and decode over a shared prefix against plain 64-bit
attention on the same packed caches."""
import os

import numpy as np
import pytest
import torch

import rows_plain as plain
import workloads as wl

pytestmark = pytest.mark.gpu

DT = {0: torch.float32, 1: torch.bfloat16}


def packed(B, H, d, M, r, cap, group=32, fmt=0, page=0, seed=0, poison=None):
    """A random packed cache; ``poison``: lengths behind which every stream holds
    what no kernel may use (scales, zeros and coefficients NaN and infinite)."""
    s = wl.Spec("t", seed, B=B, H_q=H, H_kv=H, d=d, M=M, C=1, r=r, T=cap, n_new=0, capacity=cap, n_hist=1, Nq=0,
                frame_tokens=1, key_law="gaussian", top_energy=0.7, group=group)
    pc = wl.random_packed_cache(s, psac_fmt=fmt)
    if poison is not None:
        for b, n in enumerate(poison):
            pc.k_sz[b, :, n:] = 0x7E007C00
            pc.v_sz[b, :, n:] = 0x7C007E00
            if fmt == 1:
                pc.psac_scale[b, :, n:] = 0x7E00
            else:
                pc.psac[b, :, n:] = 0xFC00
            pc.cidx[b, :, n:] = 255 if M <= 256 else 65535
    if page:
        pc = wl.to_paged(pc, page, B * (pc.capacity // page) + 2, seed)
    rng = np.random.default_rng(seed + 77)
    P = np.stack([np.linalg.qr(rng.standard_normal((d, max(r, 1))))[0] for _ in range(H)]).astype(np.float32)
    return pc, torch.from_numpy(P[:, :, :r].copy())


def device_cache(pc, P):
    import bit_kv_cache_centroid_b200 as kv2
    c = kv2.Cache(pc.B, pc.H_kv, pc.d, pc.M, pc.r, pc.capacity, torch.from_numpy(pc.centroids.view(np.int16)),
                  psac_fmt=pc.psac_fmt, page_tokens=pc.page if pc.table is not None else 0,
                  num_pages=pc.k_code.shape[0] if pc.table is not None else 0, group=pc.group)
    c.load_packed(pc)
    if pc.r:
        c.P.copy_(P)
    return c


def queries(shape, seed, scale=1.5):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(torch.bfloat16)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cross_plain(pc, P, Q, lens, q_lens, scale):
    B, Nq, Hq, d = Q.shape
    G = Hq // pc.H_kv
    o = torch.zeros(Q.shape, dtype=torch.float64)
    sg = torch.zeros_like(o)
    for b in range(B):
        n = q_lens[b]
        for h in range(pc.H_kv):
            if n == 0:
                continue
            q = Q[b, :n, h * G:(h + 1) * G].double().reshape(n * G, d)
            x, y = plain.attend(q, [(plain.tokens(pc, b, h, lens[b]), pc.psac_fmt == 1)], P[h], scale)
            o[b, :n, h * G:(h + 1) * G] = x.view(n, G, d)
            sg[b, :n, h * G:(h + 1) * G] = y.view(n, G, d)
    return o, sg


def shared_plain(pre, pc, P0, P1, Q, plens, lens, scale):
    """Each cache with its own basis and centres: a score takes the basis of the cache its token is in."""
    B, Hq, d = Q.shape
    G, S = Hq // pc.H_kv, B // pre.B
    o = torch.zeros(Q.shape, dtype=torch.float64)
    sg = torch.zeros_like(o)
    for b in range(B):
        for h in range(pc.H_kv):
            q = Q[b, h * G:(h + 1) * G].double()
            ta, tb = plain.tokens(pre, b // S, h, plens[b // S]), plain.tokens(pc, b, h, lens[b])
            r0, r1 = pre.r, pc.r
            wide = lambda t, lo, hi: (t[0], t[1], torch.nn.functional.pad(t[2], (lo, hi)), t[3])
            x, y = plain.attend(q, [(wide(ta, 0, r1), pre.psac_fmt == 1), (wide(tb, r0, 0), pc.psac_fmt == 1)],
                                torch.cat([P0[h], P1[h]], 1), scale)
            o[b, h * G:(h + 1) * G], sg[b, h * G:(h + 1) * G] = x, y
    return o, sg


# B, H_kv, G, d, M, r, fmt, group, page, Nq, lens, q_lens, out dtype
CROSS = [
    (3, 2, 1, 128, 64, 8, 0, 32, 0, 1, [0, 1, 130], None, 0),                        # decode form, 16 columns
    (2, 2, 4, 128, 64, 8, 0, 32, 128, 7, [128, 127], [7, 3], 0),                      # 28 rows, 32 columns
    (4, 1, 3, 128, 300, 16, 0, 64, 0, 21, [129, 256, 0, 5], [21, 0, 2, 1], 0),        # 63 rows, odd group, u16 ids
    (2, 3, 5, 128, 16, 16, 1, 128, 256, 40, [700, 385], None, 1),                     # 200 rows, two row blocks, int8
    (1, 2, 1, 128, 256, 0, 0, 32, 0, 300, [1111], None, 0),                           # r = 0, three row blocks
    (5, 2, 8, 64, 16, 8, 0, 32, 128, 1, [1, 2, 300, 0, 128], None, 1),                # 64 channels
    (2, 2, 2, 64, 40, 16, 1, 64, 0, 33, [77, 200], [33, 20], 0),                      # 66 rows: two groups, 64 channels
    (3, 2, 2, 64, 40, 0, 0, 64, 0, 12, [640, 1, 131], [0, 0, 12], 0),
    (1, 1, 1, 128, 1, 8, 0, 32, 0, 1, [1], None, 0),                                  # one token, one centre
    (6, 2, 2, 64, 300, 16, 1, 32, 128, 1, [0, 300, 128, 1, 640, 5], [1, 0, 1, 1, 5, -3], 1),   # one query or none
    (3, 1, 8, 128, 16, 0, 0, 128, 0, 1, [200, 129, 4000], [1, 1, 1], 0),
    (3, 2, 3, 128, 16, 8, 0, 64, 256, 1, [200, 0, 1500], [1, 1, 0], 0),               # one query, odd group
]


@pytest.mark.parametrize("i", range(len(CROSS)))
def test_cross(i):
    import bit_kv_cache_centroid_b200 as kv2
    B, H, G, d, M, r, fmt, group, page, Nq, lens, q_lens, dt = CROSS[i]
    unit = page or 16
    cap = (max(max(lens), 1) + unit) // unit * unit
    pc, P = packed(B, H, d, M, r, cap, group, fmt, page, seed=i, poison=lens)
    c = device_cache(pc, P)
    Q = queries((B, Nq, H * G, d), 100 + i, (0.4, 1.5)[i % 2])      # even weights, where every token counts; uneven ones
    out = torch.full(Q.shape, 7.0, dtype=DT[dt], device="cuda")
    ql = [min(max(x, 0), Nq) for x in q_lens or [Nq] * B]
    got = kv2.kv2_attention_cross(c, ints(lens), Q.cuda(), d ** -0.5, dt, q_lens=None if q_lens is None else ints(q_lens),
                                  max_len=max(max(lens), 1), out=out)
    want, sigma = cross_plain(pc, P, Q, lens, ql, d ** -0.5)
    got = got.cpu()
    for b in range(B):
        plain.check(got[b, :ql[b]], want[b, :ql[b]], sigma[b, :ql[b]], DT[dt], f"sequence {b}")
        assert (got[b, ql[b]:] == 7.0).all(), "rows behind the queries were written"


# groups, per, H_kv, G, d, (M, r, fmt, group, page) of prefix and cache, prefix lens, lens, out dtype
SHARED = [
    (1, 3, 2, 4, 128, (64, 8, 0, 32, 0), (64, 8, 0, 32, 0), [300], [1, 0, 129], 0),
    (2, 2, 2, 2, 128, (64, 8, 0, 32, 128), (300, 16, 1, 128, 256), [0, 257], [5, 0, 128, 127], 0),
    (3, 11, 1, 3, 64, (16, 16, 1, 64, 0), (16, 0, 0, 32, 128), [1, 640, 127], [1 + 7 * k for k in range(33)], 1),
    (1, 40, 2, 4, 128, (64, 8, 0, 64, 0), (64, 8, 0, 64, 0), [1500], [3 * k for k in range(40)], 0),
    (2, 1, 2, 1, 64, (8, 8, 0, 32, 0), (8, 8, 0, 32, 0), [0, 40], [0, 0], 0),
    # more own caches than SMs: their part by the split decode kernel
    (3, 31, 2, 2, 128, (64, 8, 0, 32, 0), (64, 8, 1, 32, 128), [200, 0, 513], [(7 * k) % 400 for k in range(93)], 1),
    (1, 160, 1, 8, 64, (16, 16, 0, 32, 0), (300, 8, 0, 64, 0), [300], [(11 * k) % 260 for k in range(160)], 0),
    (2, 90, 1, 3, 64, (16, 0, 0, 32, 0), (16, 0, 0, 32, 0), [64, 300], [(5 * k) % 200 for k in range(180)], 0),
]


@pytest.mark.parametrize("i", range(len(SHARED)))
def test_shared(i):
    import bit_kv_cache_centroid_b200 as kv2
    N, S, H, G, d, fa, fb, plens, lens, dt = SHARED[i]
    caches = []
    for B, f, ls, seed in ((N, fa, plens, 10 + i), (N * S, fb, lens, 30 + i)):
        M, r, fmt, group, page = f
        unit = page or 16
        pc, P = packed(B, H, d, M, r, (max(ls) // unit + 1) * unit, group, fmt, page, seed=seed, poison=ls)
        caches.append((pc, P, device_cache(pc, P)))
    (pre, P0, cp), (pc, P1, c) = caches
    Q = queries((N * S, H * G, d), 200 + i, (0.4, 1.5)[i % 2])
    got = kv2.kv2_attention_shared(cp, ints(plens), c, ints(lens), Q.cuda(), d ** -0.5, dt).cpu()
    want, sigma = shared_plain(pre, pc, P0, P1, Q, plens, lens, d ** -0.5)
    plain.check(got, want, sigma, DT[dt], "shared")


@pytest.mark.parametrize("B,H,G,Nq,r,fmt,dt", [(30, 4, 4, 80, 8, 0, 1), (100, 4, 3, 20, 16, 1, 0), (7, 12, 1, 400, 0, 0, 0)])
def test_many_units_a_cta(B, H, G, Nq, r, fmt, dt):
    """More row blocks than SMs, of several heads each: query rows, fragments of P and output rows change from unit to
    unit in every CTA, and borders fall inside units."""
    import bit_kv_cache_centroid_b200 as kv2
    lens = [(53 * b) % 390 for b in range(B)]
    ql = [(29 * b + 11) % (Nq + 1) for b in range(B)]
    pc, P = packed(B, H, 128, 32, r, 400, fmt=fmt, seed=41, poison=lens)
    c = device_cache(pc, P)
    Q = queries((B, Nq, H * G, 128), 42, 0.8)
    out = torch.full(Q.shape, 7.0, dtype=DT[dt], device="cuda")
    got = kv2.kv2_attention_cross(c, ints(lens), Q.cuda(), 0.09, dt, q_lens=ints(ql), out=out).cpu()
    want, sigma = cross_plain(pc, P, Q, lens, ql, 0.09)
    for b in range(B):
        plain.check(got[b, :ql[b]], want[b, :ql[b]], sigma[b, :ql[b]], DT[dt], f"sequence {b}")
        assert (got[b, ql[b]:] == 7.0).all(), "rows behind the queries were written"


@pytest.mark.parametrize("scale", [-0.09, 0.0])
def test_negative_and_zero_scale(scale):
    import bit_kv_cache_centroid_b200 as kv2
    pc, P = packed(2, 2, 128, 16, 8, 256, seed=44)
    c = device_cache(pc, P)
    lens = [200, 77]
    for Nq in (1, 9, 150):
        Q = queries((2, Nq, 4, 128), 45 + Nq)
        want, sigma = cross_plain(pc, P, Q, lens, [Nq] * 2, scale)
        got = kv2.kv2_attention_cross(c, ints(lens), Q.cuda(), scale).cpu()
        plain.check(got, want, sigma, torch.float32, f"{Nq} queries")
    Q = queries((2, 4, 128), 46)
    want, sigma = shared_plain(pc, pc, P, P, Q, lens, lens, scale)
    plain.check(kv2.kv2_attention_shared(c, ints(lens), c, ints(lens), Q.cuda(), scale).cpu(), want, sigma, torch.float32, "shared")


def test_no_tokens_at_all_gives_zeros():
    import bit_kv_cache_centroid_b200 as kv2
    pc, P = packed(2, 2, 64, 16, 8, 128, seed=47, poison=[0, 0])
    c = device_cache(pc, P)
    for Nq, G in ((1, 1), (1, 3), (5, 2), (200, 2)):
        got = kv2.kv2_attention_cross(c, None, queries((2, Nq, 2 * G, 64), 48).cuda(), 0.125, max_len=0)
        assert (got == 0).all()
    got = kv2.kv2_attention_shared(c, None, c, None, queries((2, 4, 64), 49).cuda(), 0.125, max_prefix_len=0, max_len=0)
    assert (got == 0).all()


def test_two_calls_at_once_with_their_own_workspaces():
    """Two streams, the same caches: each call gives what it gives alone."""
    import bit_kv_cache_centroid_b200 as kv2
    pc, P = packed(3, 4, 128, 64, 8, 2048, seed=51)
    c = device_cache(pc, P)
    Qs = [queries((3, n, 8, 128), n).cuda() for n in (40, 300)]
    alone = [kv2.kv2_attention_cross(c, None, q, 0.09).clone() for q in Qs]
    wss = [torch.zeros(kv2.kv2_attention_cross_workspace_size(c, 8, q.shape[1], 2048), dtype=torch.uint8, device="cuda") for q in Qs]
    outs = [torch.empty(q.shape, device="cuda") for q in Qs]
    streams = [torch.cuda.Stream() for _ in Qs]
    torch.cuda.synchronize()
    for _ in range(5):
        for q, ws, o, st in zip(Qs, wss, outs, streams):
            with torch.cuda.stream(st):
                kv2.kv2_attention_cross(c, None, q, 0.09, out=o, ws=ws)
    torch.cuda.synchronize()
    for a, o in zip(alone, outs):
        assert torch.equal(a, o)


def test_one_workspace_for_calls_in_sequence():
    """Calls of different kinds and sizes, one after another on one workspace and stream: each gives what it gives
    alone, and the rotary append between them too."""
    import bit_kv_cache_centroid_b200 as kv2
    pc, P = packed(80, 2, 128, 16, 8, 272, seed=61)
    pre, P0 = packed(2, 2, 128, 16, 8, 1024, seed=62)
    c, cp = device_cache(pc, P), device_cache(pre, P0)
    Qs, Qw, Qd = (queries(x, 63, 0.8).cuda() for x in ((80, 8, 128), (2, 200, 8, 128), (2, 1, 8, 128)))
    ls = ints([(13 * k) % 250 for k in range(80)])
    rot = kv2.Rotary(torch.randn(512, 128, generator=torch.Generator().manual_seed(1)).cuda())
    K, V = (queries((80, 1, 2, 128), n).cuda() for n in (64, 65))
    place = ints([260] * 80)
    Q = Qs.unsqueeze(1).contiguous()
    calls = [lambda ws: kv2.kv2_attention_cross(cp, None, Qw, 0.09, ws=ws),
             lambda ws: kv2.kv2_rotary_append(c, rot, K, V, place.view(80, 1), place, 4, Q=Q, ws=ws),
             lambda ws: kv2.kv2_attention_shared(cp, None, c, ls, Qs, 0.09, ws=ws),
             lambda ws: kv2.kv2_attention_cross(cp, None, Qd, 0.09, ws=ws),
             lambda ws: kv2.kv2_attention_cross(c, ls, Q, 0.09, ws=ws)]
    size = max(kv2.kv2_attention_cross_workspace_size(cp, 8, 200, 1024), kv2.kv2_rotary_append_workspace_size(c, 1),
               kv2.kv2_attention_shared_workspace_size(cp, c, 8, 1024, 272), kv2.kv2_attention_cross_workspace_size(c, 8, 1, 272))
    alone = []
    for f in calls:
        alone.append(f(None))
        torch.cuda.synchronize()
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    got = [f(ws) for _ in range(4) for f in calls]
    torch.cuda.synchronize()
    assert ws[:4].view(torch.int32).item() == 0
    for i, g in enumerate(got):
        assert torch.equal(g, alone[i % len(calls)]), f"call {i}"


def test_a_call_on_a_given_stream_owns_its_workspace_there():
    """Output and workspace of a call on another stream than the current one come from that stream's memory: what the
    current stream allocates meanwhile does not fall on them."""
    import bit_kv_cache_centroid_b200 as kv2
    pc, P = packed(2, 4, 128, 64, 8, 2048, seed=53)
    c = device_cache(pc, P)
    Q = queries((2, 300, 8, 128), 54).cuda()
    want = kv2.kv2_attention_cross(c, None, Q, 0.09)
    side = torch.cuda.Stream()
    size = kv2.kv2_attention_cross_workspace_size(c, 8, 300, 2048)
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
        got.append(kv2.kv2_attention_cross(c, None, Q, 0.09, stream=side))
        torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g, want)


def test_shared_without_prefix_is_a_ragged_decode():
    """Prefix lengths of zero, and cross attention of one query: both the plain attention over the sequences' own
    caches. (The two take different kernels: one rounds reconstructed keys to fp16, 2^-11 of their size, the other does
    not, so they agree with each other only within the first one's bound.)"""
    import bit_kv_cache_centroid_b200 as kv2
    pc, P = packed(4, 2, 128, 64, 8, 512, seed=3)
    pre, _ = packed(1, 2, 128, 64, 8, 16, seed=4)
    c, cp = device_cache(pc, P), device_cache(pre, P)
    Q = queries((4, 8, 128), 5)
    lens = [512, 1, 200, 0]
    want, sigma = cross_plain(pc, P, Q.unsqueeze(1), lens, [1] * 4, 0.09)
    a = kv2.kv2_attention_shared(cp, ints([0]), c, ints(lens), Q.cuda(), 0.09)
    plain.check(a.cpu(), want[:, 0], sigma[:, 0], torch.float32, "shared")
    b = kv2.kv2_attention_cross(c, ints(lens), Q.unsqueeze(1).cuda(), 0.09)
    plain.check(b.cpu(), want, sigma, torch.float32, "cross")


def test_rising_scores_refresh_the_running_maximum():
    """Every tile holds a score far above all before it: the running maximum moves (and O is rescaled) at each."""
    import bit_kv_cache_centroid_b200 as kv2
    pc, P = packed(1, 1, 128, 64, 0, 1024, seed=9)
    scale = np.repeat(2.0 ** (np.arange(1024) / 170.0), 4).reshape(1, 1, 1024, 4) * 0.2
    pc.k_sz[:] = wl.f16_bits(scale).astype(np.uint32)          # zeros 0, codes grow with the token
    pc.k_code[:] = 0xFFFFFFFF
    c = device_cache(pc, P)
    for nq, seed in ((1, 1), (20, 2), (60, 3), (128, 4)):
        Q = queries((1, nq, 1, 128), seed).abs()
        got = kv2.kv2_attention_cross(c, ints([1024]), Q.cuda(), 128 ** -0.5).cpu()
        want, sigma = cross_plain(pc, P, Q, [1024], [nq], 128 ** -0.5)
        plain.check(got, want, sigma, torch.float32, f"{nq} queries")


def test_a_bad_query_row_stays_alone():
    import bit_kv_cache_centroid_b200 as kv2
    pc, P = packed(1, 1, 128, 64, 8, 256, seed=12)
    c = device_cache(pc, P)
    Q = queries((1, 70, 2, 128), 6)
    ok = kv2.kv2_attention_cross(c, None, Q.cuda(), 0.09).cpu()
    bad = Q.clone()
    bad[0, 3, 1, 5] = float("nan")
    bad[0, 40, 0, 7] = float("inf")
    bad[0, 41, 0] = 1e30                                   # finite and huge: one token takes all the weight
    got = kv2.kv2_attention_cross(c, None, bad.cuda(), 0.09).cpu()
    assert torch.isnan(got[0, 3, 1]).all() and torch.isnan(got[0, 40, 0]).all()
    keep = torch.ones(70, 2, dtype=torch.bool)
    keep[3, 1] = keep[40, 0] = keep[41, 0] = False
    assert torch.equal(got[0][keep], ok[0][keep])
    assert torch.isfinite(got[0, 41, 0]).all()


def test_captured_call_replays_with_other_lengths_on_another_stream():
    import bit_kv_cache_centroid_b200 as kv2
    pc, P = packed(3, 2, 128, 64, 8, 640, seed=15)
    pre, P0 = packed(1, 2, 128, 64, 8, 1024, seed=16)
    c, cp = device_cache(pc, P), device_cache(pre, P0)
    Q = queries((3, 8, 128), 8)
    Qd, lens, plens = Q.cuda(), ints([640, 3, 0]), ints([1000])
    out = torch.zeros(3, 8, 128, device="cuda")
    ws = torch.zeros(kv2.kv2_attention_shared_workspace_size(cp, c, 8, 1024, 640), dtype=torch.uint8, device="cuda")
    run = lambda: kv2.kv2_attention_shared(cp, plens, c, lens, Qd, 0.09, out=out, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            run()
    torch.cuda.synchronize()
    for ls, pl in (([640, 3, 0], [1000]), ([1, 639, 200], [0]), ([0, 0, 5], [129])):
        lens.copy_(ints(ls))
        plens.copy_(ints(pl))
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.current_stream())
            g.replay()
        torch.cuda.synchronize()
        want, sigma = shared_plain(pre, pc, P0, P, Q, pl, ls, 0.09)
        plain.check(out, want, sigma, torch.float32, f"lens {ls}")
        first = out.clone()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, out), "two replays differ"


def test_lengths_beyond_the_bounds_are_taken_into_them():
    import bit_kv_cache_centroid_b200 as kv2
    pc, P = packed(3, 1, 64, 16, 8, 256, seed=18)
    c = device_cache(pc, P)
    Q = queries((3, 5, 2, 64), 9).cuda()
    a = kv2.kv2_attention_cross(c, ints([-7, 1 << 30, 60]), Q, 0.125, q_lens=ints([9, 5, -1]), max_len=200)
    b = kv2.kv2_attention_cross(c, ints([0, 200, 60]), Q, 0.125, q_lens=ints([5, 5, 0]), max_len=200)
    assert torch.equal(a, b)


def test_long_prefix_agrees_with_the_split_decode():
    """30,011 shared tokens: against kv2_attention_decode, whose own error is far below, on each sequence's whole cache."""
    import bit_kv_cache_centroid_b200 as kv2
    T, S = 30011, 5
    pre, P = packed(1, 2, 128, 64, 8, 30016, seed=21)
    one, _ = packed(1, 2, 128, 64, 8, 16, seed=22)
    cp, c1 = device_cache(pre, P), device_cache(one, P)
    c = kv2.Cache(S, 2, 128, 64, 8, 16, c1.centroids)
    c.set_fit(P, c1.w, c1.Wg)
    Q = queries((S, 8, 128), 11).cuda()
    got = kv2.kv2_attention_shared(cp, ints([T]), c, ints([0] * S), Q, 128 ** -0.5)
    want = torch.stack([kv2.kv2_attention_decode(cp, T, Q[b:b + 1], 128 ** -0.5)[0] for b in range(S)])
    # equal weights over many tokens: independent roundings of keys (score error about 4e-4), values and weights
    # (2^-11 / sqrt 3 each) on outputs of the size of |v| / sqrt T: 3 x 6e-4 relative in the 2-norm
    rel = (got - want).norm() / want.norm()
    assert rel <= 1.8e-3, rel


def test_wait_timeout_is_reported(monkeypatch):
    import bit_kv_cache_centroid_b200 as kv2
    pc, P = packed(1, 1, 128, 16, 8, 256, seed=24)
    c = device_cache(pc, P)
    Q = queries((1, 3, 1, 128), 12).cuda()
    ws = torch.zeros(kv2.kv2_attention_cross_workspace_size(c, 1, 3, 256), dtype=torch.uint8, device="cuda")
    good = kv2.kv2_attention_cross(c, None, Q, 0.09, ws=ws).clone()
    assert ws[:4].view(torch.int32).item() == 0
    monkeypatch.setenv("KV2_FORCE_WAIT_TIMEOUT", "1")
    bad = kv2.kv2_attention_cross(c, None, Q, 0.09, ws=ws)
    torch.cuda.synchronize()
    assert ws[:4].view(torch.int32).item() == 1 and torch.isnan(bad).all()
    monkeypatch.delenv("KV2_FORCE_WAIT_TIMEOUT")
    again = kv2.kv2_attention_cross(c, None, Q, 0.09, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(again, good)
    assert ws[:4].view(torch.int32).item() == 1                # sticky until the caller clears it
