"""Rotary append: codes, ids, scales and rotated queries bit for bit against
the oracle's quantizer on keys turned on the host; and a serving loop of
rotary appends with shared-prefix and cross attention."""
import numpy as np
import pytest
import torch

import rows_plain as plain
import workloads as wl
from helpers import f16_ulp_diff

pytestmark = pytest.mark.gpu


def table(rows, rot, seed):
    a = np.random.default_rng(seed).uniform(-300, 300, (rows, rot // 2))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def turn(x_bits, cs, inter):
    """bf16 bits [n, heads, d] with rows cs [n, rot]: fp32, every product and sum rounded, then bf16."""
    x = wl.bf16_values(x_bits)
    rot, half = cs.shape[1], cs.shape[1] // 2
    c, s = cs[:, None, :half], cs[:, None, half:]
    ia, ib = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if inter else (np.arange(half), np.arange(half, rot))
    a, b = x[..., ia], x[..., ib]
    y = x.copy()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return wl.bf16_bits(y)


class Setup:
    """A cache with random contents, and its host copy with the oracle's result."""

    def __init__(self, orc, B, n, H, G, d, M, C, r, fmt=0, group=32, page=0, rot=None, inter=False, cap=None, start=None,
                 count=None, seed=0):
        import bit_kv_cache_centroid_b200 as kv2
        rng = np.random.default_rng(seed)
        unit = page or 16
        self.cap = cap or (max(start or [0]) + n + unit) // unit * unit
        self.B, self.n, self.H, self.Hq, self.d, self.M, self.C, self.r = B, n, H, H * G, d, M, C, r
        self.fmt, self.group, self.inter, self.rot = fmt, group, inter, rot or d
        bf = lambda *s: wl.bf16_bits(rng.standard_normal(s).astype(np.float32))
        self.K, self.V, self.Q = bf(B, n, H, d), bf(B, n, H, d), bf(B, n, self.Hq, d)
        self.cent = wl.f16_bits(rng.standard_normal((H, M, d)).astype(np.float32))
        self.fit = orc.fit(bf(64, self.Hq, d), H, r, group)
        self.rows = 977
        self.cs = table(self.rows, self.rot, seed)
        self.pos = rng.integers(0, self.rows, (B, n)).astype(np.int32)
        self.start = np.asarray(start if start is not None else [0] * B, np.int32)
        self.count = None if count is None else np.asarray(count, np.int32)
        s = wl.Spec("t", seed, B=B, H_q=H, H_kv=H, d=d, M=M, C=C, r=r, T=self.cap, n_new=0, capacity=self.cap, n_hist=1, Nq=0,
                    frame_tokens=1, key_law="gaussian", top_energy=0.7, group=group)
        self.before = wl.random_packed_cache(s, centroids=self.cent, psac_fmt=fmt)
        if page:
            self.before = wl.to_paged(self.before, page, B * (self.cap // page) + 2, seed)
        self.page = page
        self.cache = kv2.Cache(B, H, d, M, r, self.cap, torch.from_numpy(self.cent.view(np.int16)), psac_fmt=fmt,
                               page_tokens=page, num_pages=self.before.k_code.shape[0] if page else 0, group=group)
        self.cache.load_packed(self.before)
        self.cache.set_fit(torch.from_numpy(self.fit.P), torch.from_numpy(self.fit.w), torch.from_numpy(self.fit.Wg))
        self.rotary = kv2.Rotary(torch.from_numpy(self.cs).cuda(), interleaved=inter)

    def dev(self, x):
        return torch.from_numpy(np.ascontiguousarray(x)).cuda()

    def call(self, **kw):
        import bit_kv_cache_centroid_b200 as kv2
        a = dict(kw)
        for name, x in (("K", self.K.view(np.int16)), ("V", self.V.view(np.int16)), ("Q", self.Q.view(np.int16)),
                        ("positions", self.pos), ("start", self.start), ("count", self.count)):
            if name not in a:
                a[name] = None if x is None else self.dev(x)
        return kv2.kv2_rotary_append(self.cache, self.rotary, a.pop("K"), a.pop("V"), a.pop("positions"), a.pop("start"),
                                     self.C, **a)

    def expect(self, orc, skip=()):
        """The streams after the call: the oracle's rows at their places, every other byte as before."""
        out = {k: getattr(self.before, k).copy() for k in ("k_code", "v_code", "k_sz", "v_sz", "cidx", "psac")}
        if self.fmt:
            out["psac_scale"] = self.before.psac_scale.copy()
        counts = [self.n] * self.B if self.count is None else [min(max(int(c), 0), self.n) for c in self.count]
        self.counts = counts
        for b, m in enumerate(counts):
            if m == 0:
                continue
            k = turn(self.K[b, :m], self.cs[self.pos[b, :m] % self.rows], self.inter)
            pc = wl.PackedCache.empty(1, self.H, self.d, self.M, self.r, m, self.cent, self.fmt, self.group)
            orc.quantize(pc, k[None], self.V[b:b + 1, :m], 0, self.C, self.fit.P, self.fit.w, self.fit.Wg)
            for t in range(m):
                if (b, t) in skip:
                    continue
                slot = int(self.start[b]) + t
                lead, at = (b, slot) if not self.page else (int(self.before.table[b, slot // self.page]), slot % self.page)
                for name in out:
                    out[name][lead, :, at] = getattr(pc, name)[0, :, t]
        return out

    def compare(self, want):
        got = self.cache.to_host()
        for name in ("k_code", "v_code", "k_sz", "v_sz", "cidx"):
            assert np.array_equal(got[name], want[name]), name
        if self.r and self.fmt == 0:
            assert f16_ulp_diff(got["psac"], want["psac"][..., :self.r]).max() <= 1
        elif self.r:
            # the sums' order may move a coefficient across a rounding border: one code, one step of the scale
            assert f16_ulp_diff(got["psac_scale"], want["psac_scale"]).max() <= 1
            assert np.abs(got["psac"].astype(int) - want["psac"].astype(int)).max() <= 1

    def compare_queries(self, out, fill=0):
        got = out.cpu().numpy().view(np.uint16)
        for b, m in enumerate(self.counts):
            if m:
                assert np.array_equal(got[b, :m], turn(self.Q[b, :m], self.cs[self.pos[b, :m]], self.inter)), b
            assert (got[b, m:] == fill).all(), "queries behind the count were written"


CASES = [
    # one token per sequence (one key per warp), its own place each
    dict(B=5, n=1, H=2, G=4, d=128, M=64, C=4, r=8, start=[0, 17, 255, 128, 3], page=128),
    dict(B=3, n=1, H=2, G=1, d=64, M=300, C=3, r=16, start=[5, 0, 9], count=[1, 0, 1], inter=True, rot=32),
    # ragged prompts (several keys per warp), counts of 0, 1 and out of range
    dict(B=4, n=45, H=2, G=2, d=128, M=64, C=4, r=8, start=[3, 130, 0, 100], count=[45, 0, 1, 99], page=128),
    dict(B=3, n=67, H=3, G=1, d=64, M=16, C=16, r=0, start=[0, 7, 1], count=[-4, 66, 31], group=64, rot=50),
    dict(B=1, n=200, H=1, G=3, d=128, M=256, C=8, r=16, fmt=1, group=128, rot=128, inter=True, start=[56]),
    dict(B=2, n=40, H=2, G=2, d=128, M=100, C=1, r=8, fmt=1, group=64, rot=96, inter=True, start=[0, 5], count=[40, 39], page=256),
    dict(B=2, n=3, H=1, G=1, d=64, M=1, C=1, r=8, rot=2, start=[0, 2]),
    dict(B=9, n=8, H=1, G=2, d=128, M=40, C=5, r=8, rot=64, start=[8 * i for i in range(9)], count=[i % 9 for i in range(9)]),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_rotary_append(orc, i):
    s = Setup(orc, seed=i, **CASES[i])
    q_out = torch.full((s.B, s.n, s.Hq, s.d), 0x1234, dtype=torch.int16, device="cuda")
    out = s.call(Q_out=q_out)
    want = s.expect(orc)
    s.compare(want)
    s.compare_queries(out, 0x1234)
    # again, over itself: the same bytes
    first = s.cache.to_host()
    s.call(Q_out=q_out)
    for name, x in s.cache.to_host().items():
        assert np.array_equal(x, first[name]), name


def test_queries_in_place_and_absent(orc):
    for inter, rot in ((False, 128), (True, 128), (False, 38), (True, 38)):
        s = Setup(orc, B=2, n=5, H=2, G=3, d=128, M=16, C=2, r=8, start=[0, 4], inter=inter, rot=rot, seed=40)
        q = s.dev(s.Q.view(np.int16))
        assert s.call(Q=q, Q_out=q) is q
        s.compare(s.expect(orc))
        s.compare_queries(q)
        s.cache.load_packed(s.before)
        assert s.call(Q=None) is None
        s.compare(s.expect(orc))


def test_tokens_without_a_place_are_dropped_and_reported(orc):
    import bit_kv_cache_centroid_b200 as kv2
    for n in (2, 80):                                              # one and several keys per warp
        s = Setup(orc, B=4, n=n, H=2, G=1, d=64, M=16, C=2, r=8, start=[0, 128, 256 - n + 1, -1], page=128, cap=256, seed=50 + n)
        s.pos[0, 0], s.pos[0, 1] = s.rows, -1                      # no such row of the table
        tab = s.before.table.copy()
        tab[1, 1] = -1                                             # an unmapped page
        s.cache.block_table.copy_(torch.from_numpy(tab))
        skip = {(0, 0), (0, 1), (2, n - 1), (3, 0)} | {(1, t) for t in range(n)}
        ws = torch.zeros(kv2.kv2_rotary_append_workspace_size(s.cache, n), dtype=torch.uint8, device="cuda")
        out = s.call(ws=ws)
        s.compare(s.expect(orc, skip))
        assert ws[:4].view(torch.int32).item() == 1
        q = out.view(torch.bfloat16).cpu()
        assert torch.isnan(q[0, :2]).all() and torch.isfinite(q[0, 2:]).all() and torch.isfinite(q[1:]).all()


def test_captured_append_replays_with_other_places(orc):
    import bit_kv_cache_centroid_b200 as kv2
    s = Setup(orc, B=3, n=30, H=2, G=2, d=128, M=64, C=4, r=8, start=[0, 40, 7], count=[30, 2, 0], cap=256, seed=60)
    t = {k: s.dev(v) for k, v in dict(K=s.K.view(np.int16), V=s.V.view(np.int16), Q=s.Q.view(np.int16), positions=s.pos,
                                     start=s.start, count=s.count).items()}
    t["ws"] = torch.zeros(kv2.kv2_rotary_append_workspace_size(s.cache, s.n), dtype=torch.uint8, device="cuda")
    t["Q_out"] = torch.zeros_like(t["Q"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.call(**t)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            s.call(**t)
    for start, count in (([100, 0, 50], [1, 30, 29]), ([3, 3, 3], [0, 0, 0]), ([200, 10, 226], [30, 30, 30])):
        torch.cuda.synchronize()
        s.cache.load_packed(s.before)
        s.start, s.count = np.asarray(start, np.int32), np.asarray(count, np.int32)
        t["start"].copy_(s.dev(s.start))
        t["count"].copy_(s.dev(s.count))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        s.compare(s.expect(orc))


def test_serving_loop_appends_and_attends(orc):
    """Two prompts enter a prefix cache, three samples of each continue them: every step appends one rotated token per
    sequence and attends to prefix and own tokens; an encoder's states are attended to on the side. Each output against
    plain 64-bit attention on the caches' bytes."""
    import bit_kv_cache_centroid_b200 as kv2
    H, G, d, M, r, C = 2, 4, 128, 64, 8, 4
    rng = np.random.default_rng(70)
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(torch.bfloat16)
    cent = torch.from_numpy(wl.f16_bits(rng.standard_normal((H, M, d)).astype(np.float32)).view(np.int16))
    fit = orc.fit(wl.bf16_bits(rng.standard_normal((64, H * G, d)).astype(np.float32)), H, r)
    make = lambda B, cap, page=0: kv2.Cache(B, H, d, M, r, cap, cent, page_tokens=page)
    pre, own_, enc = make(2, 256, 128), make(6, 64), make(6, 96)
    for c in (pre, own_, enc):
        c.set_fit(torch.from_numpy(fit.P), torch.from_numpy(fit.w), torch.from_numpy(fit.Wg))
    rot = kv2.Rotary(torch.from_numpy(table(300, d, 1)).cuda())
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    plens = ints([150, 33])
    at = torch.arange(150, dtype=torch.int32, device="cuda").repeat(2, 1)
    kv2.kv2_rotary_append(pre, rot, bf(2, 150, H, d).cuda(), bf(2, 150, H, d).cuda(), at, ints([0, 0]), C, count=plens)
    elens = ints([96, 1, 0, 40, 95, 13])
    kv2.kv2_quantize_append(enc, bf(6, 96, H, d).cuda(), bf(6, 96, H, d).cuda(), 0, C)
    lens = ints([0, 5, 0, 1, 0, 20])                                # places that differ from the start
    zero = torch.zeros(6, 20, H, d, dtype=torch.bfloat16, device="cuda")
    kv2.kv2_rotary_append(own_, rot, bf(6, 20, H, d).cuda(), zero, torch.zeros(6, 20, dtype=torch.int32, device="cuda"),
                          ints([0] * 6), C, count=lens)
    P = torch.from_numpy(fit.P)

    def host(c):
        pc = wl.PackedCache.empty(c.B, H, d, M, r, c.capacity, cent.numpy().view(np.uint16))
        for k, v in c.to_host().items():
            setattr(pc, k, v)
        if c.block_table is not None:
            pc.table, pc.page = c.block_table.cpu().numpy(), c.page_tokens
        return pc

    for step in range(4):
        pos = (plens.repeat_interleave(3) + lens)[:, None].contiguous()
        q = kv2.kv2_rotary_append(own_, rot, bf(6, 1, H, d).cuda(), bf(6, 1, H, d).cuda(), pos, lens, C, Q=bf(6, 1, H * G, d).cuda())
        lens = lens + 1
        a = kv2.kv2_attention_shared(pre, plens, own_, lens, q[:, 0], d ** -0.5).cpu()
        x = kv2.kv2_attention_cross(enc, elens, q, d ** -0.5).cpu()
        hp, ho, he = host(pre), host(own_), host(enc)
        qh = q.view(torch.bfloat16).cpu().double()
        for b in range(6):
            for h in range(H):
                qq = qh[b, 0, h * G:(h + 1) * G]
                parts = [(plain.tokens(hp, b // 3, h, int(plens[b // 3])), False), (plain.tokens(ho, b, h, int(lens[b])), False)]
                o, sg = plain.attend(qq, parts, P[h], d ** -0.5)
                plain.check(a[b, h * G:(h + 1) * G], o, sg, torch.float32, f"step {step} sequence {b}")
                o, sg = plain.attend(qq, [(plain.tokens(he, b, h, int(elens[b])), False)], P[h], d ** -0.5)
                plain.check(x[b, 0, h * G:(h + 1) * G], o, sg, torch.float32, f"cross, step {step} sequence {b}")
