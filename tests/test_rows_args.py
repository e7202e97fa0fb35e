"""Argument checks of cross attention and shared-prefix decode (no device
work), and the plain attention of the tests against mistakes planted in it."""
import ctypes

import numpy as np
import pytest
import torch

import rows_plain as plain
import workloads as wl


@pytest.fixture(scope="module")
def lib():
    import bit_kv_cache_centroid_b200 as kv2
    from bit_kv_cache_centroid_b200 import build
    build.build()
    return kv2.lib


def desc(**kw):
    import bit_kv_cache_centroid_b200 as kv2
    base = dict(B=2, H_kv=2, d=128, M=64, r=8, capacity=256, k_code=0x1000, v_code=0x2000, k_sz=0x3000, v_sz=0x4000,
                cidx=0x5000, psac=0x6000, centroids=0x7000, P=0x8000, w=0x9000, Wg=0xA000, psac_fmt=0, psac_scale=0,
                block_table=0, page_tokens=0, group=0)
    base.update(kw)
    return kv2.kv2_cache(**base)


def cross(lib, c, lens=0, max_len=256, Q=0x100, q_lens=0, Nq=3, H_q=4, out=0x200, dt=0, ws=0x300, n=1 << 30):
    return lib.kv2_attention_cross(None if c is None else ctypes.byref(c), lens or None, max_len, Q or None, q_lens or None,
                                   Nq, H_q, 1.0, out or None, dt, ws or None, n, None)


def shared(lib, p, c, plens=0, mp=256, lens=0, ml=256, Q=0x100, H_q=4, out=0x200, dt=0, ws=0x300, n=1 << 30):
    return lib.kv2_attention_shared(ctypes.byref(p), plens or None, mp, ctypes.byref(c), lens or None, ml, Q or None, H_q,
                                    1.0, out or None, dt, ws or None, n, None)


def test_cross_refusals(lib):
    c = desc()
    assert cross(lib, None) == 1
    assert cross(lib, desc(d=96)) == 2
    assert cross(lib, desc(r=24)) == 2 and b"r=24" in lib.kv2_last_error()
    assert cross(lib, c, H_q=5) == 2
    assert cross(lib, c, max_len=257) == 3 and b"max_len" in lib.kv2_last_error()
    assert cross(lib, c, max_len=-1) == 3
    assert cross(lib, c, lens=0x1002) == 1 and cross(lib, c, q_lens=0x1001) == 1
    assert cross(lib, c, Nq=-1) == 1
    assert cross(lib, c, Nq=(1 << 30) // 8 + 1) == 2                 # rows above 2^30
    assert cross(lib, c, Q=0) == 1 and cross(lib, c, Q=0x108) == 1 and cross(lib, c, out=0x204) == 1
    assert cross(lib, c, dt=2) == 1 and cross(lib, c, ws=0) == 1
    need = lib.kv2_attention_cross_workspace_size(ctypes.byref(c), 4, 3, 256)
    assert need > 0 and cross(lib, c, n=need - 1) == 6
    assert cross(lib, c, Nq=0) == 0                            # nothing to do
    assert lib.kv2_attention_cross_workspace_size(ctypes.byref(c), 5, 3, 256) == 0


def test_shared_refusals(lib):
    p, c = desc(B=1), desc(B=6)
    assert shared(lib, desc(B=4), c) == 1 and b"6 sequences for 4" in lib.kv2_last_error()
    assert shared(lib, desc(B=1, H_kv=4), c) == 1
    assert shared(lib, desc(B=1, d=64), c) == 1
    assert shared(lib, desc(B=1, r=10), c) == 2 and shared(lib, p, desc(B=6, r=32)) == 2
    assert shared(lib, p, c, mp=1000) == 3 and shared(lib, p, c, ml=1000) == 3
    assert shared(lib, p, c, plens=0x1001) == 1 and shared(lib, p, c, lens=0x1003) == 1
    assert shared(lib, p, c, Q=0) == 1 and shared(lib, p, c, ws=0x308) == 1
    need = lib.kv2_attention_shared_workspace_size(ctypes.byref(p), ctypes.byref(c), 4, 256, 256)
    assert need > 0 and shared(lib, p, c, n=need - 1) == 6
    assert lib.kv2_attention_shared_workspace_size(ctypes.byref(desc(B=4)), ctypes.byref(c), 4, 256, 256) == 0


def test_binding_refuses_wrong_tensors():
    import bit_kv_cache_centroid_b200 as kv2
    c = kv2.Cache(2, 2, 64, 16, 8, 256, np.zeros((2, 16, 64), np.int16), device="cpu")
    Q = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16)
    lens = torch.zeros(2, dtype=torch.int32)
    for bad in (dict(Q=Q[:, :, :, :32]), dict(Q=Q.float()), dict(Q=Q[0]), dict(Q=Q.transpose(1, 2)), dict(lens=lens.long()),
                dict(lens=lens[:1]), dict(Q=Q.transpose(1, 2).contiguous().transpose(1, 2))):
        a = dict(Q=Q, lens=lens, **{}) | bad
        with pytest.raises(ValueError):
            kv2.kv2_attention_cross(c, a["lens"], a["Q"], 1.0)
    with pytest.raises(ValueError):
        kv2.kv2_attention_shared(c, lens, c, lens, Q, 1.0)
    with pytest.raises(ValueError):
        kv2.kv2_attention_shared(c, lens[:1], c, lens, Q[:, 0], 1.0)


def _small(fmt=0, r=8):
    s = wl.Spec("t", 5, B=1, H_q=1, H_kv=1, d=64, M=16, C=1, r=r, T=160, n_new=0, capacity=160, n_hist=1, Nq=0,
                frame_tokens=1, key_law="gaussian", top_energy=0.7)
    pc = wl.random_packed_cache(s, psac_fmt=fmt)
    P = torch.linalg.qr(torch.randn(64, max(r, 1), generator=torch.Generator().manual_seed(1)))[0]
    return pc, P[:, :r]


def test_plain_attention_agrees_with_the_oracle(orc):
    """The tests' 64-bit form equals the oracle's decode; mistakes planted in it do not pass the tests' bound."""
    for fmt in (0, 1):
        pc, P = _small(fmt)
        rng = np.random.default_rng(3)
        Q = wl.bf16_bits(rng.standard_normal((1, 1, 64)).astype(np.float32) * 0.4)      # even weights: every token counts
        want = torch.from_numpy(orc.decode(pc, P.numpy()[None], 40, Q, 0.125))[0]
        tok = plain.tokens(pc, 0, 0, 40)
        o, sigma = plain.attend(plain.bf16(Q[0]), [(tok, fmt == 1)], P, 0.125)
        assert torch.allclose(o, want, rtol=1e-9, atol=1e-12)
        plain.check(want.float(), o, sigma, torch.float32)
        q = plain.bf16(Q[0])
        mistakes = {
            "a token less": plain.attend(q, [(tuple(x[:39] for x in tok), 0)], P, 0.125)[0],
            "a token more": plain.attend(q, [(plain.tokens(pc, 0, 0, 41), 0)], P, 0.125)[0],
            "no compensation": plain.attend(q, [((tok[0], tok[1], tok[2] * 0, tok[3]), 0)], P, 0.125)[0],
            "scale of another head size": plain.attend(q, [(tok, 0)], P, 128 ** -0.5)[0],
            "two tokens swapped in the values": plain.attend(q, [((*tok[:3], tok[3].roll(1, 0)), 0)], P, 0.125)[0],
        }
        for name, wrong in mistakes.items():
            with pytest.raises(AssertionError):
                plain.check(wrong.float(), o, sigma, torch.float32, name)


def rotary(lib, c, cs=0x100, positions=500, rot=128, inter=0, K=0x200, V=0x300, Q=0, Qo=0, H_q=4, pos=0x400, start=0x500,
           count=0, n=3, C=4, ws=0x600, nb=1 << 30):
    import bit_kv_cache_centroid_b200 as kv2
    r = kv2.kv2_rotary(cs, positions, rot, inter)
    return lib.kv2_rotary_append(ctypes.byref(c), ctypes.byref(r), K or None, V or None, Q or None, Qo or None, H_q, pos or None,
                                 start or None, count or None, n, C, ws or None, nb, None)


def test_rotary_refusals(lib):
    c = desc()
    assert lib.kv2_rotary_append(ctypes.byref(c), None, 0x200, 0x300, None, None, 4, 0x400, 0x500, None, 3, 4, 0x600, 1 << 30,
                                 None) == 1
    for rot in (0, 1, 63, 130, -2):
        assert rotary(lib, c, rot=rot) == 2, rot
    assert rotary(lib, c, positions=-1) == 1 and rotary(lib, c, inter=2) == 1
    assert rotary(lib, c, n=-1) == 1 and rotary(lib, c, C=0) == 1 and rotary(lib, c, C=65) == 1
    assert rotary(lib, c, n=(1 << 30) // 2) == 2                  # rows above 2^30 with two heads
    assert rotary(lib, c, cs=0) == 1 and rotary(lib, c, cs=0x104) == 1
    assert rotary(lib, c, K=0) == 1 and rotary(lib, c, V=0x308) == 1
    assert rotary(lib, c, Q=0x700) == 1 and rotary(lib, c, Q=0x700, Qo=0x708) == 1 and rotary(lib, c, Q=0x700, Qo=0x700, H_q=0) == 1
    assert rotary(lib, c, pos=0) == 1 and rotary(lib, c, start=0) == 1 and rotary(lib, c, count=0x501) == 1
    assert rotary(lib, c, ws=0) == 1
    need = lib.kv2_rotary_append_workspace_size(ctypes.byref(c), 3)
    assert need == 256 + 256 + 2 * 3 * 2 * 128 * 2 and rotary(lib, c, nb=need - 1) == 6
    assert rotary(lib, c, n=0) == 0
    assert rotary(lib, desc(w=0)) == 1


def test_rotary_binding_refuses_wrong_tensors():
    import bit_kv_cache_centroid_b200 as kv2
    c = kv2.Cache(2, 2, 64, 16, 8, 256, np.zeros((2, 16, 64), np.int16), device="cpu")
    rot = kv2.Rotary(torch.zeros(10, 64))
    K = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)
    pos, start = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    Q = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16)
    call = lambda K=K, V=K, pos=pos, start=start, **kw: kv2.kv2_rotary_append(c, rot, K, V, pos, start, 4, **kw)
    for bad in (dict(K=K[:1]), dict(V=K.float()), dict(pos=pos.long()), dict(pos=pos[:, :2]), dict(start=start[:1]),
                dict(count=start.long()), dict(Q=Q[:, :2]), dict(Q=Q[0]), dict(Q_out=Q), dict(start=None)):
        with pytest.raises((ValueError, AttributeError)):
            call(**bad)
    with pytest.raises(ValueError):
        kv2.Rotary(torch.zeros(10, 64, dtype=torch.float64))
    with pytest.raises(ValueError):
        kv2.Rotary(torch.zeros(10))
