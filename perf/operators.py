"""Measured operators of the packed 2-bit cache: rotary append, decode over a
shared prefix, cross attention.

Each operator has a plain form (elementary torch operations, fp32, rounded once
at the end) and the library's own call; both take the same state.

* ``rotary_append``: keys and queries are rotated by their positions, and keys
  and values are quantized into the packed cache at per-sequence places.
* ``shared_decode``: one query per sequence against a prefix that groups of
  sequences share (stored once) and each sequence's own cache.
* ``cross``: queries of one length against cached states of another length per
  sequence (an encoder's), without a mask between them; one query per sequence
  is its decode form.
"""
import math
import random

import torch

own = False

F16, BF16, F32, F64 = torch.float16, torch.bfloat16, torch.float32, torch.float64


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _append(name, B, n, H, Hq, d, M, C, r, **kw):
    return {"name": name, "op": "append", "B": B, "n": n, "H": H, "Hq": Hq, "d": d, "M": M, "C": C, "r": r,
            "group": 32, "page": 0, "pages": 1, "rot": d, "interleaved": False, "ragged": False, "salt": 1, **kw}


def _shared(name, groups, per, H, Hq, d, M, r, prefix, own_len, **kw):
    return {"name": name, "op": "shared", "groups": groups, "per": per, "H": H, "Hq": Hq, "d": d, "M": M, "r": r,
            "prefix": prefix, "own_len": own_len, "group": 32, "fmt": 0, "page": 0, "ragged": True, "salt": 1, **kw}


def _cross(name, B, nq, H, Hq, d, M, r, length, **kw):
    return {"name": name, "op": "cross", "B": B, "nq": nq, "H": H, "Hq": Hq, "d": d, "M": M, "r": r,
            "length": length, "group": 32, "fmt": 0, "page": 0, "ragged": True, "ragged_q": False, "salt": 1, **kw}


def listed():
    return [
        # one decode step's append for the LLM-shaped cache: 8 sequences, each at its own place of a paged cache
        _append("append_step", 8, 1, 8, 32, 128, 64, 4, 8, page=128, pages=16),
        # prompts of different lengths (padded batch) entering a paged cache, a part of the channels rotated
        _append("append_prompts", 6, 777, 8, 32, 128, 64, 4, 8, page=256, pages=4, rot=64, ragged=True),
        # a video chunk's three latent frames, 40 heads, contiguous cache; the pairs are neighbouring channels
        _append("append_chunk", 1, 4680, 40, 40, 128, 256, 8, 8, interleaved=True),
        # a small model's prompts: 64 channels a head, one scale and zero for all of them
        _append("append_narrow", 3, 211, 4, 8, 64, 16, 4, 8, group=64, ragged=True),

        # a short instruction shared by a few short continuations: launch latency counts
        _shared("shared_short", 1, 4, 8, 32, 128, 64, 8, 200, 60),
        # eight continuations of one 32,768-token prompt (the LLM decode workload's shapes)
        _shared("shared_prompt", 1, 8, 8, 32, 128, 64, 8, 32768, 256),
        # many samples of the same long prompt, the smallest cache format (83 bytes a token and head)
        _shared("shared_samples", 1, 64, 8, 32, 128, 64, 8, 32768, 515, group=128, fmt=1),
        # three prompts of different length, 64 channels, one query head per KV head, ids of 16 bits, paged
        _shared("shared_groups", 3, 11, 12, 12, 64, 300, 16, 5001, 700, page=128),

        # one decode step's cross attention over encoder states of about 30 s of sound, ragged batch
        _cross("cross_step", 16, 1, 8, 32, 128, 64, 8, 1500),
        # a prompt's cross attention, padded on both sides
        _cross("cross_prompt", 4, 509, 8, 32, 128, 64, 8, 2047, ragged_q=True, page=128),
        # a video chunk's queries against a text encoder's 512 states, 40 heads
        _cross("cross_chunk", 1, 4680, 40, 40, 128, 256, 8, 512, ragged=False),
        # narrow heads, int8 coefficients, few states
        _cross("cross_narrow", 2, 130, 6, 12, 64, 16, 16, 77, group=64, fmt=1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "shared", "cross"])
    d = rng.choice([64, 128, 128])
    H = rng.choice([1, 2, 4, 8, 8, 12, 16])
    G = rng.choice([1, 2, 4, 4, 8])
    M = _log(rng, 4, 500)
    r = rng.choice([0, 8, 8, 16])
    group = rng.choice([g for g in (32, 64, 128) if g <= d])
    page = rng.choice([0, 128, 256])
    salt = rng.randrange(1 << 30)
    if op == "append":
        B = _log(rng, 1, 32)
        n = rng.choice([1, _log(rng, 1, max(1, 20000 // (B * H)))])
        pages = max(2, -(-2 * n // page)) if page else 1
        return _append("", B, n, H, H * G, d, M, rng.randint(1, min(M, 12)), r, group=group, page=page, pages=pages,
                       rot=rng.choice([d, d, d // 2, 2 * rng.randint(1, d // 2)]), interleaved=rng.random() < 0.5,
                       ragged=rng.random() < 0.7, salt=salt)
    if op == "shared":
        groups, per = rng.choice([1, 1, 2, 5]), _log(rng, 1, 40)
        return _shared("", groups, per, H, H * G, d, M, r, _log(rng, 1, 20000 // groups), _log(rng, 1, 600), group=group,
                       fmt=rng.choice([0, 1]), page=page, salt=salt)
    B = _log(rng, 1, 12)
    nq = rng.choice([1, _log(rng, 1, max(1, 20000 // (B * H * G)))])
    return _cross("", B, nq, H, H * G, d, M, r, _log(rng, 1, 4000), group=group, fmt=rng.choice([0, 1]), page=page,
                  ragged=rng.random() < 0.8, ragged_q=rng.random() < 0.5, salt=salt)


# Lengths belong to the case (the same for every seed): they decide its work.

def _ragged(rng, n, most):
    """n lengths of 0..most, the longest present; the rest between a fifth and all of it."""
    out = [rng.randint(most // 5, most) for _ in range(n)]
    out[rng.randrange(n)] = most
    return out


def _lengths(case):
    """The case's whole numbers: lengths (and, for appends, places) per sequence."""
    rng = random.Random(case["salt"])
    if case["op"] == "append":
        count = _ragged(rng, case["B"], case["n"]) if case["ragged"] else [case["n"]] * case["B"]
        cap = _capacity(case)
        return {"count": count, "start": [rng.randint(0, cap - case["n"]) for _ in count]}
    if case["op"] == "shared":
        pre = _ragged(rng, case["groups"], case["prefix"])
        return {"prefix": pre, "own_len": _ragged(rng, case["groups"] * case["per"], case["own_len"])}
    lens = _ragged(rng, case["B"], case["length"]) if case["ragged"] else [case["length"]] * case["B"]
    q = _ragged(rng, case["B"], case["nq"]) if case["ragged_q"] else [case["nq"]] * case["B"]
    return {"lens": lens, "q_lens": q}


def _capacity(case):
    if case["op"] == "append":
        return case["page"] * case["pages"] if case["page"] else (case["n"] + 16 + 15) // 16 * 16
    raise KeyError(case["op"])


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=F32)


def _basis(g, H, d, r):
    return torch.linalg.qr(_randn(g, H, d, max(r, 1)).double())[0][:, :, :max(r, 1)].float().contiguous()


def _table(g, B, cap, page):
    """A block table over a pool with a few pages to spare, in random order."""
    n = B * (cap // page)
    order = torch.randperm(n + 3, generator=g, device="cuda")[:n]
    return order.to(torch.int32).view(B, cap // page).contiguous(), n + 3


def _packed(g, B, H, length, d, M, r, group, fmt, page):
    """A filled packed cache: uniform codes and ids, log-normal scales, zeros near -1.5 scales, small coefficients.
    Beyond a sequence's length the streams hold whatever was there before (other codes)."""
    unit = page or 16
    cap = -(-length // unit) * unit
    c = {"B": B, "H": H, "d": d, "M": M, "r": r, "group": group, "fmt": fmt, "page": page, "cap": cap}
    if page:
        c["table"], pages = _table(g, B, cap, page)
        lead = (pages, H, page)
    else:
        c["table"], lead = None, (B, H, cap)
    words = lambda: torch.randint(-2 ** 31, 2 ** 31, lead + (d // 16,), generator=g, device="cuda", dtype=torch.int64).int()
    c["k_code"], c["v_code"] = words(), words()
    for s in ("k_sz", "v_sz"):
        scale = 0.5 * torch.exp(0.4 * _randn(g, *lead, d // group))
        zero = -1.5 * scale + 0.1 * _randn(g, *lead, d // group)
        c[s] = torch.stack([scale.half(), zero.half()], -1).view(torch.int32).squeeze(-1).contiguous()
    ids = torch.randint(0, M, lead, generator=g, device="cuda")
    c["cidx"] = ids.to(torch.uint8) if M <= 256 else ids.to(torch.int16)
    coef = 0.05 * _randn(g, *lead, max(r, 1))
    if fmt == 1:
        scale = (coef.abs().amax(-1) / 127).half()
        c["psac"] = (coef / scale.float().clamp_min(1e-7).unsqueeze(-1)).round().clamp(-127, 127).to(torch.int8)
        c["psac_scale"] = scale.view(torch.int16)
    else:
        c["psac"], c["psac_scale"] = coef.half().view(torch.int16), None
    c["centroids"] = _randn(g, H, M, d).half().view(torch.int16)
    c["P"] = _basis(g, H, d, r)
    return c


def _handle(c):
    """The library's cache object over the streams of ``c``."""
    import bit_kv_cache_centroid_b200 as kv2
    h = kv2.Cache(1, c["H"], c["d"], c["M"], c["r"], 16, c["centroids"], psac_fmt=c["fmt"], group=c["group"])
    h.B, h.capacity, h.page_tokens, h.block_table = c["B"], c["cap"], c["page"], c["table"]
    h.num_pages = c["k_code"].shape[0] if c["page"] else 0
    for n in ("k_code", "v_code", "k_sz", "v_sz", "cidx", "psac", "psac_scale", "P"):
        setattr(h, n, c[n])
    if "w" in c:
        h.w, h.Wg = c["w"], c["Wg"]
    return h


def _workspace(size):
    return torch.zeros(size, dtype=torch.uint8, device="cuda")


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    n = _lengths(case)
    H, Hq, d = case["H"], case["Hq"], case["d"]
    s = {"case": case, "scale": d ** -0.5}
    if case["op"] == "append":
        B, M, r, rot = case["B"], case["M"], case["r"], case["rot"]
        cap = _capacity(case)
        c = _packed(g, B, H, cap, d, M, r, case["group"], 0, case["page"])
        for name in ("k_code", "v_code", "k_sz", "v_sz", "cidx", "psac"):
            c[name].zero_()
        # channels of uneven size; centres drawn like the keys, each key near one of them
        channel = torch.exp(0.7 * _randn(g, H, 1, d))
        cent = _randn(g, H, M, d) * channel
        c["centroids"] = cent.half().view(torch.int16)
        near = torch.randint(0, M, (B, case["n"], H), generator=g, device="cuda")
        keys = cent[torch.arange(H, device="cuda"), near] + 0.6 * channel[:, 0] * _randn(g, B, case["n"], H, d)
        s["K"] = keys.to(BF16).view(torch.int16)
        s["V"] = _randn(g, B, case["n"], H, d).to(BF16).view(torch.int16)
        s["Q"] = _randn(g, B, case["n"], Hq, d).to(BF16).view(torch.int16)
        c["w"] = torch.exp(_randn(g, H, d))
        c["Wg"] = c["w"].view(H, d // case["group"], case["group"]).sum(-1)
        far = torch.randint(0, 1000, (B, 1), generator=g, device="cuda")
        start = _ints(n["start"])
        pos = start[:, None] + far + torch.arange(case["n"], device="cuda")
        s["positions"] = pos.to(torch.int32).contiguous()
        s["start"], s["count"] = start, _ints(n["count"])
        rows = cap + 1000
        freq = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=F64) / rot)
        angle = torch.arange(rows, device="cuda", dtype=F64)[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["Q_out"] = torch.zeros_like(s["Q"])
        s["cache"] = c
        if own:
            import bit_kv_cache_centroid_b200 as kv2
            s["handle"] = _handle(c)
            s["rotary"] = kv2.Rotary(s["cos_sin"], interleaved=case["interleaved"])
            s["ws"] = _workspace(kv2.kv2_rotary_append_workspace_size(s["handle"], case["n"]))
        return s
    if case["op"] == "shared":
        B = case["groups"] * case["per"]
        args = (d, case["M"], case["r"], case["group"], case["fmt"], case["page"])
        s["prefix"] = _packed(g, case["groups"], H, case["prefix"], *args)
        s["cache"] = _packed(g, B, H, case["own_len"], *args)
        for name in ("centroids", "P"):
            s["cache"][name] = s["prefix"][name]
        s["prefix_lens"], s["lens"] = _ints(n["prefix"]), _ints(n["own_len"])
        s["Q"] = (1.5 * _randn(g, B, Hq, d)).to(BF16).view(torch.int16)
        s["out"] = torch.zeros((B, Hq, d), dtype=BF16, device="cuda")
        if own:
            import bit_kv_cache_centroid_b200 as kv2
            s["handle"], s["prefix_handle"] = _handle(s["cache"]), _handle(s["prefix"])
            s["ws"] = _workspace(kv2.kv2_attention_shared_workspace_size(s["prefix_handle"], s["handle"], Hq, case["prefix"],
                                                                     case["own_len"]))
        return s
    B = case["B"]
    s["cache"] = _packed(g, B, H, case["length"], d, case["M"], case["r"], case["group"], case["fmt"], case["page"])
    s["lens"] = _ints(n["lens"])
    s["q_lens"] = _ints(n["q_lens"]) if case["ragged_q"] else None
    s["Q"] = (1.5 * _randn(g, B, case["nq"], Hq, d)).to(BF16).view(torch.int16)
    s["out"] = torch.zeros((B, case["nq"], Hq, d), dtype=BF16, device="cuda")
    if own:
        import bit_kv_cache_centroid_b200 as kv2
        s["handle"] = _handle(s["cache"])
        s["ws"] = _workspace(kv2.kv2_attention_cross_workspace_size(s["handle"], Hq, case["nq"], case["length"]))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    if case["op"] == "append":
        return _plain_append(s, case)
    if case["op"] == "shared":
        return _plain_shared(s, case)
    return _plain_cross(s, case)


def _run_own(s, case):
    import bit_kv_cache_centroid_b200 as kv2
    if case["op"] == "append":
        kv2.kv2_rotary_append(s["handle"], s["rotary"], s["K"], s["V"], s["positions"], s["start"], case["C"],
                              count=s["count"], Q=s["Q"], Q_out=s["Q_out"], ws=s["ws"])
        return _append_outputs(s)
    if case["op"] == "shared":
        return kv2.kv2_attention_shared(s["prefix_handle"], s["prefix_lens"], s["handle"], s["lens"], s["Q"], s["scale"],
                                        kv2.KV2_OUT_BF16, max_prefix_len=case["prefix"], max_len=case["own_len"],
                                        out=s["out"], ws=s["ws"])
    return kv2.kv2_attention_cross(s["handle"], s["lens"], s["Q"], s["scale"], kv2.KV2_OUT_BF16, q_lens=s["q_lens"],
                                   max_len=case["length"], out=s["out"], ws=s["ws"])


def _append_outputs(s):
    c = s["cache"]
    out = [c["k_code"], c["v_code"], c["k_sz"], c["v_sz"], c["cidx"]]
    if c["r"]:
        out.append(c["psac"].view(F16))
    return out + [s["Q_out"].view(BF16)]


# plain forms ---------------------------------------------------------------

def _rotate(x, cos_sin, interleaved, rot):
    """x [..., d] (fp32) with channel pairs turned by the angles of cos_sin [..., rot], each product and sum rounded."""
    half = rot // 2
    cos, sin = cos_sin[..., :half], cos_sin[..., half:]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :half], x[..., half:rot])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _toward(x, up):
    """fp32 -> fp16 rounded down (or up)."""
    h = x.half()
    bits = h.view(torch.int16)
    off = h.float() < x if up else h.float() > x
    away = bits < 0 if not up else bits >= 0                # the next value that way has the larger magnitude
    return torch.where(off, torch.where(away, bits + 1, bits - 1), bits).view(F16)


def _scale_zero(x):
    """fp16 zero (range's low end) and scale (a third of the range) of groups x [..., group]."""
    zero = _toward(x.amin(-1), False)
    return _toward((x.amax(-1) - zero.float()) / 3.0, True), zero


def _encode(x, group):
    """INT2 codec of rows x [H, n, d]: code words [H, n, d/16], scale and zero words [H, n, d/group], what the codes leave."""
    H, n, d = x.shape
    xg = x.reshape(H, n, d // group, group)
    scale, zero = _scale_zero(xg)
    sf, zf = scale.float().unsqueeze(-1), zero.float().unsqueeze(-1)
    code = torch.where(sf > 0, ((xg - zf) / sf).round().clamp(0, 3), torch.zeros_like(xg))
    left = (xg - (code * sf + zf)).view(H, n, d)
    shifts = torch.arange(0, 32, 2, device=x.device)
    words = (code.view(H, n, d // 16, 16).long() << shifts).sum(-1)
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).int()
    return words, torch.stack([scale, zero], -1).view(torch.int32).squeeze(-1), left


def _fma(a, b, c):
    """fp32 a * b + c, rounded once (the product is exact in 64 bits)."""
    return (a.double() * b.double() + c.double()).float()


def _choose(k, mu, w, Wg, C, group):
    """The centre of each key: k [H, n, d], mu [H, M, d]. The C nearest by the weighted distance, of those the one whose
    residual's scales cost least. The distance is defined as a chain of fp32 fused multiply-adds over the channels;
    which of two near centres is nearer depends on that order, so the chain is taken step by step."""
    H, n, d = k.shape
    M = mu.shape[1]
    dist = torch.zeros((H, n, M), device=k.device)
    for c in range(d):
        t = k[:, :, c:c + 1] - mu[:, None, :, c]
        dist = _fma(w[:, c, None, None] * t, t, dist)
    order = torch.sort(dist, dim=2, stable=True)[1][:, :, :C]
    head = torch.arange(H, device=k.device)[:, None, None]
    resid = (k[:, :, None, :] - mu[head, order]).view(H, n, C, d // group, group)
    scale = _scale_zero(resid)[0].float()
    cost = torch.zeros((H, n, C), device=k.device)
    for g in range(d // group):
        cost = _fma(Wg[:, g, None, None] * scale[..., g], scale[..., g], cost)
    best = cost == cost.amin(2, keepdim=True)
    return torch.where(best, order, torch.full_like(order, M)).amin(2)


def _plain_append(s, case):
    c, H, d, rot = s["cache"], case["H"], case["d"], case["rot"]
    used = torch.arange(case["n"], device="cuda") < s["count"][:, None]
    b, t = used.nonzero(as_tuple=True)
    turn = s["cos_sin"][s["positions"][b, t].long()][:, None, :]
    K = _rotate(s["K"].view(BF16)[b, t].float(), turn, case["interleaved"], rot).to(BF16).float()
    s["Q_out"].view(BF16)[b, t] = _rotate(s["Q"].view(BF16)[b, t].float(), turn, case["interleaved"], rot).to(BF16)
    V = s["V"].view(BF16)[b, t].float()
    slot = s["start"][b].long() + t
    if case["page"]:
        lead, at = c["table"][b, slot // case["page"]].long(), slot % case["page"]
    else:
        lead, at = b, slot
    mu = c["centroids"].view(F16).float()
    k, v = K.transpose(0, 1), V.transpose(0, 1)             # [H, n, d]
    j = _choose(k, mu, c["w"], c["Wg"], case["C"], case["group"])
    head = torch.arange(H, device="cuda")[:, None]
    words, sz, left = _encode(k - mu[head, j], case["group"])
    c["k_code"][lead, head, at], c["k_sz"][lead, head, at] = words, sz
    c["cidx"][lead, head, at] = j.to(c["cidx"].dtype)
    if case["r"]:
        c["psac"].view(F16)[lead, head, at] = (left @ c["P"]).half()
    words, sz, _ = _encode(v, case["group"])
    c["v_code"][lead, head, at], c["v_sz"][lead, head, at] = words, sz
    return _append_outputs(s)


def _rows(c, name):
    """A stream of the cache as [B, H, cap, ...], pages put in order."""
    x = c[name]
    if c["table"] is None:
        return x
    y = x[c["table"].long()].transpose(1, 2)                # [B, H, pages, page, ...]
    return y.reshape((c["B"], c["H"], c["cap"]) + x.shape[3:])


def _values(c, code, sz):
    words, two = _rows(c, code), _rows(c, sz).view(F16)
    shifts = torch.arange(0, 32, 2, device="cuda", dtype=torch.int32)
    q = ((words.unsqueeze(-1) >> shifts) & 3).flatten(-2).float()
    scale, zero = (two[..., i::2].float().repeat_interleave(c["group"], -1) for i in (0, 1))
    return q * scale + zero


def _keys(c):
    """Reconstructed keys with the coefficients' compensation: q . (k + P a) is the compensated score."""
    ids = _rows(c, "cidx").long() & (0xFF if c["M"] <= 256 else 0xFFFF)
    mu = c["centroids"].view(F16).float()
    k = _values(c, "k_code", "k_sz") + mu[torch.arange(c["H"], device="cuda")[:, None], ids]
    if not c["r"]:
        return k
    if c["fmt"] == 1:
        a = _rows(c, "psac").float() * _rows(c, "psac_scale").view(F16).float().unsqueeze(-1)
    else:
        a = _rows(c, "psac").view(F16).float()
    return k + a @ c["P"].transpose(1, 2)


def _masked(scores, lens, length):
    """scores [B, ..., length] with the positions at and beyond each sequence's length at minus infinity."""
    dead = torch.arange(length, device="cuda") >= lens.view(-1, *([1] * (scores.dim() - 1)))
    return scores.masked_fill(dead, -math.inf)


def _weights(scores):
    """Softmax numerators (0 where nothing is left) and their sum."""
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    return p, p.sum(-1, keepdim=True)


def _plain_shared(s, case):
    pre, c = s["prefix"], s["cache"]
    N, S, H, d = case["groups"], case["per"], case["H"], case["d"]
    G = case["Hq"] // H
    q = s["Q"].view(BF16).float().view(N, S, H, G, d) * s["scale"]
    qh = q.permute(0, 2, 1, 3, 4).reshape(N, H, S * G, d)
    a = _masked(qh @ _keys(pre).transpose(2, 3), s["prefix_lens"], pre["cap"])        # [N, H, S*G, Lp]
    a = a.view(N, H, S, G, -1).permute(0, 2, 1, 3, 4)                                      # [N, S, H, G, Lp]
    b = _masked(q.reshape(N * S, H, G, d) @ _keys(c).transpose(2, 3), s["lens"], c["cap"]).view(N, S, H, G, -1)
    p, total = _weights(torch.cat([a, b], -1))
    pa, pb = p[..., :pre["cap"]], p[..., pre["cap"]:]
    oa = pa.permute(0, 2, 1, 3, 4).reshape(N, H, S * G, -1) @ _values(pre, "v_code", "v_sz")
    oa = oa.view(N, H, S, G, d).permute(0, 2, 1, 3, 4)
    ob = (pb.reshape(N * S, H, G, -1) @ _values(c, "v_code", "v_sz")).view(N, S, H, G, d)
    out = (oa + ob) / torch.where(total > 0, total, torch.ones_like(total))
    s["out"].copy_(out.reshape(N * S, case["Hq"], d))
    return s["out"]


def _plain_cross(s, case):
    c, B, nq, H, d = s["cache"], case["B"], case["nq"], case["H"], case["d"]
    G = case["Hq"] // H
    q = s["Q"].view(BF16).float().view(B, nq, H, G, d).permute(0, 2, 1, 3, 4).reshape(B, H, nq * G, d) * s["scale"]
    p, total = _weights(_masked(q @ _keys(c).transpose(2, 3), s["lens"], c["cap"]))
    out = (p @ _values(c, "v_code", "v_sz")) / torch.where(total > 0, total, torch.ones_like(total))
    out = out.view(B, H, nq, G, d).permute(0, 2, 1, 3, 4).reshape(B, nq, case["Hq"], d).to(BF16)
    if s["q_lens"] is None:
        s["out"].copy_(out)
    else:                                                   # rows behind a sequence's queries stay as they were
        live = torch.arange(nq, device="cuda") < s["q_lens"][:, None]
        s["out"].copy_(torch.where(live[:, :, None, None], out, s["out"]))
    return s["out"]


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "shared": _exact_shared, "cross": _exact_cross}[case["op"]](s, case)


def _exact_rot(x, turn, case):
    """x [n, heads, d] with its channel pairs, as complex numbers, times cos + i sin of the table's rows turn [n, rot]."""
    half = case["rot"] // 2
    y, z = x.double().clone(), torch.complex(turn[:, :half].double(), turn[:, half:].double())[:, None]
    if case["interleaved"]:
        pairs = torch.view_as_complex(y[..., :2 * half].unflatten(-1, (half, 2)).contiguous())
        y[..., :2 * half] = torch.view_as_real(pairs * z).flatten(-2)
    else:
        pairs = torch.complex(y[..., :half], y[..., half:2 * half]) * z
        y[..., :2 * half] = torch.cat([pairs.real, pairs.imag], -1)
    return y


def _exact_append(s, case):
    """The coefficients and rotated queries; codes, scales and ids are decisions taken in fp32 and have no such value.
    The key that is coded is the rotated one rounded to bf16, its rotation defined in fp32: a part of the decisions."""
    c, H, d, group = s["cache"], case["H"], case["d"], case["group"]
    n = _lengths(case)
    pos = s["positions"]
    q_out = torch.zeros(s["Q_out"].shape, dtype=F64, device="cuda")
    coef = torch.zeros(c["psac"].shape, dtype=F64, device="cuda")
    for b in range(case["B"]):
        m, first = n["count"][b], n["start"][b]
        if m == 0:
            continue
        turn = s["cos_sin"][pos[b, :m].long()]
        q_out[b, :m] = _exact_rot(s["Q"][b, :m].view(BF16), turn, case)
        if not case["r"]:
            continue
        k = _rotate(s["K"][b, :m].view(BF16).float(), turn[:, None, :], case["interleaved"], case["rot"]).to(BF16).double()
        slots = torch.arange(first, first + m, device="cuda")
        lead, at = (c["table"][b].long()[slots // case["page"]], slots % case["page"]) if case["page"] else (torch.full_like(slots, b), slots)
        for h in range(H):
            mu, w = c["centroids"][h].view(F16).double(), c["w"][h].double()
            x = k[:, h]
            near = ((x * x) @ w)[:, None] - 2 * (x * w) @ mu.T + (mu * mu) @ w
            ids = near.topk(case["C"], dim=1, largest=False)[1].sort(1)[0]
            res = x[:, None] - mu[ids]
            g = res.reshape(m, case["C"], d // group, group)
            low = _toward(g.amin(-1).float(), False).double()
            step = _toward(((g.amax(-1) - low) / 3).float(), True).double()
            pick = (step * step * c["Wg"][h].double()).sum(-1).argmin(1)
            rows = torch.arange(m, device="cuda")
            g, low, step = g[rows, pick], low[rows, pick][..., None], step[rows, pick][..., None]
            ratio = ((g - low).float() / step.float()).double()     # (the code is a decision in fp32 too)
            code = torch.where(step > 0, ratio.round().clamp(0, 3), torch.zeros_like(g))
            coef[lead, h, at] = (g - (code * step + low)).reshape(m, d) @ c["P"][h].double()
    return [None] * 5 + ([coef] if case["r"] else []) + [q_out]


def _exact_kv(c, b, h, length):
    """Keys (compensated) and values of one sequence and head in 64 bits."""
    at = torch.arange(length, device="cuda")
    lead, at = (c["table"][b].long()[at // c["page"]], at % c["page"]) if c["page"] else (b, at)
    out = []
    for code, sz in (("k_code", "k_sz"), ("v_code", "v_sz")):
        byte = c[code][lead, h, at].contiguous().view(torch.uint8).int()                    # 4 channels a byte
        q = torch.stack([(byte // 4 ** i) % 4 for i in range(4)], -1).reshape(length, c["d"]).double()
        two = c[sz][lead, h, at].contiguous().view(F16).double().view(length, c["d"] // c["group"], 2)
        q = q.view(length, c["d"] // c["group"], c["group"])
        out.append((q * two[:, :, 0:1] + two[:, :, 1:2]).reshape(length, c["d"]))
    ids = c["cidx"][lead, h, at].long() % (256 if c["M"] <= 256 else 65536)
    k = out[0] + c["centroids"][h].view(F16).double()[ids]
    if c["r"]:
        a = c["psac"][lead, h, at]
        a = a.double() * c["psac_scale"][lead, h, at].view(F16).double()[:, None] if c["fmt"] == 1 else a.contiguous().view(F16).double()
        k = k + a @ c["P"][h].double().T
    return k, out[1]


def _exact_attend(q, k, v, scale):
    if k.shape[0] == 0:
        return torch.zeros_like(q)
    return torch.softmax(q @ k.T * scale, -1) @ v


def _exact_shared(s, case):
    n, H, S, d = _lengths(case), case["H"], case["per"], case["d"]
    G = case["Hq"] // H
    q = s["Q"].view(BF16).double().view(-1, H, G, d)
    out = torch.zeros_like(q)
    for p in range(case["groups"]):
        for h in range(H):
            kp, vp = _exact_kv(s["prefix"], p, h, n["prefix"][p])
            for b in range(p * S, (p + 1) * S):
                ko, vo = _exact_kv(s["cache"], b, h, n["own_len"][b])
                out[b, h] = _exact_attend(q[b, h], torch.cat([kp, ko]), torch.cat([vp, vo]), s["scale"])
    return out.view(-1, case["Hq"], d)


def _exact_cross(s, case):
    n, H, d = _lengths(case), case["H"], case["d"]
    G = case["Hq"] // H
    q = s["Q"].view(BF16).double().view(case["B"], case["nq"], H, G, d)
    out = torch.zeros_like(q)
    for b in range(case["B"]):
        m = n["q_lens"][b]
        for h in range(H):
            k, v = _exact_kv(s["cache"], b, h, n["lens"][b])
            out[b, :m, h] = _exact_attend(q[b, :m, h].reshape(m * G, d), k, v, s["scale"]).view(m, G, d)
    return out.view(case["B"], case["nq"], case["Hq"], d)


# ---------------------------------------------------------------------------
# what one pass cannot do without
# ---------------------------------------------------------------------------

def _token_bytes(case, fmt):
    """Packed bytes of one token and KV head."""
    d, r = case["d"], case["r"]
    return 2 * (d // 4) + 8 * (d // case["group"]) + (1 if case["M"] <= 256 else 2) + ((r + 2 if r else 0) if fmt else 2 * r)


def _tables(case):
    return case["H"] * (case["M"] * case["d"] * 2 + case["d"] * case["r"] * 4)


def work(case):
    n, H, Hq, d = _lengths(case), case["H"], case["Hq"], case["d"]
    if case["op"] == "append":
        rows = sum(n["count"])
        per_key = 2 * case["M"] * d + 3 * case["C"] * d + 2 * case["r"] * d + 8 * d
        move = rows * (H * (4 * d + _token_bytes(case, 0)) + Hq * 4 * d + 4 * case["rot"] + 4)
        return {"bytes": move + _tables(case) + H * (d + d // case["group"]) * 4, "flops": rows * (H * per_key + 3 * (H + Hq) * case["rot"])}
    if case["op"] == "shared":
        B, per = case["groups"] * case["per"], case["per"]
        tokens = sum(n["prefix"]) + sum(n["own_len"])
        pairs = Hq * (per * sum(n["prefix"]) + sum(n["own_len"]))
        return {"bytes": tokens * H * _token_bytes(case, case["fmt"]) + _tables(case) + B * Hq * d * 4,
                "flops": pairs * (4 * d + 2 * case["r"])}
    pairs = Hq * sum(a * b for a, b in zip(n["lens"], n["q_lens"]))
    return {"bytes": sum(n["lens"]) * H * _token_bytes(case, case["fmt"]) + _tables(case) + sum(n["q_lens"]) * Hq * d * 4,
            "flops": pairs * (4 * d + 2 * case["r"])}
