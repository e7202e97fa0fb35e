"""Plain 64-bit attention over a host packed cache, with the size of the
error that the tensor-core kernel's roundings leave (tests only).

Per output channel c of a row with weights w_t, values v_t and result o, the
kernel's independent roundings are, with u = 2^-11 (half a step of fp16):

* of each key: z + mu, then code s + that, each uniform within u of the value
  (variance u^2 x^2 / 3), and of an int8 coefficient's product with its scale;
  they move the score s_t by delta_t, whose variance is computed below, and the
  output by sum_t w_t delta_t (v_t - o);
* of the projected query u_i, common to all tokens: the output moves by
  sum_i e_i sum_t w_t a_ti (v_t - o);
* of each value (one rounding) and each probability (one rounding):
  sum_t w_t (e_t + e'_t) v_t.

fp32 sums, exponentials (2^-22) and tensor-core accumulation (measured 2^-19 of
the sum of magnitudes) are far below; 2^-17 of the magnitudes covers them.
``sigma`` is the standard deviation of the sum; an element is allowed 8 of it
(the roundings are bounded, so no tail is longer), the whole output's root mean
square 3, on top of the output type's own half step.
"""
import numpy as np
import torch

U = 2.0 ** -11


def f16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits)).view(torch.float16).double()


def bf16(bits):
    return torch.from_numpy((np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).copy()).double()


def tokens(pc, b, h, n):
    """Fields of the first n tokens: (z + mu, khat, a, values, coefficient is a rounded product)."""
    if pc.table is not None:
        t = np.arange(n)
        at = (pc.table[b][t // pc.page], h, t % pc.page)
    else:
        at = (b, h, np.arange(n))
    d, g = pc.d, pc.group

    def field(code, sz):
        words = code[at].astype(np.uint32)
        q = ((words[:, :, None] >> np.arange(0, 32, 2, dtype=np.uint32)) & 3).reshape(n, d).astype(np.float64)
        w = sz[at]
        s = np.repeat((w & 0xFFFF).astype(np.uint16).view(np.float16).astype(np.float64), g, -1)
        z = np.repeat((w >> 16).astype(np.uint16).view(np.float16).astype(np.float64), g, -1)
        return torch.from_numpy(q * s), torch.from_numpy(z)

    kq, kz = field(pc.k_code, pc.k_sz)
    vq, vz = field(pc.v_code, pc.v_sz)
    zmu = kz + f16(pc.centroids[h][pc.cidx[at].astype(np.int64)])
    if pc.r == 0:
        a = torch.zeros(n, 0, dtype=torch.float64)
    elif pc.psac_fmt == 1:
        a = torch.from_numpy(pc.psac[at].astype(np.float64)) * f16(pc.psac_scale[at])[:, None]
    else:
        a = f16(pc.psac[at])
    return zmu, kq + zmu, a, vq + vz


def attend(q, parts, P, scale):
    """q [R, d] (fp64) against the tokens of ``parts`` (tuples of tokens(), each
    with whether its coefficients are int8) -> (o [R, d], sigma [R, d])."""
    R, d = q.shape
    zmu, k, a, v = (torch.cat([p[0][i] for p in parts]) for i in range(4))
    if k.shape[0] == 0:
        return torch.zeros(R, d, dtype=torch.float64), torch.zeros(R, d, dtype=torch.float64)
    r8 = torch.cat([torch.full((p[0][1].shape[0],), float(p[1]), dtype=torch.float64) for p in parts])
    u = q @ P.double()
    s = scale * (q @ k.T + u @ a.T)
    w = torch.softmax(s, -1)
    o = w @ v
    var_s = scale ** 2 * U ** 2 / 3 * ((q ** 2) @ (zmu ** 2 + k ** 2).T + (u ** 2) @ ((a ** 2) * r8[:, None]).T)
    # sum_t w_t^2 var_t (v_t - o)^2 expanded, per channel
    ww = w ** 2 * var_s
    var = ww @ (v ** 2) - 2 * o * (ww @ v) + o ** 2 * ww.sum(-1, keepdim=True)
    for i in range(a.shape[1]):
        wa = w * a[:, i]
        var = var + (scale * u[:, i:i + 1]) ** 2 * U ** 2 / 3 * (wa @ v - o * wa.sum(-1, keepdim=True)) ** 2
    var = var.clamp_min(0) + 2 * U ** 2 / 3 * (w ** 2) @ (v ** 2)
    return o, var.sqrt() + 2.0 ** -20 * (w @ v.abs())


def check(got, want, sigma, dtype, what=""):
    """Element and root-mean-square bounds (see the module's text)."""
    got = got.double().cpu()
    if got.numel() == 0:
        return
    assert torch.isfinite(got).all(), f"{what}: not finite"
    half = torch.finfo(dtype).eps / 2
    err = (got - want).abs()
    room = 8 * sigma + half * want.abs() * 1.01 + 2.0 ** -120
    over = (err - room).max().item()
    assert over <= 0, f"{what}: {int((err > room).sum())} elements over, worst by {over:.3e} (error {err.max().item():.3e})"
    rms, allow = err.square().mean().sqrt(), 3 * sigma.square().mean().sqrt() + (half * want).square().mean().sqrt()
    assert rms <= allow + 1e-30, f"{what}: rms {rms:.3e} above {allow:.3e}"
