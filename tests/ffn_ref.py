"""The gated feed-forward block and the 4-bit matrix-vector products in 64 bits, with what the kernels
may be off by. Plain torch on FP64 tensors (any device).

Bounds. A binary32 sum of K exact products is within K 2^-24 S of the exact sum in any order, S the sum
of the products' magnitudes; SUM doubles that for the matrix core's inner steps. A rounding to BF16 is
within 2^-8 of the value (2^-134 below its normal numbers), one to binary32 within 2^-24. sigma: its
exponential's argument, rounded in binary32, is off by 2^-24 relative, so e^-|g| by |g| 2^-24, at most
87.4 2^-24 < 2^-17.5 where it is not 0; with an ulp or two for each further step, EVAL = 2^-17 holds for sigma,
1 - sigma and what is made of them. Where e^-|g| is below 2^-126 it is 0: off by up to 2^-126."""

import torch

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
BF16, F32, EVAL, TINY, SUB = 2.0 ** -8, 2.0 ** -24, 2.0 ** -17, 2.0 ** -134, 2.0 ** -125
SUM = 2.0 * F32


def wide(fmt: str, q, s=None, t=None):
    """What operand rows stand for, FP64; t: the FP32 scale of each row, or one for all."""
    if fmt == "bf16":
        return q.double()
    if fmt == "mxfp8":
        v = q.view(torch.float8_e4m3fn).double()
    else:
        pairs = torch.tensor([[E2M1[b % 16], E2M1[b // 16]] for b in range(256)], dtype=torch.float64, device=q.device)
        v = pairs[q.long()].reshape(q.shape[0], -1)
    scale = s.view(torch.float8_e4m3fn).double() if fmt == "nvfp4" else torch.exp2(s.double() - 127.0)
    v = v * scale.repeat_interleave(v.shape[1] // max(s.shape[1], 1), 1)
    return v if t is None else v * t.double().reshape(-1, 1)


def product(a, b):
    """a b^T and the bound of its binary32 sum."""
    return a @ b.T, (SUM * a.shape[-1]) * (a.abs() @ b.abs().T)


def half_step(v):
    return BF16 * v.abs() + TINY


def gated(y, err):
    """(h, its bound, gate_up's bound) of products y = (g | u) that are within err."""
    g, u = y.chunk(2, -1)
    eg, eu = err.chunk(2, -1)
    s = torch.sigmoid(g)
    h = g * s * u
    off = 1.1 * (eg * (u.abs() + eu)) + (g * s).abs() * eu + EVAL * h.abs() + SUB * (g * u).abs()
    return h, (1 + BF16) * off + half_step(h), (1 + BF16) * err + half_step(y)


def through(dh, err, gate_up):
    """((d_gate_up, its bound), (h, its bound)) of dh within err."""
    g, u = gate_up.double().chunk(2, -1)
    s, c = torch.sigmoid(g), torch.sigmoid(-g)
    dg, du, h = dh * u * s * (1 + g * c), dh * g * s, g * s * u
    ds = s * (1 + g.abs() * c)                              # the size of what is added up in the derivative
    sub = SUB * (1 + g.abs())
    eg = u.abs() * ((dh.abs() + err) * (EVAL * ds + sub) + err * ds)
    eu = (dh.abs() + err) * (EVAL * (g * s).abs() + sub) + err * (g * s).abs()
    eh = EVAL * h.abs() + sub * u.abs()
    d, e = torch.cat([dg, du], -1), torch.cat([eg, eu], -1)
    return (d, (1 + BF16) * e + half_step(d)), (h, (1 + BF16) * eh + half_step(h))


def check(got, want, bound, what: str):
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    off = (got - want).abs()
    bad = ~(off <= bound)                                   # NaN is bad
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds; first at {i}: got {got[i].item()!r}, "
                             f"expected {want[i].item()!r} within {bound[i].item():.3e}")
