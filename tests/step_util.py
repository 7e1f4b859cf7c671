"""Plain 64-bit implementations of the operators around the attention and the expert layers, and their error bounds.

u(t) is half a step of a type: a rounding to it is off by at most that, relative to the value."""
import math

import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24, torch.float8_e4m3fn: 2.0 ** -4}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}  # half of the smallest subnormal


def near(got, want, bound, what=""):
    """|got - want| <= bound everywhere; names the worst place."""
    got, want = got.double(), want.double()
    assert got.shape == want.shape
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    over = (got - want).abs() - bound
    at = int(over.argmax())
    assert float(over.max()) <= 0, (f"{what}: at {at} got {float(got.flatten()[at])!r}, want {float(want.flatten()[at])!r}, "
                                    f"bound {float((bound + 0 * want).flatten()[at])!r}")


# ------------------------------------------------------------------ norm
# y in fp32 before its rounding: the squares are summed by fused multiply-adds, at most 64 in a thread, then at most 5 + 7 joins: the mean
# is off by 78 roundings at most with 1/d and eps, its root by half of that, and the root, the reciprocal,
# the three products, the factor's addition and h's own rounding add 7: below 64 roundings.
NORM = 64 * 2.0 ** -24


def norm(x, weight, offset, eps, residual=None):
    h = x.double() + (0 if residual is None else residual.double())
    f = offset if weight is None else weight.double() + offset
    mean = h.square().mean(-1, keepdim=True) + eps
    return h, torch.where(mean > 0, h / mean.sqrt(), 0.0) * f


def check_norm(want, h=None, y=None, y8=None, y8_scale=None):
    hh, yy = want
    if h is not None:
        near(h, hh, hh.abs() * (U[h.dtype] + 2.0 ** -24 + 2.0 ** -30) + TINY[h.dtype], "h")
    if y is not None:
        near(y, yy, yy.abs() * (U[y.dtype] + NORM * 1.01) + TINY[y.dtype], "y")
    if y8 is not None:
        g = yy.unflatten(-1, (-1, 64))
        most = g.abs().amax(-1)
        some = most >= 2.0 ** -100
        near(y8_scale, torch.where(some, most / 448, 0.0), most / 448 * (NORM + 4 * 2.0 ** -24), "y8_scale")
        value = (y8.double().unflatten(-1, (-1, 64)) * y8_scale.double()[..., None])
        # half a step of e4m3, or of its subnormals (2^-9 apart); the scale and its inverse are roundings of their own
        bound = g.abs() * (U[torch.float8_e4m3fn] + 2 * NORM) + (most / 448 * 2.0 ** -10 * 1.01)[..., None]
        near(value, torch.where(some[..., None], g, 0.0), bound, "y8")


# ------------------------------------------------------------------ 4-bit matrix
def matrix_parts(q, scale, bias):
    """Codes [rows][K] and the scales and biases of each channel in fp64."""
    code = torch.stack([q & 15, q >> 4], -1).flatten(-2).double()
    return code, scale.double().repeat_interleave(64, -1), bias.double().repeat_interleave(64, -1)


def matvec(q, scale, bias, x, x_scale=None):
    """Result in fp64 and its error bound before the output's rounding."""
    code, s, b = matrix_parts(q, scale, bias)
    x = x.double() if x_scale is None else x.double() * x_scale.double().repeat_interleave(64, -1)
    want = x @ (code * s + b).T
    # every product and sum on the way is at most this much, in magnitudes
    most = x.abs() @ (code * s.abs() + b.abs()).T
    # roundings on one path: 4 mma of 17 terms (an mma may cut what it adds, so 2 each), x's sum (18), factors and
    # scale (5), 2 a group, the join of 64 at most, and the last factor
    rounds = 4 * 17 * 2 + 18 + 5 + 2 * (x.shape[1] // 64) + 64 + 1
    error = most * rounds * 2.0 ** -24
    if x_scale is None:
        # x as fp16 times a power of two that brings the largest of 256 channels into [2^14, 2^15), odd channels over 16: what is not a
        # multiple of fp16's 2^-24 after that is off by at most 16 * 2^-25, 2^-35 of the largest
        pad = -x.shape[1] % 256
        largest = torch.nn.functional.pad(x.abs(), (0, pad)).unflatten(-1, (-1, 256)).amax(-1).repeat_interleave(256, -1)[:, :x.shape[1]]
        error = error + (2.0 ** -35 * largest) @ (code * s.abs()).T
    return want, error


def make_matrix(rows, K, seed=0, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 256, (rows, K // 2), generator=g, dtype=torch.uint8)
    scale = (0.01 + 0.01 * torch.rand((rows, K // 64), generator=g)).to(torch.bfloat16)
    bias = (-7.5 * scale.float() + 0.02 * torch.randn((rows, K // 64), generator=g)).to(torch.bfloat16)
    return q.to(device), scale.to(device), bias.to(device)


# ------------------------------------------------------------------ rotary positions
def frequencies(rot, theta=10000.0, scaling="none", factor=1.0, original=0.0, low=1.0, high=32.0):
    out = []
    for i in range(rot // 2):
        f = (theta * factor ** (rot / (rot - 2)) if scaling == "base" and rot > 2 else theta) ** (-2 * i / rot)
        if scaling == "linear":
            f /= factor
        if scaling == "parts":
            turns = original * f / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - low) / (high - low)))
            f = f * keep + f * (1 - keep) / factor
        out.append(f)
    return torch.tensor(out, dtype=torch.float64)


def rope(x, positions, f, interleaved, amplitude=1.0):
    """Result in fp64 and the bound: the output's rounding, and fp32 sines and cosines off by at most 2^-22 (an angle
    off by pi 2^-31, sincospif's own 2 units of 2^-24, the amplitude, two products and a sum)."""
    x = x.double().cpu()
    out, n = x.clone(), 2 * len(f)
    # the angle modulo a turn, in whole numbers: exact for the table's entries
    turn = [round(float(v) / (2 * math.pi) * 2 ** 64) for v in f]
    angle = torch.tensor([[int(p) * t % 2 ** 64 / 2 ** 63 * math.pi for t in turn] for p in positions.tolist()], dtype=torch.float64)
    c, s = (angle.cos() * amplitude)[:, None], (angle.sin() * amplitude)[:, None]
    i, j = (slice(0, n, 2), slice(1, n, 2)) if interleaved else (slice(0, n // 2), slice(n // 2, n))
    a, b = x[..., i], x[..., j]
    out[..., i], out[..., j] = a * c - b * s, a * s + b * c
    bound = out.abs() * U[torch.bfloat16] * 1.001 + TINY[torch.bfloat16]
    bound[..., n:] = 0
    extra = (a.abs() + b.abs()) * abs(amplitude) * 2.0 ** -21
    bound[..., i] += extra
    bound[..., j] += extra
    return out, bound


# ------------------------------------------------------------------ drafts
def units(p):
    """p in units of 2^-62, rounded down, as Python integers."""
    return [int(math.ldexp(_clamped(v), 62)) for v in p]


def _clamped(v):
    return min(max(float(v), 0.0), 1.0) if v == v else 0.0


def verify(p, q, drafts, cu, u, r):
    """accepted and tokens by whole numbers (numpy fp32 and int arrays)."""
    accepted, tokens = [], []
    V = p.shape[1]
    for b in range(len(r)):
        c0, m = int(cu[b]), int(cu[b + 1] - cu[b])
        n = 0
        while n < m:
            x = int(drafts[c0 + n])
            if not 0 <= x < V:
                break
            qx = 1.0 if q is None else _clamped(q[c0 + n, x])
            if not float(u[c0 + n]) * qx < _clamped(p[c0 + b + n, x]):
                break
            n += 1
        whole = units(p[c0 + b + n])
        w = list(whole)
        if n < m:
            if q is None:
                if 0 <= drafts[c0 + n] < V:
                    w[int(drafts[c0 + n])] = 0
            else:
                w = [max(a - c, 0) for a, c in zip(w, units(q[c0 + n]))]
            if not any(w):
                w = whole
        below, token, upto = sum(w) * int(math.ldexp(float(r[b]), 64)) >> 64, -1, 0
        for v, a in enumerate(w):
            upto += a
            if upto > below:
                token = v
                break
        accepted.append(n)
        tokens += [int(t) for t in drafts[c0:c0 + n]] + [token] + [-1] * (m - n)
    return np.array(accepted, np.int32), np.array(tokens, np.int32)
