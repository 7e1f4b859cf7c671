"""How far the angles of the rotary positions are off, against fractions with pi to 60 digits: what the header promises, by the arithmetic
that the table and the kernel use, and the outputs at positions to both ends of 32 bits."""
import math
import os
import re
from fractions import Fraction

import numpy as np
import pytest
import torch

import bit_grouped_expert_top_gb300 as lm
import step_util as su

TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494")
HEADER = os.path.join(os.path.dirname(__file__), "..", "include", "lily_moe.h")
POSITIONS = [0, 1, -1, 2, 7, 4095, -32768, 131071, 1000003, 2 ** 20 + 1, 16777217, -(2 ** 24) - 3, 2 ** 30 + 7, 2 ** 31 - 1, 1 - 2 ** 31, -2 ** 31]
POSITIONS += [int(v) for v in np.random.default_rng(7).integers(-2 ** 31, 2 ** 31, 50)]
SCALINGS = [("none", {}), ("linear", {"factor": 8.0}), ("base", {"factor": 4.0}), ("parts", {"factor": 8.0, "original": 8192.0})]


def promised():
    """Half-turns, and radians for each position and unit of frequency."""
    with open(HEADER) as f:
        s = re.sub(r"\s*\n \*\s*", " ", f.read())
    s = s[s.index("Rotary positions on queries"):s.index("} lily_rope_shape;")]
    fixed = re.search(r"angle[^.]*?2\^-(\d+) half-turns", s)
    grows = re.search(r"\|positions\[n\]\| \* f_i \* 2\^-(\d+) radians", s)
    return 2.0 ** -int(fixed[1]), 2.0 ** -int(grows[1]) if grows else 0.0


@pytest.mark.parametrize("scaling,kw", SCALINGS)
def test_angles_are_off_by_no_more_than_the_header_says(scaling, kw):
    half_turns, each = promised()
    for theta, rot in ((10000.0, 128), (1e6, 64)):
        f = lm.rope_frequencies(rot, theta, scaling, **kw)
        table = lm.make_rope_table(f, "cpu")
        worst = 0.0
        for pos in POSITIONS:
            for x, t in zip(f.tolist(), table.tolist()):
                got = float(np.float32(np.uint32(pos * t % 2 ** 64 >> 32).astype(np.int32))) * 2.0 ** -31   # the kernel's argument
                exact = pos * Fraction(x) / TWO_PI
                off = abs(float((Fraction(got) / 2 - exact + Fraction(1, 2)) % 1 - Fraction(1, 2))) * 2   # half-turns
                assert off <= half_turns + abs(pos) * x * each / math.pi, (pos, x, off)
                worst = max(worst, off)
        assert worst >= half_turns / 8   # and no promise that is far from what it does


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("scaling,kw", SCALINGS)
def test_outputs_at_far_positions(scaling, kw, interleaved):
    D = rot = 128
    f = lm.rope_frequencies(rot, 10000.0, scaling, **kw)
    g = torch.Generator().manual_seed(3)
    x = torch.randn((len(POSITIONS), 2, D), generator=g).to(torch.bfloat16).cuda()
    x[:, 1, ::3] = 0
    out = torch.empty_like(x)
    lm.lily_rope(x, None, torch.tensor(POSITIONS, dtype=torch.int32, device="cuda"), lm.make_rope_table(f), out, interleaved=interleaved, amplitude=1.2)
    turn = [[pos * Fraction(v) / TWO_PI % 1 for v in f.tolist()] for pos in POSITIONS]
    angle = torch.tensor([[2 * math.pi * float(t) for t in row] for row in turn], dtype=torch.float64)
    c, s = 1.2 * angle.cos()[:, None], 1.2 * angle.sin()[:, None]
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x.double().cpu()[..., i], x.double().cpu()[..., j]
    want = torch.empty(x.shape, dtype=torch.float64)
    want[..., i], want[..., j] = a * c - b * s, a * s + b * c
    # radians: the argument pi (2^-25 + 2^-31), sincospif 2 units of 2^-24, the amplitude, two products and a sum 2^-24 each: below 2^-21;
    # the table |pos| f 2^-52
    radians = 2.0 ** -21 + torch.tensor(POSITIONS, dtype=torch.float64).abs()[:, None, None] * f * 2.0 ** -52
    bound = want.abs() * su.U[torch.bfloat16] * 1.001 + su.TINY[torch.bfloat16]
    for part in (i, j):
        bound[..., part] += (a.abs() + b.abs()) * 1.2 * radians
    su.near(out.cpu(), want, bound)
