"""Products of e4m3 tokens over the range of their scales: all that the norm gives, up to the largest fp32 number over 448."""
import pytest
import torch

import bit_grouped_expert_top_gb300 as lm
import step_util as su

pytestmark = pytest.mark.gpu
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
LARGEST = torch.finfo(F32).max / 448


def _matrix(rows, K, by, seed):
    q, s, b = su.make_matrix(rows, K, seed=seed)
    return q, s * by, b * by


def _check(parts, y8, scale, what):
    for out_type in (F32, BF):
        out = torch.empty((len(y8), len(parts[0])), dtype=out_type, device="cuda")
        lm.lily_q4_matvec(lm.make_q4(*parts), y8, out, x_scale=scale)
        want, bound = su.matvec(*parts, y8, scale)
        su.near(out, want, bound + (want.abs() + bound) * su.U[out_type] + su.TINY[out_type], what)


@pytest.mark.parametrize("T,K", [(1, 256), (5, 2048), (12, 320), (20, 2112), (32, 4096)])
@pytest.mark.parametrize("by", [2.0 ** -90, 2.0 ** -40, 2.0 ** 60, 2.0 ** 100, 2.0 ** 109, 2.0 ** 110, 2.0 ** 112, 2.0 ** 118, LARGEST / 2])
def test_scales(T, K, by):
    g = torch.Generator().manual_seed(T)
    y8 = (100 * torch.randn((T, K), generator=g)).clamp(-448, 448).to(F8).cuda()
    scale = (by * (1 + torch.rand((T, K // 64), generator=g).double())).clamp(max=LARGEST).to(F32).cuda()
    _check(_matrix(70, K, 2.0 ** -50 if by > 1 else 2.0 ** 20, T), y8, scale, f"scales of {by!r}")


@pytest.mark.parametrize("T", [3, 30])
def test_scales_of_very_different_size_in_a_token(T):
    g = torch.Generator().manual_seed(T)
    y8 = (100 * torch.randn((T, 512), generator=g)).clamp(-448, 448).to(F8).cuda()
    scale = torch.full((T, 8), 2.0 ** -30, device="cuda")
    scale[:, 2], scale[1, 5], scale[2, 0] = 2.0 ** 30, 2.0 ** 115, LARGEST
    _check(_matrix(40, 512, 2.0 ** -30, T), y8, scale, "mixed")


@pytest.mark.parametrize("d", [256, 2048])
def test_what_the_norm_gives_for_the_largest_weights(d):
    """A norm whose weights bring y next to the largest fp32 number, and the product of its codes."""
    g = torch.Generator().manual_seed(d)
    x = torch.randn((4, d), generator=g).clamp(-3, 3).cuda()
    weight = torch.full((d,), 2.0 ** 125, device="cuda")
    y8, scale = torch.empty((4, d), dtype=F8, device="cuda"), torch.empty((4, d // 64), device="cuda")
    lm.lily_rms_norm(x, weight, y8=y8, y8_scale=scale)
    assert bool((scale > 2.0 ** 116).all()) and bool(torch.isfinite(scale).all())
    _check(_matrix(50, d, 2.0 ** -60, d), y8, scale, "norm")
