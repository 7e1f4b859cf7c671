"""Norms of rows that are not finite, and the kernel's forms of many rows of up to 512 channels: several rows a warp, four vectors a
thread of which the last are missing."""
import pytest
import torch

import bit_grouped_expert_top_gb300 as lm
import step_util as su

pytestmark = pytest.mark.gpu
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
NAN, INF = float("nan"), float("inf")


def _rand(*size, seed=0, dtype=BF, by=1.0):
    g = torch.Generator().manual_seed(seed + sum(s * 31 ** i for i, s in enumerate(size)))
    return (torch.randn(size, generator=g) * by).to(dtype).cuda()


def _norm(x, weight=None, offset=1.0, eps=1e-6, residual=None):
    codes = x.shape[-1] % 64 == 0
    o = {"y": torch.empty(x.shape, dtype=BF, device="cuda")}
    if codes:
        o["y8"] = torch.empty(x.shape, dtype=F8, device="cuda")
        o["y8_scale"] = torch.empty(x.shape[:-1] + (x.shape[-1] // 64,), device="cuda")
    if residual is not None:
        o["h"] = torch.empty_like(residual)
    lm.lily_rms_norm(x, weight, residual=residual, eps=eps, weight_offset=offset, **o)
    torch.cuda.synchronize()
    return o


# (rows, channels): a row of several CTA forms, alone in its warp and among others of it
FORMS = [(9, 8), (9, 64), (9, 256), (9, 1000), (2049, 128), (2049, 256), (2049, 448), (2049, 512), (9, 2048), (9, 4096), (9, 8192), (9, 16384)]


@pytest.mark.parametrize("N,d", FORMS)
@pytest.mark.parametrize("eps", [1e-6, 0.0])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_row_with_a_nan_is_nan_throughout(N, d, eps, dtype):
    x, w = _rand(N, d, dtype=dtype), _rand(d, by=0.3)
    clean = _norm(x, w, eps=eps)
    bad = [1, 4, 6]
    for i, n in enumerate(bad):
        x[n, (i * 37 + 5) % d] = NAN
    x[6, 0] = INF  # beside an infinity as well
    o = _norm(x, w, eps=eps)
    assert bool(torch.isnan(o["y"][bad]).all())
    if "y8" in o:
        assert bool(torch.isnan(o["y8"].float()[bad]).all()) and float(o["y8_scale"][bad].abs().max()) == 0
    keep = [n for n in range(N) if n not in bad]
    for n in o:
        assert torch.equal(o[n][keep].view(torch.uint8), clean[n][keep].view(torch.uint8)), n


@pytest.mark.parametrize("N,d", FORMS)
def test_a_nan_that_the_residual_brings(N, d):
    x, r = _rand(N, d, dtype=F32), _rand(N, d, seed=2)
    r[3, d - 1] = NAN
    o = _norm(x, None, residual=r)
    assert bool(torch.isnan(o["y"][3]).all()) and int(torch.isnan(o["h"][3]).sum()) == 1
    assert bool(torch.isfinite(o["y"][[0, 1, 2, 4, 5]].float()).all())


@pytest.mark.parametrize("N,d", FORMS)
def test_a_row_with_an_infinity(N, d):
    """The formula's limit: zeros, and NaN (infinity times zero) where the infinities are."""
    x = _rand(N, d, dtype=F32)
    x[2, 1], x[2, d // 2] = INF, -INF
    o = _norm(x, _rand(d, by=0.3))
    row = o["y"][2].float()
    at = torch.isinf(x[2])
    assert bool(torch.isnan(row[at]).all()) and float(row[~at].abs().max()) == 0
    if "y8" in o:
        row = o["y8"][2].float()
        assert bool(torch.isnan(row[at]).all()) and float(row[~at].abs().max()) == 0 and float(o["y8_scale"][2].abs().max()) == 0


@pytest.mark.parametrize("N", [2048, 2049, 5003])
@pytest.mark.parametrize("d", [72, 128, 136, 200, 256, 264, 320, 448, 504, 512, 520, 1000])
def test_many_rows_of_few_channels(N, d):
    w = _rand(d, by=0.3)
    for x, kw in ((_rand(N, d), {"weight": w}), (_rand(N, d, dtype=F32), {"weight": w.float(), "offset": 0.0, "residual": _rand(N, d, seed=1)})):
        o = _norm(x, **kw)
        su.check_norm(su.norm(x, kw["weight"], kw.get("offset", 1.0), 1e-6, kw.get("residual")), **o)


@pytest.mark.parametrize("d", [128, 256, 320, 512])
@pytest.mark.parametrize("by", [2.0 ** 100, 2.0 ** 66, 2.0 ** -70, 2.0 ** -120])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
def test_many_rows_whose_squares_leave_fp32(d, by, eps):
    """Rows of ordinary size between them, in the same warp."""
    x = _rand(2051, d, dtype=F32)
    x[::3] *= by
    x[7], x[11] = 0, 0
    o = _norm(x, _rand(d, by=0.3), eps=eps)
    su.check_norm(su.norm(x, _rand(d, by=0.3), 1.0, eps), **o)


@pytest.mark.parametrize("N,H,d,pad", [(1025, 2, 448, 16), (300, 16, 320, 64), (4099, 1, 512, 8)])
def test_many_strided_heads(N, H, d, pad):
    x = _rand(N, H * d + pad)[:, :H * d].unflatten(-1, (H, d))
    o = _norm(x, _rand(d, by=0.2))
    su.check_norm(su.norm(x, _rand(d, by=0.2), 1.0, 1e-6), **o)
