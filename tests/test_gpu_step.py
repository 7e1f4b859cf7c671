"""The operators around the attention and the expert layers against plain 64-bit implementations (tests/step_util.py): norms, 4-bit
matrix-vector products, rotary positions and the verification of drafts, at the sizes and values where each can go
wrong, on side streams and in captured graphs."""
import numpy as np
import pytest
import torch

import bit_grouped_expert_top_gb300 as lm
import step_util as su

pytestmark = pytest.mark.gpu
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _rand(*size, seed=0, dtype=BF, by=1.0):
    g = torch.Generator().manual_seed(seed + sum(s * 31 ** i for i, s in enumerate(size)))
    return (torch.randn(size, generator=g) * by).to(dtype).cuda()


def _guarded(shape, dtype):
    """A tensor with 64 bytes-worth of rows of a known pattern behind it, and a check that they are still there."""
    n = int(np.prod(shape))
    size = torch.empty(0, dtype=dtype).element_size()
    raw = torch.full((n * size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    return raw[:n * size].view(dtype).view(shape), lambda: bool((raw[n * size:] == 0xA5).all())


# ------------------------------------------------------------------ norm
def _norm(x, weight=None, offset=0.0, eps=1e-6, residual=None, y=True, codes=False):
    want = su.norm(x, weight, offset, eps, residual)
    lead = x.shape[:-1]
    outs, guards = {}, []
    for name, on, shape, dtype in (("y", y, x.shape, BF), ("y8", codes, x.shape, F8), ("y8_scale", codes, lead + (x.shape[-1] // 64,), F32),
                                   ("h", residual is not None, x.shape, residual.dtype if residual is not None else None)):
        if on:
            outs[name], g = _guarded(shape, dtype)
            guards.append(g)
    lm.lily_rms_norm(x, weight, residual=residual, eps=eps, weight_offset=offset, **outs)
    torch.cuda.synchronize()
    assert all(g() for g in guards)
    su.check_norm(want, **outs)
    return outs


@pytest.mark.parametrize("d", [8, 16, 56, 64, 72, 128, 256, 264, 1000, 2048, 2056, 4096, 4104, 8192, 8200, 16384])
@pytest.mark.parametrize("N", [1, 3, 33])
def test_norm_sizes(N, d):
    w = _rand(d, by=0.3)
    _norm(_rand(N, d), w, 1.0)
    _norm(_rand(N, d, dtype=F32), w.float(), 0.0, residual=_rand(N, d, seed=1), codes=d % 64 == 0)


@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("ht", [None, BF, F32])
@pytest.mark.parametrize("wt", [None, BF, F32])
@pytest.mark.parametrize("y,codes", [(True, False), (False, True), (True, True)])
def test_norm_types(xt, ht, wt, y, codes):
    for N, d in ((5, 128), (7, 2048), (600, 64), (301, 2048)):
        _norm(_rand(N, d, dtype=xt), None if wt is None else _rand(d, dtype=wt, by=0.3), 1.0,
              residual=None if ht is None else _rand(N, d, dtype=ht, seed=2, by=3.0), y=y, codes=codes)


@pytest.mark.parametrize("N,H,d,pad", [(1, 16, 256, 8), (7, 3, 64, 40), (2049, 2, 128, 512), (130, 5, 72, 0), (4, 2, 2048, 16)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_of_heads_in_a_fused_projection(N, H, d, pad, dtype):
    x = _rand(N, H * d + pad, dtype=dtype)[:, pad // 16 * 8:][:, :H * d].unflatten(-1, (H, d))
    _norm(x, _rand(d, by=0.2), 1.0, codes=d % 64 == 0)


def test_norm_of_many_rows():
    for N, d in ((8192, 2048), (5000, 4096), (20000, 256), (70001, 64), (3001, 16384)):
        _norm(_rand(N, d), _rand(d), residual=_rand(N, d, seed=4, dtype=F32), codes=True)


@pytest.mark.parametrize("d", [64, 256, 2048, 4096])
@pytest.mark.parametrize("by", [2.0 ** 100, 2.0 ** 66, 2.0 ** -70, 2.0 ** -100, 2.0 ** -120])
@pytest.mark.parametrize("eps", [1e-6, 1e-30, 0.0])
def test_norm_of_values_whose_squares_leave_fp32(d, by, eps):
    # rows of ordinary size between them, in the same warp
    x = _rand(9, d, dtype=F32)
    x[::2] *= by
    _norm(x, _rand(d), 1.0, eps=eps, codes=True)
    _norm(x.to(BF), _rand(d), 1.0, eps=eps)


def test_norm_of_the_largest_values():
    x = torch.full((3, 2048), 3e38, device="cuda")
    x[1, ::2] = 1e-3
    x[2] = 0
    x[2, 5] = -3.3e38
    _norm(x, None, 1.0, codes=True)


@pytest.mark.parametrize("eps", [1e-6, 0.0])
def test_norm_of_zeros(eps):
    x = _rand(6, 256)
    x[1], x[4] = 0, 0
    out = _norm(x, _rand(256), 1.0, eps=eps, codes=True)
    assert float(out["y"][1].abs().max()) == 0 and float(out["y8_scale"][4].abs().max()) == 0
    w = _rand(256)
    w[64:128] = 0  # a group of zeros in rows of ordinary values
    out = _norm(_rand(6, 256), w, codes=True)
    assert float(out["y8_scale"][:, 1].abs().max()) == 0 and float(out["y8"][:, 64:128].float().abs().max()) == 0


def test_norm_rows_do_not_touch_each_other():
    for d in (64, 256, 2048):
        x = _rand(9, d)
        clean = torch.empty_like(x)
        lm.lily_rms_norm(x, None, y=clean, weight_offset=1.0)
        x[4, 3], x[7, 0] = float("nan"), float("inf")
        y = torch.empty_like(x)
        lm.lily_rms_norm(x, None, y=y, weight_offset=1.0)
        keep = [0, 1, 2, 3, 5, 6, 8]
        assert torch.equal(y[keep], clean[keep])


def test_norm_in_place_residual():
    for d in (64, 2048, 16384):
        x, r = _rand(17, d, dtype=F32), _rand(17, d, seed=3)
        want = su.norm(x, None, 1.0, 1e-6, r)
        y = torch.empty(17, d, dtype=BF, device="cuda")
        lm.lily_rms_norm(x, None, y=y, residual=r, h=r, weight_offset=1.0)
        su.check_norm(want, h=r, y=y)


def test_norm_refusals_of_the_binding():
    x, w = _rand(4, 256), _rand(256)
    y8, sc = torch.empty(4, 256, dtype=F8, device="cuda"), torch.empty(4, 4, device="cuda")
    y = torch.empty_like(x)
    bad = [(dict(), "expected y"), (dict(y=y[:3]), "y: expected"), (dict(y=y.float()), "y: expected"), (dict(y=y.t().contiguous().t()), "y: expected"),
           (dict(y8=y8), "go together"), (dict(y8=y8, y8_scale=sc[:, :3]), "y8_scale"), (dict(y=y, weight=w[:128]), "weight"),
           (dict(y=y, weight=w.half()), "weight"), (dict(y=y, residual=x), "go together"), (dict(y=y, residual=x, h=y.float()), "h: expected"),
           (dict(y=y, x=x.t().contiguous().t()), "contiguous"), (dict(y=y, weight=w.cpu()), "CUDA tensor")]
    for kw, match in bad:
        with pytest.raises(ValueError, match=match):
            lm.lily_rms_norm(**{"x": x, "weight": w, **kw})
    with pytest.raises(ValueError, match="groups of 64"):
        lm.lily_rms_norm(x[:, :72].contiguous(), None, y8=y8[:, :72].contiguous(), y8_scale=sc)
    with pytest.raises(lm.LilyError, match="-3"):
        lm.lily_rms_norm(_rand(4, 264)[:, 4:260], w, y=y)
    with pytest.raises(lm.LilyError, match="-1"):
        lm.lily_rms_norm(x, w, y=y, eps=-1.0)
    for N in (0, 1):
        lm.lily_rms_norm(x[:N], w, y=y[:N])


# ------------------------------------------------------------------ 4-bit matrix
def _codes(x):
    """x in the form of the norm's 8-bit output."""
    y8, sc = torch.empty(x.shape, dtype=F8, device="cuda"), torch.empty(x.shape[0], x.shape[1] // 64, device="cuda")
    lm.lily_rms_norm(x, None, y8=y8, y8_scale=sc, weight_offset=1.0)
    return y8, sc


def _matvec(parts, x, out_type, x_scale=None, what=""):
    w = lm.make_q4(*parts)
    out, guard = _guarded((x.shape[0], w.rows), out_type)
    lm.lily_q4_matvec(w, x, out, x_scale=x_scale)
    torch.cuda.synchronize()
    assert guard()
    want, bound = su.matvec(*parts, x, x_scale)
    su.near(out, want, bound + (want.abs() + bound) * su.U[out_type] + su.TINY[out_type], what)
    return out


@pytest.mark.parametrize("T", list(range(1, 33)))
def test_matvec_tokens(T):
    parts = su.make_matrix(100, 512)
    x = _rand(T, 512)
    _matvec(parts, x, F32)
    _matvec(parts, *[_codes(x)[0], BF], _codes(x)[1])


@pytest.mark.parametrize("K", [64, 128, 192, 256, 320, 512, 576, 1024, 2048, 2112, 4096, 4160, 8192, 8256, 8448, 16320, 16384])
@pytest.mark.parametrize("T", [1, 9, 17, 32])
def test_matvec_columns(K, T):
    parts = su.make_matrix(67, K, seed=K)
    x = _rand(T, K) * _rand(1, K, seed=5, dtype=F32).exp().to(BF)
    _matvec(parts, x, F32)
    y8, sc = _codes(x)
    _matvec(parts, y8, BF, sc)


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 33, 127, 129, 255, 1000, 4099, 20001])
@pytest.mark.parametrize("T,K", [(1, 2048), (8, 256), (16, 64), (32, 2048), (20, 192)])
def test_matvec_rows(rows, T, K):
    _matvec(su.make_matrix(rows, K, seed=rows), _rand(T, K), F32 if rows % 2 else BF)


@pytest.mark.parametrize("T", [1, 8, 32])
def test_matvec_large(T):
    parts = [t.repeat(8, 1) for t in su.make_matrix(16251, 2048, seed=3)]
    out = _matvec(parts, _rand(T, 2048), F32)
    first = out[:, :16251]
    assert all(torch.equal(first, out[:, i * 16251:(i + 1) * 16251]) for i in range(1, 8))


@pytest.mark.parametrize("K,rows", [(2048, 9720), (2048, 9729), (1984, 9728), (1984, 9731), (320, 38912), (320, 38997), (64, 77811), (64, 77824),
                                    (2112, 2431), (2112, 2435), (4096, 2433), (8256, 2500),
                                    (2048, 4870), (1984, 19456), (2048, 19457), (1984, 19500), (192, 77830), (4096, 4870), (4160, 5003)])
@pytest.mark.parametrize("T", [1, 8, 16, 24])
def test_matvec_around_the_steps_of_a_block(K, rows, T):
    """Rows where a block has few steps, or more, of either size."""
    parts = su.make_matrix(rows, K, seed=rows)
    x = _rand(T, K)
    _matvec(parts, x, F32)
    y8, sc = _codes(x)
    _matvec(parts, y8, BF, sc)


def test_matvec_strided_tokens():
    parts = su.make_matrix(130, 512)
    x = _rand(6, 2048)[:, 512:1024]
    _matvec(parts, x, F32)
    _matvec(parts, x[::2], F32)
    y8, sc = _codes(_rand(6, 2048))
    _matvec(parts, y8[:, 1024:1536], F32, sc[:, 16:24].contiguous())


@pytest.mark.parametrize("by", [2.0 ** 60, 2.0 ** -60, 2.0 ** -88])
def test_matvec_tokens_of_very_different_size(by):
    parts = su.make_matrix(80, 512, seed=4)
    x = _rand(5, 512)
    x[1] *= by
    x[3, 64:128] *= by            # a group of its own size
    x[4, 5::64] *= 2.0 ** -20     # channels far below the rest of their group
    x[4, 7::64] *= 2.0 ** 20
    _matvec(parts, x, F32)


def test_matvec_extreme_parameters():
    q, s, b = su.make_matrix(64, 256, seed=6)
    s[3], b[3] = 0, 1.0            # constant rows
    s[5], b[5] = -s[5], 0.0        # falling ones
    s[7], b[7] = 2.0 ** 40, -2.0 ** 43
    s[9], b[9] = 2.0 ** -40, 2.0 ** -38
    q[11] = 0
    q[12] = 0xFF
    _matvec((q, s, b), _rand(3, 256), F32)
    x = torch.zeros(3, 256, dtype=BF, device="cuda")
    x[1, 100] = 1.0
    out = _matvec((q, s, b), x, F32)
    assert float(out[0].abs().max()) == 0


def test_matvec_each_code_in_each_place():
    """One token that is 1 in one channel picks a column out: every channel, every code."""
    K = 256
    q = torch.stack([torch.full((K // 2,), (c & 15) | (15 - c & 15) << 4, dtype=torch.uint8) for c in range(16)]).cuda()
    s = torch.ones((16, K // 64), dtype=BF, device="cuda")
    b = torch.zeros_like(s)
    w = lm.make_q4(q, s, b)
    for k0 in range(0, K, 32):
        x = torch.zeros(32, K, dtype=BF, device="cuda")
        x[torch.arange(32), k0 + torch.arange(32)] = 1.0
        out = torch.empty(32, 16, device="cuda")
        lm.lily_q4_matvec(w, x, out)
        c = torch.arange(16.0, device="cuda")
        assert torch.equal(out[0::2], c.expand(16, 16)) and torch.equal(out[1::2], (15 - c).expand(16, 16))


def test_matvec_tokens_do_not_touch_each_other():
    for T in (7, 16, 31):
        parts = su.make_matrix(50, 512, seed=7)
        w, x = lm.make_q4(*parts), _rand(T, 512)
        clean, out = (torch.empty(T, 50, device="cuda") for _ in range(2))
        lm.lily_q4_matvec(w, x, clean)
        x[2, 100], x[5, 3] = float("nan"), float("-inf")
        lm.lily_q4_matvec(w, x, out)
        keep = [t for t in range(T) if t not in (2, 5)]
        assert torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("K", [256, 320, 64 * 19])
def test_matvec_rows_do_not_touch_each_other(K):
    """Parameters that are not finite: a row's own output alone, also where rows share words of them."""
    q, s, b = su.make_matrix(40, K, seed=8)
    x, clean, out = _rand(3, K), torch.empty(3, 40, device="cuda"), torch.empty(3, 40, device="cuda")
    lm.lily_q4_matvec(lm.make_q4(q, s, b), x, clean)
    s, b = s.clone(), b.clone()
    s[7], b[18], s[19, 0], b[39, -1] = float("nan"), float("inf"), float("inf"), float("nan")
    lm.lily_q4_matvec(lm.make_q4(q, s, b), x, out)
    keep = [n for n in range(40) if n not in (7, 18, 19, 39)]
    assert torch.equal(out[:, keep], clean[:, keep]) and not bool(torch.isfinite(out[:, [7, 18, 19, 39]]).any())


def test_offsets_beyond_32_bits():
    """Arrays of more than 2^32 bytes: the last rows, tokens and probabilities."""
    rows, K = 540001, 16384       # 4.4 GB of codes
    part = su.make_matrix(65, K, seed=9)
    q = torch.zeros((rows, K // 2), dtype=torch.uint8, device="cuda")
    s, b = (torch.zeros((rows, K // 64), dtype=BF, device="cuda") for _ in "sb")
    q[-65:], s[-65:], b[-65:] = part
    for T in (3, 20):
        x, out, small = _rand(T, K), torch.empty(T, rows, device="cuda"), torch.empty(T, 65, device="cuda")
        lm.lily_q4_matvec(lm.make_q4(q, s, b), x, out)
        lm.lily_q4_matvec(lm.make_q4(*part), x, small)
        want, bound = su.matvec(*part, x)
        su.near(out[:, -65:], want, bound * 2 + want.abs() * 2.0 ** -20)
        su.near(small, want, bound * 2 + want.abs() * 2.0 ** -20)
        assert float(out[:, :-65].abs().max()) == 0
    del q, s, b, out
    N, d = 270001, 8192           # 4.4 GB of bf16
    x = torch.zeros(N, d, dtype=BF, device="cuda")
    x[-3:] = _rand(3, d)
    y = torch.empty_like(x)
    lm.lily_rms_norm(x, None, y=y, weight_offset=1.0)
    su.check_norm(su.norm(x[-3:], None, 1.0, 1e-6), y=y[-3:])
    assert float(y[:-3].abs().max()) == 0
    # the same memory as heads of 64 channels
    heads, pos = x.view(N, d // 64, 64), torch.arange(N, dtype=torch.int32, device="cuda")
    f = lm.rope_frequencies(64)
    before = heads[-3:].clone()
    lm.lily_rope(heads, None, pos, lm.make_rope_table(f))
    su.near(heads[-3:].cpu(), *su.rope(before, pos[-3:], f, False))
    del x, y, heads
    V = 1 << 20                   # rows 4.8 GB apart
    p, _, drafts, cu, u, r = _case([1], V, seed=4)
    far = torch.zeros(1200000000 + V, device="cuda").as_strided((2, V), (1200000000, 1))
    far.copy_(p.cuda())
    acc, tok, ws = torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda"), lm.alloc_draft_workspace()
    for v in (0.0, 0.999999):
        u[0] = v
        lm.lily_draft_verify(far, None, drafts.cuda(), cu.cuda(), u.cuda(), r.cuda(), acc, tok, ws)
        want = su.verify(p.numpy(), None, drafts.numpy(), cu.numpy(), u.numpy(), r.numpy())
        assert np.array_equal(acc.cpu().numpy(), want[0]) and np.array_equal(tok.cpu().numpy(), want[1])


def test_matvec_refusals_of_the_binding():
    parts = su.make_matrix(64, 256)
    w, x, out = lm.make_q4(*parts), _rand(4, 256), torch.empty(4, 64, device="cuda")
    sc = torch.ones(4, 4, device="cuda")
    for kw, match in [(dict(x=x[:, :128]), "x: expected"), (dict(x_scale=sc), "x_scale"), (dict(x=x.to(F8)), "x_scale"),
                      (dict(x=x.to(F8), x_scale=sc[:3]), "x_scale"), (dict(out=out[:3]), "out: expected"), (dict(out=out.half()), "out: expected"),
                      (dict(out=torch.empty(64, 4, device="cuda").t()), "out: expected"), (dict(x=_rand(256, 4).t()), "contiguous")]:
        with pytest.raises(ValueError, match=match):
            lm.lily_q4_matvec(**{"w": w, "x": x, "out": out, **kw})
    with pytest.raises(lm.LilyError, match="-2"):
        lm.lily_q4_matvec(w, _rand(33, 256), torch.empty(33, 64, device="cuda"))
    with pytest.raises(ValueError, match="scale"):
        lm.make_q4(parts[0], parts[1][:, :3], parts[2])
    with pytest.raises(ValueError, match="contiguous"):
        lm.make_q4(parts[0][:, :64], parts[1][:, :2], parts[2][:, :2])
    lm.lily_q4_matvec(w, x[:0], out[:0])


# ------------------------------------------------------------------ rotary positions
def _rope(N, H_q, H_k, D, rot, interleaved, far=1000, scaling="none", kw={}, amplitude=1.0, positions=None, seed=0):
    fused = _rand(N, (H_q + 2 * H_k) * D + 16, seed=seed)
    q = fused[:, :H_q * D].unflatten(-1, (H_q, D))
    k = fused[:, H_q * D:(H_q + H_k) * D].unflatten(-1, (H_k, D)) if H_k else None
    if positions is None:
        positions = torch.randint(0, far, (N,), generator=torch.Generator().manual_seed(N)).to(torch.int32)
    positions = positions.cuda()
    f = lm.rope_frequencies(rot, 10000.0, scaling, **kw)
    table = lm.make_rope_table(f)
    wants = [None if x is None else su.rope(x, positions, f, interleaved, amplitude) for x in (q, k)]
    outs = [(None, None) if x is None else _guarded(x.shape, BF) for x in (q, k)]
    lm.lily_rope(q, k, positions, table, outs[0][0], outs[1][0], interleaved=interleaved, amplitude=amplitude)
    # in place, in the strided slices
    lm.lily_rope(q, k, positions, table, interleaved=interleaved, amplitude=amplitude)
    for x, want, (out, guard) in zip((q, k), wants, outs):
        if x is not None:
            su.near(out.cpu(), *want)
            assert guard() and torch.equal(out, x)
    assert torch.equal(fused[:, (H_q + H_k) * D:], _rand(N, (H_q + 2 * H_k) * D + 16, seed=seed)[:, (H_q + H_k) * D:])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(16, 16), (64, 16), (64, 64), (128, 32), (128, 128), (128, 112), (256, 64), (256, 240), (80, 48), (512, 256)])
@pytest.mark.parametrize("N,H_q,H_k", [(1, 16, 2), (5, 1, 1), (37, 6, 3), (3, 4, 0)])
def test_rope_shapes(N, H_q, H_k, D, rot, interleaved):
    _rope(N, H_q, H_k, D, rot, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_many_tokens(interleaved):
    _rope(1500, 16, 2, 256, 64, interleaved)
    _rope(2001, 8, 8, 128, 128, interleaved)
    _rope(700, 5, 1, 64, 32, interleaved)


@pytest.mark.parametrize("scaling,kw", [("linear", {"factor": 8.0}), ("base", {"factor": 4.0}), ("parts", {"factor": 8.0, "original": 8192.0})])
def test_rope_scaled(scaling, kw):
    _rope(50, 4, 2, 128, 128, False, far=60000, scaling=scaling, kw=kw, amplitude=1.2)
    _rope(50, 4, 2, 128, 64, True, far=60000, scaling=scaling, kw=kw, amplitude=-0.5)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_far_and_negative_positions(interleaved):
    edge = torch.tensor([0, 1, -1, 2 ** 20, 2 ** 20 + 1, 2 ** 30 + 7, 2 ** 31 - 1, -2 ** 31, -12345, 16777217], dtype=torch.int32)
    _rope(len(edge), 2, 1, 128, 128, interleaved, positions=edge)


def test_rope_turns_back():
    x = _rand(64, 4, 128)
    table = lm.make_rope_table(lm.rope_frequencies(128))
    pos = torch.arange(64, dtype=torch.int32, device="cuda") * 1000
    there, back = torch.empty_like(x), torch.empty_like(x)
    lm.lily_rope(x, None, pos, table, there)
    lm.lily_rope(there, None, -pos, table, back)
    # two roundings of each of a pair's channels
    size = (x.double().unflatten(-1, (2, 64)) ** 2).sum(-2, keepdim=True).sqrt().expand(-1, -1, 2, -1).flatten(-2)
    su.near(back, x, size * 3 * 2.0 ** -8)


def test_rope_refusals_of_the_binding():
    q, k, pos = _rand(4, 2, 64), _rand(4, 1, 64), torch.zeros(4, dtype=torch.int32, device="cuda")
    table = lm.make_rope_table(lm.rope_frequencies(64))
    for kw, match in [(dict(q=q.float()), "q: expected"), (dict(q=q.transpose(0, 1)), "contiguous"), (dict(positions=pos[:3]), "positions"),
                      (dict(positions=pos.long()), "positions"), (dict(table=table.to(torch.int32)), "table"), (dict(k=k[:3]), "k: "),
                      (dict(q_out=q[:, :1]), "q_out"), (dict(k_out=k.float()), "k_out"), (dict(k=None, k_out=k), "together"), (dict(k=k.cpu()), "CUDA tensor")]:
        with pytest.raises(ValueError, match=match):
            lm.lily_rope(**{"q": q, "k": k, "positions": pos, "table": table, **kw})
    with pytest.raises(lm.LilyError, match="-1"):
        lm.lily_rope(q, k, pos, lm.make_rope_table(lm.rope_frequencies(128)))
    with pytest.raises(lm.LilyError, match="-2"):
        lm.lily_rope(q, k, pos, lm.make_rope_table(lm.rope_frequencies(24)))
    lm.lily_rope(q[:0], k[:0], pos[:0], table)


# ------------------------------------------------------------------ drafts
def _distributions(n, V, seed, sharp=2.0):
    g = torch.Generator().manual_seed(seed)
    return torch.softmax(sharp * torch.randn((n, V), generator=g), -1)


def _verify(p, q, drafts, cu, u, r, status=0, ws=None):
    """The library on host tensors, against whole numbers."""
    want = su.verify(p.numpy(), None if q is None else q.numpy(), drafts.numpy(), cu.numpy(), u.numpy(), r.numpy())
    B, N = len(r), len(drafts)
    acc, tok = (torch.full((n + 8,), 12345, dtype=torch.int32, device="cuda") for n in (B, N + B))
    ws = lm.alloc_draft_workspace()
    d = [None if t is None else t.cuda() for t in (p, q, drafts, cu, u, r)]
    lm.lily_draft_verify(*d, acc[:B], tok[:N + B], ws)
    assert lm.lily_moe_device_status(ws) == status
    assert bool((acc[B:] == 12345).all()) and bool((tok[N + B:] == 12345).all())
    acc, tok = acc[:B].cpu().numpy(), tok[:N + B].cpu().numpy()
    assert np.array_equal(acc, want[0]), (acc, want[0])
    assert np.array_equal(tok[:len(want[1])], want[1]), (tok, want[1])
    return acc, tok


def _case(lens, V, seed=0, draft=True, near=0.5):
    N, B = sum(lens), len(lens)
    g = torch.Generator().manual_seed(seed + 1)
    p = _distributions(N + B, V, seed)
    rows = torch.tensor([sum(lens[:b]) + b + i for b in range(B) for i in range(lens[b])], dtype=torch.long)
    q = torch.softmax((p[rows] + 1e-30).log() + near * torch.randn((N, V), generator=g), -1)
    drafts = torch.multinomial(q if draft else p[rows], 1, generator=g)[:, 0].to(torch.int32) if N else torch.zeros(0, dtype=torch.int32)
    cu = torch.tensor([sum(lens[:b]) for b in range(B + 1)], dtype=torch.int32)
    return p, q if draft else None, drafts, cu, torch.rand(N, generator=g), torch.rand(B, generator=g)


@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 127, 128, 129, 1000, 4096, 32003])
@pytest.mark.parametrize("draft", [True, False])
def test_verify_vocabularies(V, draft):
    for seed in range(3):
        _verify(*_case([4, 0, 1, 7, 3], V, seed=seed, draft=draft))


@pytest.mark.parametrize("draft", [True, False])
def test_verify_many_sequences(draft):
    g = torch.Generator().manual_seed(9)
    lens = torch.randint(0, 6, (200,), generator=g).tolist()
    acc, _ = _verify(*_case(lens, 300, seed=5, draft=draft))
    assert 0 < (acc < np.array(lens)).sum() < 200  # both kinds are met


def test_verify_no_drafts_and_one_long_draft():
    _verify(*_case([0], 500))
    _verify(*_case([0, 0, 0], 77, draft=False))
    c = _case([1300], 40, near=0.01)
    _verify(*c[:4], c[4] * 0.9, c[5])          # refused far along, or never
    _verify(*c[:4], c[4] * 0, c[5])


def test_verify_all_accepted_and_all_refused():
    p, q, drafts, cu, u, r = _case([5, 2], 100)
    _verify(p, q, drafts, cu, u * 0, r)
    p[torch.arange(7) + torch.tensor([0] * 5 + [1] * 2), drafts.long()] = 0  # the target excludes the drafts
    acc, _ = _verify(p, q, drafts, cu, u, r)
    assert (acc == 0).all()
    _verify(p, None, drafts, cu, u, r)


def test_verify_at_borders():
    """Random numbers that fall on the border of a token's share: the next token, as sums are exact."""
    p = torch.full((3, 8), 1 / 8)
    cu = torch.tensor([0, 0, 0, 0], dtype=torch.int32)
    none = torch.zeros(0, dtype=torch.int32)
    _, tok = _verify(p, None, none, cu, torch.zeros(0), torch.tensor([0.0, 0.375, 0.999]))
    assert tok.tolist() == [0, 3, 7]
    p[0, :4] = 0
    _, tok = _verify(p, None, none, cu, torch.zeros(0), torch.tensor([0.0, 1 - 2.0 ** -24, 2.0 ** -30]))
    assert tok.tolist() == [4, 7, 0]
    # u q = p is a refusal, one unit below is not
    p = torch.full((2, 4), 0.25)
    q = torch.full((1, 4), 0.5)
    for u, n in ((0.5, 0), (0.5 - 2.0 ** -25, 1)):
        acc, _ = _verify(p, q, torch.tensor([2], dtype=torch.int32), torch.tensor([0, 1], dtype=torch.int32), torch.tensor([u]), torch.tensor([0.3]))
        assert acc[0] == n


def test_verify_single_likely_tokens():
    V = 50000
    p = torch.zeros(4, V)
    for i, v in enumerate((0, V - 1, 12345, 390)):
        p[i, v] = 1.0
    cu = torch.tensor([0, 1, 2], dtype=torch.int32)
    _verify(p, p[[0, 2]].clone(), torch.tensor([0, 5], dtype=torch.int32), cu, torch.tensor([0.999, 0.0]), torch.tensor([0.5, 0.999]))
    _verify(p, None, torch.tensor([0, 5], dtype=torch.int32), cu, torch.tensor([0.999, 0.0]), torch.tensor([0.5, 0.0]))


def test_verify_tiny_and_odd_probabilities():
    p, q, drafts, cu, u, r = _case([3, 2], 200, seed=8)
    p[:, ::3] *= 2.0 ** -50
    q[:, 1::3] *= 2.0 ** -60
    p[0, 7], p[1, 9], q[0, 3] = float("nan"), -1.0, float("nan")
    p[2, 11] = 1e-45
    _verify(p, q, drafts, cu, u, r)
    _verify(p, None, drafts, cu, u, r)


def test_verify_of_drafts_without_a_probability():
    """At the draft itself: NaN and what is below 0 count as 0, what is above 1 as 1."""
    nan, inf = float("nan"), float("inf")
    odd = [(0.5, nan), (nan, 0.5), (0.0, -1.0), (-1.0, 0.0), (nan, nan), (0.25, inf), (inf, 0.25), (0.0, 0.0), (1e-30, 0.0), (3.0, 2.0)]
    p, q = _distributions(2 * len(odd), 64, 1), _distributions(len(odd), 64, 2)
    for i, (a, b) in enumerate(odd):
        p[2 * i, 7], q[i, 7] = a, b
    n = len(odd)
    for u in (0.0, 0.3, 0.999):
        _verify(p, q, torch.full((n,), 7, dtype=torch.int32), torch.arange(n + 1, dtype=torch.int32), torch.full((n,), u), torch.full((n,), 0.4))
        _verify(p, None, torch.full((n,), 7, dtype=torch.int32), torch.arange(n + 1, dtype=torch.int32), torch.full((n,), u), torch.full((n,), 0.4))


def test_verify_where_the_target_is_nowhere_above_the_draft():
    p, q, drafts, cu, u, r = _case([2], 64, seed=3)
    q[0] = p[0]
    drafts[0] = 5
    q[0, 5] *= 1.5
    u[0] = 0.9  # refused, and nothing of p is above q: from p itself
    acc, _ = _verify(p, q, drafts, cu, u, r)
    assert acc[0] == 0


def test_verify_strided_rows():
    p, q, drafts, cu, u, r = _case([4, 3], 501)
    want = su.verify(p.numpy(), q.numpy(), drafts.numpy(), cu.numpy(), u.numpy(), r.numpy())
    wide_p, wide_q = torch.rand(len(p), 700).cuda(), torch.rand(len(q), 999).cuda()
    wide_p[:, 100:601], wide_q[:, 8:509] = p.cuda(), q.cuda()
    acc, tok, ws = torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty(9, dtype=torch.int32, device="cuda"), lm.alloc_draft_workspace()
    lm.lily_draft_verify(wide_p[:, 100:601], wide_q[:, 8:509], drafts.cuda(), cu.cuda(), u.cuda(), r.cuda(), acc, tok, ws)
    assert np.array_equal(acc.cpu().numpy(), want[0]) and np.array_equal(tok.cpu().numpy(), want[1])


def test_verify_reports_bad_indexes():
    p, q, drafts, cu, u, r = _case([3, 2, 2], 100, seed=2)
    drafts[1], drafts[5] = 100, -1
    _verify(p, q, drafts, cu, u * 0.5, r, status=-7)
    _verify(p, None, drafts, cu, u * 0.5, r, status=-7)
    # bounds that descend or leave the drafts: that sequence is left alone, the others are not
    good = _case([3, 2, 2], 100, seed=2)
    want = su.verify(*[t.numpy() for t in good])
    for bad in ([0, 3, 2, 7], [-1, 3, 5, 7], [0, 3, 5, 8]):
        acc, tok = torch.full((3,), 77, dtype=torch.int32, device="cuda"), torch.full((10,), 77, dtype=torch.int32, device="cuda")
        ws = lm.alloc_draft_workspace()
        c = torch.tensor(bad, dtype=torch.int32).cuda()
        lm.lily_draft_verify(good[0].cuda(), good[1].cuda(), good[2].cuda(), c, good[4].cuda(), good[5].cuda(), acc, tok, ws)
        assert lm.lily_moe_device_status(ws) == -7
        for b in range(3):
            if bad[b:b + 2] == [0, 3, 5, 7][b:b + 2]:
                assert acc[b] == want[0][b]
            elif bad[b] < 0 or bad[b + 1] < bad[b] or bad[b + 1] > 7:
                assert acc[b] == 77


def test_verify_reports_rows_without_weight():
    p, q, drafts, cu, u, r = _case([1, 1], 100, seed=2)
    p[:2] = 0
    _verify(p, q, drafts, cu, u, r, status=-9)


@pytest.mark.parametrize("V", [1000, 1001, 100003])
@pytest.mark.parametrize("draft", [False, True])
def test_verify_rows_that_are_no_distributions(V, draft):
    """A sum beyond the fixed point's range still writes a token of the vocabulary, or -1, and nothing else."""
    B, N = 7, 7 if draft else 0
    p = torch.ones((N + B, V), device="cuda")
    q = torch.full((N, V), 0.25, device="cuda") if draft else None
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * (1 if draft else 0)
    drafts = torch.full((N,), 3, dtype=torch.int32, device="cuda")
    u = torch.full((N,), 8.0, device="cuda")  # refused: 8 / 4 > 1
    acc, tok = (torch.full((n + 8,), -7, dtype=torch.int32, device="cuda") for n in (B, N + B))
    lm.lily_draft_verify(p, q, drafts, cu, u, torch.linspace(0, 0.999, B, device="cuda"), acc[:B], tok[:N + B], lm.alloc_draft_workspace())
    acc, tok = acc.tolist(), tok.tolist()
    assert acc == [0] * B + [-7] * 8 and tok[N + B:] == [-7] * 8
    assert all(-1 <= t < V for t in tok[:N + B])


def test_verify_refusals_of_the_binding():
    p, q, drafts, cu, u, r = (t.cuda() for t in _case([2, 1], 50))
    acc, tok, ws = torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty(5, dtype=torch.int32, device="cuda"), lm.alloc_draft_workspace()
    base = dict(p=p, q=q, drafts=drafts, cu=cu, u=u, r=r, accepted=acc, tokens=tok, ws=ws)
    for kw, match in [(dict(p=p[:4]), "p: expected"), (dict(p=p.double()), "p: expected"), (dict(q=q[:2]), "q: expected"), (dict(drafts=drafts.long()), "drafts"),
                      (dict(cu=cu[:2]), "cu"), (dict(u=u[:1]), "u: "), (dict(accepted=acc[:1]), "accepted"), (dict(tokens=tok[:4]), "tokens"),
                      (dict(ws=ws.float()), "ws"), (dict(p=p.t().contiguous().t()), "contiguous"), (dict(r=r.cpu()), "CUDA tensor")]:
        with pytest.raises(ValueError, match=match):
            lm.lily_draft_verify(**{**base, **kw})
    lm.lily_draft_verify(p[:0], None, drafts[:0], cu[:1], u[:0], r[:0], acc[:0], tok[:0], ws)


# ------------------------------------------------------------------ streams and graphs
def _all_four():
    """Inputs, outputs and a function that runs each operator once."""
    x, res, w = _rand(6, 512, dtype=F32), _rand(6, 512, seed=1), _rand(512)
    mat = su.make_matrix(700, 512, seed=2)
    matrix, table = lm.make_q4(*mat), lm.make_rope_table(lm.rope_frequencies(64))
    q, k, pos = _rand(6, 4, 128), _rand(6, 2, 128), torch.arange(6, dtype=torch.int32, device="cuda")
    v = [t.cuda() for t in _case([2, 1, 0], 3001)]
    o = {"h": torch.empty_like(res), "y": torch.empty_like(res), "y8": torch.empty(6, 512, dtype=F8, device="cuda"),
         "y8_scale": torch.empty(6, 8, device="cuda"), "out": torch.empty(6, 700, device="cuda"), "q": torch.empty_like(q), "k": torch.empty_like(k),
         "acc": torch.empty(3, dtype=torch.int32, device="cuda"), "tok": torch.empty(6, dtype=torch.int32, device="cuda")}
    ws = lm.alloc_draft_workspace()

    def run(stream=None):
        lm.lily_rms_norm(x, w, y=o["y"], y8=o["y8"], y8_scale=o["y8_scale"], residual=res, h=o["h"], stream=stream)
        lm.lily_q4_matvec(matrix, o["y8"], o["out"], x_scale=o["y8_scale"], stream=stream)
        lm.lily_rope(q, k, pos, table, o["q"], o["k"], stream=stream)
        lm.lily_draft_verify(*v, o["acc"], o["tok"], ws, stream=stream)

    return run, o, x, (mat, matrix, table, res, w, q, k, pos, v, ws)


def test_other_stream_and_captured_graph_give_the_same_bits():
    run, o, x, keep = _all_four()
    run()
    torch.cuda.synchronize()
    want = {n: t.clone() for n, t in o.items()}

    def same():
        torch.cuda.synchronize()
        return all(torch.equal(t.view(torch.uint8), want[n].view(torch.uint8)) for n, t in o.items())

    def clear():
        for t in o.values():
            t.view(torch.uint8).zero_()
        torch.cuda.synchronize()

    clear()
    side = torch.cuda.Stream()
    run(side)
    assert same()
    clear()
    with torch.cuda.stream(side):
        run()
    assert same()
    graph = torch.cuda.CUDAGraph()
    clear()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        clear()
        graph.replay()
        assert same()
    x.mul_(-1.5)  # a replay reads what is there now
    graph.replay()
    torch.cuda.synchronize()
    got = {n: t.clone() for n, t in o.items()}
    run()
    torch.cuda.synchronize()
    assert not torch.equal(got["out"], want["out"])
    assert all(torch.equal(got[n].view(torch.uint8), o[n].view(torch.uint8)) for n in o)


def test_two_calls_at_once():
    parts = su.make_matrix(3000, 2048)
    w, xs = lm.make_q4(*parts), [_rand(5, 2048, seed=s) for s in range(2)]
    outs, streams = [torch.empty(5, 3000, device="cuda") for _ in range(4)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(2):
        lm.lily_q4_matvec(w, xs[i], outs[i])
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            lm.lily_q4_matvec(w, xs[i], outs[2 + i], stream=streams[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
