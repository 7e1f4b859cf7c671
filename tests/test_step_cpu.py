"""Host-side checks of the operators around the attention and the expert layers: refusals, which are made before anything is
enqueued, and the frequencies of the rotary positions.  Nothing here touches a GPU."""
import ctypes
import math

import pytest
import torch

import bit_grouped_expert_top_gb300 as lm
import step_util as su
from bit_grouped_expert_top_gb300 import _abi

FAKE = 0x10000000  # an aligned address that is never dereferenced
NAN, INF = float("nan"), float("inf")


def _norm(N=4, H=1, d=256, xt=0, ht=0, wt=0, x=FAKE, xs=None, residual=FAKE, h=FAKE, w=FAKE, offset=0.0, eps=1e-6, y=FAKE, y8=FAKE,
          sc=FAKE, shape=True):
    s = _abi.lily_norm_shape(N, H, d, xt, ht, wt) if shape else None
    return lm.load().lily_rms_norm(s, x, H * d if xs is None else xs, residual, h, w, offset, eps, y, y8, sc, None)


def test_norm_refusals():
    assert _norm(shape=False) == -1
    for kw in ({"N": -1}, {"H": 0}, {"d": 0}, {"eps": -1e-6}, {"eps": NAN}, {"eps": INF}, {"offset": NAN}, {"x": None},
               {"y": None, "y8": None, "sc": None}, {"y8": None}, {"sc": None}, {"residual": None}, {"h": None}, {"xs": 248},
               {"xs": -256}, {"xs": 1 << 40}):
        assert _norm(**kw) == -1, kw
    for kw in ({"xt": 2}, {"ht": 2}, {"wt": 3}, {"xt": -1}, {"d": 250}, {"d": 200}, {"d": 16448}, {"N": 1 << 30, "H": 2}):
        assert _norm(**kw) == -2, kw
    for kw in ({"xs": 260}, {"x": FAKE + 8}, {"residual": FAKE + 8}, {"h": FAKE + 4}, {"w": FAKE + 2}, {"y": FAKE + 8}, {"y8": FAKE + 8},
               {"sc": FAKE + 4}):
        assert _norm(**kw) == -3, kw
    assert _norm(N=0) == 0 and _norm(N=0, x=None) == 0


def _matvec(T=4, rows=8, K=256, xt=0, ot=0, w=FAKE, s=FAKE, b=FAKE, x=FAKE, xs=None, sc=None, out=FAKE, shape=True, matrix=True):
    return lm.load().lily_q4_matvec(_abi.lily_q4_shape(T, rows, K, xt, ot) if shape else None, _abi.lily_q4(w, s, b) if matrix else None,
                                    x, K if xs is None else xs, sc, out, None)


def test_matvec_refusals():
    assert _matvec(shape=False) == -1 and _matvec(matrix=False) == -1
    for kw in ({"T": -1}, {"rows": 0}, {"K": 0}, {"w": None}, {"s": None}, {"b": None}, {"x": None}, {"out": None}, {"sc": FAKE},
               {"xt": 2}, {"xs": 248}):
        assert _matvec(**kw) == -1, kw
    for kw in ({"T": 33}, {"K": 100}, {"K": 16448}, {"rows": 1 << 30}, {"xt": 1}, {"ot": 2}):
        assert _matvec(**kw) == -2, kw
    for kw in ({"w": FAKE + 8}, {"s": FAKE + 2}, {"b": FAKE + 8}, {"x": FAKE + 8}, {"out": FAKE + 4}, {"xs": 260}, {"xt": 2, "sc": FAKE + 4},
               {"xt": 2, "sc": FAKE, "xs": 264}):
        assert _matvec(**kw) == -3, kw
    assert _matvec(T=0, x=None, out=None) == 0


def _rope(N=4, H_q=2, H_k=1, D=64, rot=32, il=0, q=FAKE, qs=None, k=FAKE, ks=None, pos=FAKE, table=FAKE, amp=1.0, qo=FAKE + 4096, qos=None,
          ko=FAKE + 8192, kos=None, shape=True):
    dq, dk = H_q * D, H_k * D
    return lm.load().lily_rope(_abi.lily_rope_shape(N, H_q, H_k, D, rot, il) if shape else None, q, dq if qs is None else qs, k,
                               dk if ks is None else ks, pos, table, amp, qo, dq if qos is None else qos, ko, dk if kos is None else kos, None)


def test_rope_refusals():
    assert _rope(shape=False) == -1
    for kw in ({"N": -1}, {"H_q": 0}, {"H_k": -1}, {"D": 0}, {"rot": 0}, {"rot": 80}, {"il": 2}, {"il": -1}, {"amp": NAN}, {"q": None}, {"k": None},
               {"pos": None}, {"table": None}, {"qo": None}, {"ko": None}, {"qs": 120}, {"ks": 56}, {"qos": 64}, {"kos": 0},
               {"qo": FAKE, "qs": 256}, {"ko": FAKE, "k": FAKE, "kos": 128}):
        assert _rope(**kw) == -1, kw
    for kw in ({"D": 72, "rot": 16}, {"D": 528}, {"rot": 24}, {"N": 1 << 28}, {"N": 1, "H_q": 1 << 20}):
        assert _rope(**kw) == -2, kw
    for kw in ({"q": FAKE + 8}, {"k": FAKE + 8}, {"pos": FAKE + 4}, {"table": FAKE + 8}, {"qo": FAKE + 2}, {"ko": FAKE + 8}, {"qs": 132}, {"kos": 68}):
        assert _rope(**kw) == -3, kw
    assert _rope(N=0, q=None, k=None, pos=None, table=None, qo=None, ko=None) == 0


def _verify(B=2, N=3, V=100, p=FAKE, ps=100, q=FAKE, qs=100, dr=FAKE, cu=FAKE, u=FAKE, r=FAKE, acc=FAKE, tok=FAKE, ws=FAKE, n=256, shape=True):
    return lm.load().lily_draft_verify(_abi.lily_draft_shape(B, N, V) if shape else None, p, ps, q, qs, dr, cu, u, r, acc, tok, ws, n, None)


def test_verify_refusals():
    assert _verify(shape=False) == -1
    for kw in ({"B": -1}, {"N": -1}, {"V": 0}, {"p": None}, {"dr": None}, {"cu": None}, {"u": None}, {"r": None}, {"acc": None}, {"tok": None},
               {"ws": None}, {"ps": 99}, {"qs": 99}):
        assert _verify(**kw) == -1, kw
    for kw in ({"B": 65537}, {"V": (1 << 24) + 1, "ps": 1 << 25, "qs": 1 << 25}, {"N": (1 << 31) - 1}):
        assert _verify(**kw) == -2, kw
    for kw in ({"p": FAKE + 4}, {"q": FAKE + 4}, {"dr": FAKE + 4}, {"cu": FAKE + 8}, {"u": FAKE + 4}, {"r": FAKE + 4}, {"acc": FAKE + 4}, {"tok": FAKE + 4},
               {"ws": FAKE + 16}):
        assert _verify(**kw) == -3, kw
    assert _verify(n=255) == -4
    assert _verify(B=0, p=None, r=None, acc=None, tok=None, cu=None) == 0


# ------------------------------------------------------------------ the binding's own checks (tensors on the host are refused)
def test_binding_refuses_host_tensors_and_wrong_forms():
    def t(*size, dtype=torch.bfloat16):
        return torch.zeros(size, dtype=dtype)

    i32, f32 = torch.int32, torch.float32
    x = t(4, 256)
    for kw, match in [(dict(y=t(4, 256)), "CUDA tensor"), (dict(x=t(256), y=x), "x: expected"), (dict(x=t(4, 256, dtype=torch.float16), y=x), "x: expected"),
                      (dict(x=t(2, 3, 4, 8), y=x), "x: expected")]:
        with pytest.raises(ValueError, match=match):
            lm.lily_rms_norm(**{"x": x, "weight": None, **kw})
    with pytest.raises(ValueError, match="CUDA tensor"):
        lm.make_q4(t(8, 128, dtype=torch.uint8), t(8, 4), t(8, 4))
    with pytest.raises(ValueError, match="K a multiple of 64"):
        lm.make_q4(t(8, 100, dtype=torch.uint8), t(8, 4), t(8, 4))
    w = _abi.lily_q4(FAKE, FAKE, FAKE)
    w.rows, w.K, w.device = 8, 256, 0
    for kw, match in [({}, "CUDA tensor"), (dict(x=t(4, 128)), "x: expected"), (dict(x=t(4, 256, dtype=f32)), "x: expected")]:
        with pytest.raises(ValueError, match=match):
            lm.lily_q4_matvec(**{"w": w, "x": x, "out": t(4, 8), **kw})
    q, pos, table = t(4, 2, 64), t(4, dtype=i32), t(16, dtype=torch.int64)
    for args, match in [((q, q, pos, table), "CUDA tensor"), ((t(4, 128), q, pos, table), "q: expected"),
                        ((t(4, 2, 64, dtype=f32), q, pos, table), "q: expected")]:
        with pytest.raises(ValueError, match=match):
            lm.lily_rope(*args)
    p = t(5, 10, dtype=f32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        lm.lily_draft_verify(p, None, t(3, dtype=i32), t(3, dtype=i32), t(3, dtype=f32), t(2, dtype=f32), t(2, dtype=i32), t(5, dtype=i32),
                             t(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="p: expected"):
        lm.lily_draft_verify(p, None, t(4, dtype=i32), t(3, dtype=i32), t(4, dtype=f32), t(2, dtype=f32), t(2, dtype=i32), t(6, dtype=i32),
                             t(256, dtype=torch.uint8))


# ------------------------------------------------------------------ frequencies and their table
@pytest.mark.parametrize("rot", [2, 16, 64, 128, 256])
@pytest.mark.parametrize("scaling,kw", [("none", {}), ("linear", {"factor": 4.0}), ("base", {"factor": 8.0}),
                                        ("parts", {"factor": 8.0, "original": 32768.0}),
                                        ("parts", {"factor": 32.0, "original": 8192.0, "low": 1.0, "high": 4.0})])
def test_frequencies(rot, scaling, kw):
    got = lm.rope_frequencies(rot, 1000000.0, scaling, **kw)
    want = su.frequencies(rot, 1000000.0, scaling, **kw)
    assert got.shape == (rot // 2,) and torch.allclose(got, want, rtol=1e-14, atol=0)   # pow's last bits differ by library
    table = lm.make_rope_table(got, "cpu")
    assert table.dtype == torch.int64
    for f, t in zip(got.tolist(), table.tolist()):
        # a turn in 64-bit steps; fp64 has 53 bits of it
        assert abs(t % 2 ** 64 - f / (2 * math.pi) * 2 ** 64) <= f / (2 * math.pi) * 2.0 ** (64 - 51) + 1


def test_scaled_frequencies_keep_the_fast_pairs_and_stretch_the_slow_ones():
    plain, parts = lm.rope_frequencies(128, 1e6), lm.rope_frequencies(128, 1e6, "parts", factor=8.0, original=32768.0)
    assert torch.equal(plain[:8], parts[:8])
    assert torch.allclose(plain[-8:] / 8.0, parts[-8:], rtol=1e-14)


def test_frequency_refusals():
    L, out = lm.load(), (ctypes.c_double * 64)()

    def call(kind=0, theta=1e4, factor=2.0, original=100.0, low=1.0, high=4.0, rot=64, to=out):
        return L.lily_rope_frequencies(_abi.lily_rope_scaling(kind, theta, factor, original, low, high), rot, to)

    assert call() == 0 and call(kind=3) == 0
    assert L.lily_rope_frequencies(None, 64, out) == -1 and call(to=None) == -1
    assert call(rot=0) == -1 and call(rot=63) == -1 and call(theta=0.0) == -1 and call(theta=NAN) == -1 and call(theta=INF) == -1
    assert call(kind=4) == -2 and call(kind=-1) == -2
    assert call(factor=NAN) == 0 and call(kind=1, factor=0.0) == -1 and call(kind=2, factor=NAN) == -1
    for kw in ({"original": 0.0}, {"original": NAN}, {"low": 4.0}, {"high": NAN}, {"high": INF}):
        assert call(kind=3, **kw) == -1, kw
    with pytest.raises(ValueError, match="scaling"):
        lm.rope_frequencies(64, scaling="other")
    with pytest.raises(lm.LilyError):
        lm.rope_frequencies(63)
    for bad in ([7.0], [-0.1], [NAN], [INF], [2 * math.pi]):
        with pytest.raises(lm.LilyError):
            lm.make_rope_table(bad, "cpu")
    with pytest.raises(ValueError, match="vector"):
        lm.make_rope_table([[1.0]], "cpu")
    assert lm.make_rope_table([0.0, math.pi], "cpu").tolist() == [0, -2 ** 63]


def test_the_plain_verification_draws_from_the_target():
    """The oracle itself: over all random numbers on a grid, the tokens come out as the target has them."""
    import numpy as np

    p = np.array([[1 / 8, 4 / 8, 1 / 8, 2 / 8], [1 / 4] * 4], np.float32)
    q = np.array([[2 / 8, 1 / 8, 4 / 8, 1 / 8]], np.float32)
    for given, drafts in ((q, range(4)), (None, [2])):
        count = np.zeros(4)
        for x in drafts:
            for u in range(64):
                for r in range(64):
                    _, tokens = su.verify(p, given, np.array([x], np.int32), np.array([0, 1]), np.array([u / 64], np.float32), np.array([r / 64], np.float32))
                    count[tokens[0]] += (q[0, x] if given is not None else 1.0) / 4096
        assert np.abs(count - p[0]).max() <= 4 / 64, (given is None, count)  # a grid of 64 in each of at most four pieces
