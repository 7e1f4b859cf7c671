"""Host-side checks of the quantised-cache entry points: every refusal is made
before anything is enqueued, so none of this touches a GPU."""
import ctypes

import pytest
import torch

import bit_grouped_expert_top_gb300 as lm
from bit_grouped_expert_top_gb300 import _abi

FAKE = 0x10000000  # an aligned address that is never dereferenced
by = ctypes.byref


def _shape(**kw):
    base = dict(B=2, H_q=16, H_kv=2, D=256, block_size=64, max_blocks=8, bits=4)
    base.update(kw)
    return lm.make_kvq_shape(**base)


def _cache(s, n_blocks=10, **kw):
    c = _abi.lily_kvq_cache(FAKE, FAKE, FAKE, FAKE, n_blocks, n_blocks * s.H_kv * s.D * s.block_size * s.bits // 8)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("kw,ok", [
    ({}, True), ({"bits": 8}, True), ({"D": 64}, True), ({"block_size": 128}, True), ({"H_q": 2}, True),
    ({"H_q": 6, "H_kv": 3}, True), ({"max_blocks": 1 << 24}, True),
    ({"bits": 2}, False), ({"bits": 16}, False), ({"D": 96}, False), ({"D": 512}, False), ({"block_size": 16}, False),
    ({"H_q": 18}, False), ({"H_q": 15}, False), ({"B": 0}, False), ({"B": 65536}, False), ({"max_blocks": 0}, False),
    ({"H_kv": 0}, False), ({"H_q": 8192, "H_kv": 8192}, False), ({"max_blocks": 1 << 25}, False),
])
def test_supported_shapes(kw, ok):
    assert (lm.lily_kvq_workspace_bytes(_shape(**kw)) > 0) == ok
    assert (lm.lily_kvq_workspace_bytes(_shape(**kw), 100) > 0) == ok


def test_workspace_grows_with_the_query_tokens_and_stays_bounded():
    s = _shape()
    assert lm.lily_kvq_workspace_bytes(s, -1) == 0
    w = [lm.lily_kvq_workspace_bytes(s, n) for n in (0, 1, 64, 4096, 65536)]
    assert w == sorted(w) and w[-1] <= 65536 * 16 * 256 * 4 * 2 + w[0]


def _copy(fn, s, c, k=FAKE, ks=512, v=FAKE, vs=512, N=4, cu=FAKE, st=FAKE, tb=FAKE, ws=FAKE, n=1 << 32):
    return getattr(lm.load(), fn)(by(s) if s else None, by(c) if c else None, k, ks, v, vs, N, cu, st, tb, ws, n, None)


@pytest.mark.parametrize("fn", ["lily_kvq_append", "lily_kvq_read"])
def test_copy_refusals(fn):
    s = _shape()
    c = _cache(s)
    assert _copy(fn, None, c) == -1 and _copy(fn, s, None) == -1
    assert _copy(fn, _shape(bits=5), c) == -2
    for name in ("k_q", "k_sb", "v_q", "v_sb"):
        assert _copy(fn, s, _cache(s, **{name: None})) == -1
        assert _copy(fn, s, _cache(s, **{name: FAKE + 8})) == -3
    # a cache of another geometry: its bytes do not match the shape
    assert _copy(fn, s, _cache(_shape(bits=8))) == -1
    assert _copy(fn, s, _cache(s, code_bytes=1)) == -1
    assert _copy(fn, s, _cache(s, n_blocks=0)) == -1
    assert _copy(fn, s, c, N=-1) == -1
    for a in ("k", "v", "cu", "st", "tb", "ws"):
        assert _copy(fn, s, c, **{a: None}) == -1, a
        assert _copy(fn, s, c, **{a: FAKE + 4}) == -3, a
    assert _copy(fn, s, c, ks=504) == -1 and _copy(fn, s, c, vs=516) == -3 and _copy(fn, s, c, vs=-512) == -1
    assert _copy(fn, s, c, n=lm.lily_kvq_workspace_bytes(s) - 1) == -4
    # no tokens: a no-op, the token arrays may be NULL
    assert _copy(fn, s, c, N=0, k=None, v=None, cu=None, st=None, tb=None) == 0


def test_attention_refusals():
    s = _shape()
    c, L = _cache(s), lm.load()
    nan, inf = float("nan"), float("inf")

    def decode(s=s, c=c, q=FAKE, qs=4096, tb=FAKE, sl=FAKE, scale=0.0625, out=FAKE, ws=FAKE, n=1 << 40):
        return L.lily_kvq_attn_decode(by(s) if s else None, by(c) if c else None, q, qs, tb, sl, scale, out, ws, n, None)

    def prefill(s=s, c=c, q=FAKE, qs=4096, N=4, cu=FAKE, tb=FAKE, sl=FAKE, scale=0.0625, out=FAKE, ws=FAKE, n=1 << 40):
        return L.lily_kvq_attn_prefill(by(s) if s else None, by(c) if c else None, q, qs, N, cu, tb, sl, scale, out, ws,
                                       n, None)

    for call in (decode, prefill):
        assert call(s=None) == -1 and call(c=None) == -1
        assert call(s=_shape(H_q=18)) == -2 and call(c=_cache(s, code_bytes=7)) == -1
        assert call(scale=nan) == -1 and call(scale=inf) == -1
        assert call(scale=3e38) == -1   # times log2(e) it is no fp32 number
        for a in ("q", "tb", "sl", "out", "ws"):
            assert call(**{a: None}) == -1, a
            assert call(**{a: FAKE + 8}) == -3, a
        assert call(qs=4095) == -1 and call(qs=4100) == -3
    assert decode(n=lm.lily_kvq_workspace_bytes(s) - 1) == -4
    assert prefill(n=lm.lily_kvq_workspace_bytes(s, 4) - 1) == -4
    assert prefill(N=-1) == -1 and prefill(cu=None) == -1
    assert prefill(N=0, q=None, cu=None, tb=None, sl=None, out=None) == 0


def test_binding_refuses_what_the_library_cannot_see():
    s = _shape()
    c = _cache(s)
    k = torch.zeros((3, 2, 256), dtype=torch.bfloat16)
    i = torch.zeros(16, dtype=torch.int32)
    ws = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        lm.lily_kvq_append(s, c, k, k, i, i, i, ws)
    with pytest.raises(ValueError, match="bfloat16"):
        lm.lily_kvq_append(s, c, k.float(), k, i, i, i, ws)
    with pytest.raises(ValueError, match="tokens"):
        lm.lily_kvq_read(s, c, k, k[:2], i, i, i, ws)
    with pytest.raises(ValueError, match="bfloat16"):
        lm.lily_kvq_attn_decode(s, c, k, i, i, k, ws)   # 2 heads where 16 are due
    with pytest.raises(ValueError, match="uint8"):
        lm.make_kvq_cache({n: k for n in ("k_q", "k_sb", "v_q", "v_sb")})
    with pytest.raises(ValueError, match="unsupported"):
        lm.alloc_kvq_cache(_shape(D=32), 4, device="cpu")
    t = lm.alloc_kvq_cache(s, 4, device="cpu")
    assert t["k_q"].shape == (4, 2, 4, 64, 32) and t["v_sb"].shape == (4, 2, 4, 64, 2)
    with pytest.raises(ValueError, match="unlike"):
        lm.make_kvq_cache({**t, "v_sb": t["v_sb"][:3]})
    with pytest.raises(ValueError, match="CUDA tensor"):
        lm.make_kvq_cache(t)
