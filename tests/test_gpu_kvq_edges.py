"""The quantised cache's kernels at the edges of their range: groups of equal values, scales that no fp16 number holds,
values and weights of very different size.

What the results may be off by is derived at each test; references are fp64 on the values that the codes stand for."""
import numpy as np
import pytest
import torch

import bit_grouped_expert_top_gb300 as lm
from bit_grouped_expert_top_gb300.kvq_inputs import KvqConfig
from helpers import bits as raw
from kvq_util import Cache, check, error_bound, rounded
from oracle import kvq

pytestmark = pytest.mark.gpu
RANGE_ERR = -9  # LILY_ERR_DEVICE_RANGE


def _bf16(x):
    return raw(torch.as_tensor(np.asarray(x, np.float32)).to(torch.bfloat16))


def _store(c, n, b, x):
    """Quantises x [L][H_kv][D] as the whole of sequence b's K or V in the host copy."""
    code, sb = kvq.quantise(_bf16(x), c.cfg.bits)
    kvq.write_rows(c.h[n + "_q"], c.table[b], 0, kvq.pack(code, c.cfg.bits))
    kvq.write_rows(c.h[n + "_sb"], c.table[b], 0, sb)


def _queries(c, q):
    c.a["q"] = torch.from_numpy(np.array(q, np.float32, order="C")).to(torch.bfloat16)


def _decode(c, scale=None):
    out = torch.full((c.cfg.B, c.cfg.H_q, c.cfg.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lm.lily_kvq_attn_decode(c.shape, c.handle, c.d["q"], c.d["block_table"], c.d["seq_lens"], out, c.ws, scale=scale)
    return out


def _prefill(c, scale=None):
    out = torch.full((c.cfg.N, c.cfg.H_q, c.cfg.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lm.lily_kvq_attn_prefill(c.shape, c.handle, c.d["q"], c.d["cu"], c.d["block_table"], c.d["seq_lens"], out, c.ws, scale=scale)
    return out


def _reference(c, b, rows, limits, scale=None):
    kk, vv, km, vm = c.sequence(b)
    return kvq.attend_and_bound(rounded(c.a["q"])[rows], kk, vv, limits, scale, km, vm)


# lengths of decode batches: a CTA has one (sequence, KV head) each, several steps a warp; and one that is cut between CTAs
WHOLE = (1000, 700, 130, 1, 900, 300) * 6 + (1000, 0)
CUT = (2500, 700, 130)


def _one_token(lens, **kw):
    return KvqConfig("edges", lens=lens, new=(1,) * len(lens), H_q=8, H_kv=4, **kw)


def _rising(cfg, seed, rise):
    """q of one direction for every head, and per sequence keys whose scores rise by `rise` powers of two in 1,000 tokens."""
    rng = np.random.default_rng(seed)
    u = rng.choice([-1.0, 1.0], cfg.D)
    q = np.broadcast_to(u, (cfg.N, cfg.H_q, cfg.D))
    step = rise / (np.sqrt(cfg.D) * np.log2(np.e)) / 1000
    keys = [0.05 * rng.standard_normal((L, cfg.H_kv, cfg.D)) + u * (np.arange(L) * step)[:, None, None] for L in cfg.lens]
    return q, keys, rng


def _check_decode(c, scale=None):
    got = rounded(_decode(c, scale))
    assert c.status() == 0
    for b, L in enumerate(c.cfg.lens):
        ref, mags = _reference(c, b, slice(b, b + 1), [L], scale)
        check(got[b:b + 1], ref, mags, operand=0.0)


# ------------------------------------------------------------------ decode: groups of equal values
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D,bs", [(64, 32), (128, 64), (256, 32), (256, 128)])
@pytest.mark.parametrize("lens", [WHOLE, CUT])
@pytest.mark.parametrize("kind", ["zero", "equal", "prefix", "tiny"])
def test_decode_of_values_without_a_scale(kind, lens, D, bs, bits):
    # groups of equal values have scale 0; the scores rise, so that weights pass the running maximum
    cfg = _one_token(lens, D=D, block_size=bs, bits=bits, seed=D + bits)
    q, keys, rng = _rising(cfg, 11, 20.0)
    c = Cache(cfg)
    _queries(c, q)
    for b, L in enumerate(lens):
        if L == 0:
            continue
        _store(c, "k", b, keys[b])
        x = rng.standard_normal((L, cfg.H_kv, D))
        equal = np.repeat(rng.standard_normal((L, cfg.H_kv, D // 64)), 64, -1)
        _store(c, "v", b, {"zero": 0 * x, "equal": equal, "tiny": x * 2.0 ** -121,
                           "prefix": np.where((np.arange(L) < L * 2 // 3)[:, None, None], equal, x)}[kind])
    _check_decode(c.to_gpu())


# ------------------------------------------------------------------ append: equal values of any size
@pytest.mark.parametrize("bits", [4, 8])
def test_append_of_equal_values_is_exact(bits):
    sizes = np.array([2.0 ** 60, 2.0 ** 63, 2.0 ** 64, 2.0 ** 65, 1e25, 1e30, 3.3e38, 2.0 ** -30, 2.0 ** -100, 2.0 ** -126, 2.0 ** -133, 1.0])
    x = np.repeat(np.concatenate([sizes, -sizes]), 64).reshape(-1, 1, 64).astype(np.float32)
    near = x.copy()                     # the same, one value a step away
    near[:, 0, 5] *= np.float32(1 + 2.0 ** -7)
    xb = torch.from_numpy(np.concatenate([x, near])).to(torch.bfloat16)
    n = xb.shape[0]
    s = lm.make_kvq_shape(1, 1, 1, 64, 64, 1, bits)
    t, ws = lm.alloc_kvq_cache(s, 1), lm.alloc_kvq_workspace(s)
    one = dict(dtype=torch.int32, device="cuda")
    cu, zero, table = torch.tensor([0, n], **one), torch.zeros(1, **one), torch.zeros((1, 1), **one)
    handle = lm.make_kvq_cache(t)
    lm.lily_kvq_append(s, handle, xb.cuda(), (-xb).cuda(), cu, zero, table, ws)
    for name, src in (("k", xb), ("v", -xb)):
        code, sb = kvq.quantise(raw(src), bits)
        np.testing.assert_array_equal(kvq.bf16_value(raw(t[name + "_sb"]))[0, 0, 0, :n], kvq.bf16_value(sb)[:, 0, 0])
        np.testing.assert_array_equal(t[name + "_q"].cpu().numpy()[0, 0, 0, :n], kvq.pack(code, bits)[:, 0, 0])
    k, v = torch.empty_like(xb, device="cuda"), torch.empty_like(xb, device="cuda")
    lm.lily_kvq_read(s, handle, k, v, cu, zero, table, ws)
    m = 2 * len(sizes)
    assert torch.equal(k[:m].cpu(), xb[:m]) and torch.equal(v[:m].cpu(), -xb[:m])
    assert lm.lily_moe_device_status(ws) == 0


# ------------------------------------------------------------------ prefill: scales that fp16 does not hold
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [(30, 1), (200, 40)])
def test_prefill_of_groups_that_span_the_fp16_range(new, D, bits):
    # ends within fp16, a step of 8192 and more at 4 bits
    cfg = KvqConfig("wide", lens=(230, 70), new=new, D=D, bits=bits, seed=80 + D)
    rng = np.random.default_rng(12)
    c = Cache(cfg, n_query=cfg.N)
    for b, L in enumerate(cfg.lens):
        for n in "kv":
            x = rng.uniform(-60000, 57000, (L, cfg.H_kv, D))
            x[:, :, 3::64], x[:, :, 9::64] = (-65280, 57600) if n == "v" else (-65024, 64512)
            _store(c, n, b, x)
    c.to_gpu()
    got = rounded(_prefill(c, scale=1e-6))
    assert c.status() == 0
    for b, (L, m) in enumerate(zip(cfg.lens, cfg.news)):
        n0 = int(c.a["cu"][b])
        ref, mags = _reference(c, b, slice(n0, n0 + m), L - m + 1 + np.arange(m), 1e-6)
        check(got[n0:n0 + m], ref, mags)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("gain", [2.0 ** -12, 1e-4, 1e-5, 1e-6, 2.0 ** -22])
def test_prefill_of_small_values_rounds_them_once(gain, bits):
    # a value is rounded to fp16: off by 2^-11 of itself, or below 2^-14 by 2^-25; as much for a key, whose score is then off by
    # scale sum_d |q_d| 2^-25 more, and a weight by e^(2 times that)
    cfg = KvqConfig("small", lens=(1, 1, 3, 300), new=(1, 1, 3, 40), D=128, bits=bits, seed=81)
    for k_gain, v_gain in ((1.0, gain), (gain, 1.0)):
        c = Cache(cfg, n_query=cfg.N)
        rng = np.random.default_rng(13)
        for b, L in enumerate(cfg.lens):
            for n, g in (("k", k_gain), ("v", v_gain)):
                _store(c, n, b, g * rng.uniform(0.5, 1.5, (L, 1, 1)) * rng.standard_normal((L, cfg.H_kv, 128)))
        c.to_gpu()
        scale = 0.08 / k_gain
        got = rounded(_prefill(c, scale=scale))
        assert c.status() == 0 and np.isfinite(got).all()
        for b, (L, m) in enumerate(zip(cfg.lens, cfg.news)):
            rows = slice(int(c.a["cu"][b]), int(c.a["cu"][b + 1]))
            ref, mags = _reference(c, b, rows, L - m + 1 + np.arange(m), scale)
            k_abs = 2.0 ** -25 * scale * np.abs(rounded(c.a["q"])[rows]).sum(-1) * (k_gain < 1)
            bound = error_bound(ref, mags, 2.0 ** -11) + np.expm1(2 * k_abs)[..., None] * mags["value"] + 2.0 ** -25 * 1.01
            err = np.abs(got[rows] - ref)
            assert (err <= bound).all(), (b, (err / bound).max())


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("n", ["k", "v"])
@pytest.mark.parametrize("scale,bias", [(0x7FC0, 0x3F80), (0x3F80, 0x7FC0), (0x7F80, 0x3F80), (0x3F80, 0xFF80), (0xFFC0, 0xFFC0)])
def test_prefill_reports_parameters_that_are_no_numbers(scale, bias, n, bits):
    cfg = KvqConfig("nan", lens=(200, 100), new=(5, 7), D=64, bits=bits, seed=82)
    c = Cache(cfg, n_query=cfg.N).to_gpu()
    _prefill(c)
    assert c.status() == 0
    rows = kvq.rows_of(c.h[n + "_sb"], c.table[1], 50, 1)
    rows[0, 1, 0] = scale, bias
    kvq.write_rows(c.h[n + "_sb"], c.table[1], 50, rows)
    c.to_gpu()
    got = _prefill(c)
    assert c.status() == RANGE_ERR
    assert torch.isfinite(got[:5]).all()   # the other sequence is not touched by it


# ------------------------------------------------------------------ prefill: small weights
@pytest.mark.parametrize("gap", [10.3, 18.3, 22.4, 24.5, 26.2])
@pytest.mark.parametrize("D,new", [(64, 3), (128, 70), (256, 300)])
def test_prefill_of_many_small_weights_behind_a_large_one(D, new, gap):
    # one token whose score is `gap` powers of two above all others, and whose value is 0: the output is what thousands
    # of small weights add up to.  A weight is rounded to fp16 at 2^7 or more for the largest: off by 2^-11 of itself or
    # by 2^-25 / 2^7 of the largest.
    L = 4096
    cfg = KvqConfig("sink", lens=(L,), new=(new,), D=D, seed=83)
    rng = np.random.default_rng(14)
    c = Cache(cfg, n_query=cfg.N)
    _queries(c, np.ones((new, cfg.H_q, D)))
    k = np.zeros((L, cfg.H_kv, D))
    k[0] = 1.0
    v = rng.uniform(0.5, 1.5, (L, cfg.H_kv, D))
    v[0] = 0.0
    _store(c, "k", 0, k)
    _store(c, "v", 0, v)
    c.to_gpu()
    scale = gap / (D * np.log2(np.e))
    got = rounded(_prefill(c, scale=scale))
    assert c.status() == 0
    pick = np.unique(np.linspace(0, new - 1, 12).astype(int))
    ref, mags = _reference(c, 0, pick, L - new + 1 + pick, scale)
    vm = c.sequence(0)[3]
    floor = np.repeat(vm.sum(0), cfg.H_q // cfg.H_kv, 0)[None] * 2.0 ** -32
    err, bound = np.abs(got[pick] - ref), error_bound(ref, mags, 2.0 ** -11) + floor
    assert np.isfinite(got).all() and (err <= bound).all(), (err / bound).max()


# ------------------------------------------------------------------ decode: values of very different size
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("at", [0, 333, 999])
def test_decode_of_a_huge_value_with_no_weight(at, D, bits):
    # a token whose values are 2^40 times the others' and whose weight is below 2^-90 changes nothing; for one head of
    # the two it has all of the weight
    for lens in (WHOLE, CUT):
        cfg = _one_token(lens, D=D, bits=bits, seed=84)
        rng = np.random.default_rng(15)
        c = Cache(cfg)
        u = rng.choice([-1.0, 1.0], D)
        q = np.broadcast_to(u, (cfg.N, 8, D)).copy()
        q[:, 1::2] *= -1
        _queries(c, q)
        for b, L in enumerate(lens):
            if L <= at:
                continue
            k, v = 0.05 * rng.standard_normal((L, 4, D)), rng.standard_normal((L, 4, D))
            k[at] -= 100.0 / (np.sqrt(D) * np.log2(np.e)) * u
            v[at] *= 2.0 ** 40
            _store(c, "k", b, k)
            _store(c, "v", b, v)
        c.to_gpu()
        got = rounded(_decode(c))
        assert c.status() == 0
        for b, L in enumerate(lens):
            ref, mags = _reference(c, b, slice(b, b + 1), [L])
            for h in range(8):   # head by head: the check's norm is one of all that it gets
                check(got[b:b + 1, h:h + 1], ref[:, h:h + 1], {n: x[:, h:h + 1] for n, x in mags.items()}, operand=0.0)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("lens", [WHOLE, CUT])
@pytest.mark.parametrize("D", [128, 256])
def test_decode_of_groups_of_unlike_size(D, lens, bits):
    # each group of channels on its own, whatever the others hold
    cfg = _one_token(lens, D=D, bits=bits, seed=85)
    q, keys, rng = _rising(cfg, 16, 20.0)
    c = Cache(cfg)
    _queries(c, q)
    gain = 2.0 ** np.repeat(np.array([40.0, -20.0, 0.0, -45.0])[:D // 64], 64)
    for b, L in enumerate(lens):
        if L:
            _store(c, "k", b, keys[b])
            _store(c, "v", b, rng.standard_normal((L, cfg.H_kv, D)) * gain)
    c.to_gpu()
    got = rounded(_decode(c))
    assert c.status() == 0
    for b, L in enumerate(lens):
        ref, mags = _reference(c, b, slice(b, b + 1), [L])
        for g in range(D // 64):
            cut = slice(64 * g, 64 * g + 64)
            check(got[b:b + 1, :, cut], ref[..., cut], {"score": mags["score"], "value": mags["value"][..., cut]}, operand=0.0)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("gain", [2.0 ** 100, 2.0 ** 121, 2.0 ** 126])
def test_decode_of_the_largest_values(gain, D, bits):
    # sums of weights times values stay finite up to the end of the type; equal scores, and scores that rise
    for rise, lens in ((0.0, WHOLE), (20.0, WHOLE), (20.0, CUT)):
        cfg = _one_token(lens, D=D, bits=bits, seed=86)
        q, keys, rng = _rising(cfg, 17, rise)
        c = Cache(cfg)
        _queries(c, q)
        for b, L in enumerate(lens):
            if L:
                _store(c, "k", b, keys[b])
                _store(c, "v", b, gain * rng.uniform(0.5, 1.9, (L, cfg.H_kv, D)))
        _check_decode(c.to_gpu())


@pytest.mark.parametrize("gap", [10.3, 18.3, 22.4, 24.5])
@pytest.mark.parametrize("D,bits", [(64, 4), (128, 8), (256, 4)])
def test_decode_of_many_small_weights_behind_a_large_one(D, bits, gap):
    # as for prefill above; the scales of the values lie within 2^7 of each other and the small weights have the larger ones:
    # a weight times a scale is 2^5 or more in fp16 where the largest weight has it, so off by 2^-25 / 2^5 of the largest at most
    cfg = _one_token((4096, 900) * 5, D=D, bits=bits, seed=87)
    rng = np.random.default_rng(18)
    c = Cache(cfg)
    _queries(c, np.ones((cfg.N, cfg.H_q, D)))
    for b, L in enumerate(cfg.lens):
        k = np.zeros((L, cfg.H_kv, D))
        k[0] = 1.0
        v = rng.uniform(0.5, 1.5, (L, cfg.H_kv, D))
        v[0] *= 0.02
        _store(c, "k", b, k)
        _store(c, "v", b, v)
    c.to_gpu()
    scale = gap / (D * np.log2(np.e))
    got = rounded(_decode(c, scale))
    assert c.status() == 0
    for b, L in enumerate(cfg.lens):
        ref, mags = _reference(c, b, slice(b, b + 1), [L], scale)
        floor = np.repeat(c.sequence(b)[3].sum(0), cfg.H_q // cfg.H_kv, 0)[None] * 2.0 ** -30
        err, bound = np.abs(got[b:b + 1] - ref), error_bound(ref, mags, 0.0) + floor
        assert np.isfinite(got).all() and (err <= bound).all(), (err / bound).max()
