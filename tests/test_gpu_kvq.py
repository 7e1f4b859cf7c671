"""GPU parity of the quantised KV cache (lily_kvq_append, lily_kvq_read) and of
the attention over it (lily_kvq_attn_decode, lily_kvq_attn_prefill).

Codes, parameters and values read back are compared bit for bit with the
oracle.  The attention's bound is derived in kvq_util.error_bound."""
import numpy as np
import pytest
import torch

import bit_grouped_expert_top_gb300 as lm
from bit_grouped_expert_top_gb300.kvq_inputs import KVQ_CONFIGS, KvqConfig
from helpers import bits as raw
from kvq_util import Cache, check, rounded
from oracle import kvq

pytestmark = pytest.mark.gpu
INDEX_ERR = -7  # LILY_ERR_DEVICE_INDEX


def _bytes(t):
    return raw(t) if t.dtype == torch.bfloat16 else t.cpu().numpy()


# ------------------------------------------------------------------ append and read back
def _fresh(c):
    """A device cache of bytes 0xA5 and the handle of it."""
    t = {k: torch.full_like(v.view(torch.uint8), 0xA5).view(v.dtype) for k, v in c.t.items()}
    return t, lm.make_kvq_cache(t)


def _strided(x, pad):
    """The same [N][H][D] values as a slice of rows that are `pad` elements wider."""
    wide = torch.full((x.shape[0], x.shape[1] * x.shape[2] + pad), float("nan"), dtype=x.dtype, device=x.device)
    view = wide[:, 8:8 + x.shape[1] * x.shape[2]].unflatten(1, x.shape[1:])
    view.copy_(x)
    return view


@pytest.mark.parametrize("bits,D,bs,H_q,H_kv,lens", [
    (4, 256, 64, 16, 2, (1, 100, 777)), (8, 256, 64, 16, 2, (64, 0, 65)), (4, 64, 32, 4, 4, (31, 32, 33)),
    (8, 64, 128, 6, 3, (127, 128, 129, 0)), (4, 128, 128, 2, 1, (300,)), (8, 128, 32, 8, 2, (5, 1, 1, 2)),
    (4, 256, 32, 4, 4, (1,)), (4, 128, 64, 16, 2, (2500, 0, 1, 613)),
])
def test_append_and_read_back_are_exact(bits, D, bs, H_q, H_kv, lens):
    cfg = KvqConfig("exact", lens=lens, H_q=H_q, H_kv=H_kv, D=D, block_size=bs, bits=bits, seed=len(lens) + D + bits)
    c = Cache(cfg).to_gpu()
    t, handle = _fresh(c)
    k, v = _strided(c.d["k_all"], 24), _strided(c.d["v_all"], 8)
    lm.lily_kvq_append(c.shape, handle, k, v, c.d["cu_all"], c.d["zeros"], c.d["block_table"], c.ws)
    for n, ref in c.h.items():   # rows that no token owns keep their 0xA5
        np.testing.assert_array_equal(_bytes(t[n]), ref, err_msg=n)
    # all of it, into strided outputs
    ko, vo = _strided(torch.zeros_like(k), 16), _strided(torch.zeros_like(v), 40)
    lm.lily_kvq_read(c.shape, handle, ko, vo, c.d["cu_all"], c.d["zeros"], c.d["block_table"], c.ws)
    assert c.status() == 0
    at = 0
    for b, L in enumerate(lens):
        kk, vv, _, _ = c.sequence(b)
        for got, ref in ((ko, kk), (vo, vv)):
            np.testing.assert_array_equal(raw(got[at:at + L].contiguous()), kvq.bf16_round(ref.astype(np.float32)))
        at += L


@pytest.mark.parametrize("bits", [4, 8])
def test_values_at_the_edges_of_the_type(bits):
    # 20 tokens of one group each: equal values, signed zeros, the whole range, tiny steps, one outlier, subnormals
    x = np.zeros((20, 1, 64), np.float32)
    rng = np.random.default_rng(9)
    x[0] = -3.25
    x[1, 0, ::2] = -0.0
    x[2, 0, 0], x[2, 0, 1] = 3.3e38, -3.3e38
    x[3, 0, 7] = 2.0 ** -126
    x[4] = 2.0 ** -120 * rng.standard_normal(64)
    x[5] = rng.standard_normal(64)
    x[5, 0, 3] = 1.0e4
    x[6] = 2.0 ** -130 * rng.integers(0, 8, 64)
    x[7] = 1.0 + 2.0 ** -7 * rng.integers(0, 2, 64)
    x[8] = np.arange(64)                              # many exact ties against the step
    x[9] = np.arange(64) * 0.5 - 15.5
    x[10] = (np.arange(64) % 31) * 0.5                # step 1 at 4 bits: every odd multiple of 0.5 is a tie
    x[11] = (np.arange(64) % 51) * 0.1
    x[12:] = rng.standard_normal((8, 1, 64)) * np.float32(10.0) ** np.arange(-20, 20, 5)[:, None, None]
    xb = torch.from_numpy(x).to(torch.bfloat16)
    s = lm.make_kvq_shape(1, 1, 1, 64, 32, 1, bits)
    t = {k: v for k, v in lm.alloc_kvq_cache(s, 1).items()}
    ws = lm.alloc_kvq_workspace(s)
    one = dict(dtype=torch.int32, device="cuda")
    lm.lily_kvq_append(s, lm.make_kvq_cache(t), xb.cuda(), (-xb).cuda(), torch.tensor([0, 20], **one), torch.zeros(1, **one),
                       torch.zeros((1, 1), **one), ws)
    for n, src in (("k", xb), ("v", -xb)):
        code, sb = kvq.quantise(raw(src), bits)
        # -0.0 and +0.0 are one value: compare the parameters as values
        np.testing.assert_array_equal(kvq.bf16_value(_bytes(t[n + "_sb"])[0, 0, 0, :20]), kvq.bf16_value(sb)[:, 0, 0])
        np.testing.assert_array_equal(_bytes(t[n + "_q"])[0, 0, 0, :20], kvq.pack(code, bits)[:, 0, 0])


def test_append_in_the_middle_with_padding_and_an_idle_sequence():
    # tokens go to positions starts + i; NaN padding rows behind cu[B] are not read; other rows stay
    cfg = KvqConfig("middle", lens=(200, 64, 90), new=(37, 0, 1), D=128, seed=5)
    c = Cache(cfg).to_gpu()
    before = {k: v.clone() for k, v in c.t.items()}
    N = cfg.N
    new = {n: torch.full((N + 30, cfg.H_kv, cfg.D), float("nan"), dtype=torch.bfloat16, device="cuda") for n in "kv"}
    g = torch.Generator().manual_seed(3)
    for n in "kv":
        new[n][:N] = torch.randn((N, cfg.H_kv, cfg.D), generator=g).to(torch.bfloat16).cuda()
    lm.lily_kvq_append(c.shape, c.handle, new["k"], new["v"], c.d["cu"], c.d["starts"], c.d["block_table"], c.ws)
    assert c.status() == 0
    for n in "kv":
        code, sb = kvq.quantise(raw(new[n][:N]), cfg.bits)
        for b, (at, m) in enumerate(((0, 37), (37, 0), (37, 1))):
            if m:
                kvq.write_rows(c.h[n + "_q"], c.table[b], cfg.lens[b] - m, kvq.pack(code, cfg.bits)[at:at + m])
                kvq.write_rows(c.h[n + "_sb"], c.table[b], cfg.lens[b] - m, sb[at:at + m])
        np.testing.assert_array_equal(_bytes(c.t[n + "_q"]), c.h[n + "_q"])
        np.testing.assert_array_equal(_bytes(c.t[n + "_sb"]), c.h[n + "_sb"])
    assert any(not torch.equal(before[k], c.t[k]) for k in before)
    # read back: rows behind cu[B] are left as they were
    ko, vo = (torch.full_like(new["k"], 7.0) for _ in "kv")
    lm.lily_kvq_read(c.shape, c.handle, ko, vo, c.d["cu"], c.d["starts"], c.d["block_table"], c.ws)
    assert (ko[N:] == 7).all() and (vo[N:] == 7).all() and torch.isfinite(ko).all()


def test_bad_entries_are_reported_and_their_rows_left_alone():
    cfg = KvqConfig("bad", lens=(100, 50), D=64, block_size=32, seed=6)
    for what in ("table", "negative", "start", "before"):
        c = Cache(cfg).to_gpu()
        table, starts = c.d["block_table"].clone(), c.d["zeros"].clone()
        if what == "table":
            table[0, 1] = c.a["n_blocks"] + 7
        elif what == "negative":
            table[0, 1] = -1
        elif what == "start":
            starts[1] = cfg.max_blocks * cfg.block_size - 10   # the last tokens pass the table
        else:
            starts[1] = -3
        ko, vo = (torch.full((cfg.N, cfg.H_kv, cfg.D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        lm.lily_kvq_read(c.shape, c.handle, ko, vo, c.d["cu_all"], starts, table, c.ws)
        assert c.status() == INDEX_ERR, what
        bad = range(32, 64) if what in ("table", "negative") else range(110, 150) if what == "start" else range(100, 103)
        got = ko.float().cpu().numpy()
        assert all((got[n] == 5).all() for n in bad)
        assert not (got[0] == 5).all()
        t, handle = _fresh(c)
        lm.lily_moe_clear_status(c.ws)
        lm.lily_kvq_append(c.shape, handle, c.d["k_all"], c.d["v_all"], c.d["cu_all"], starts, table, c.ws)
        assert c.status() == INDEX_ERR, what


def test_rows_beyond_four_gigabytes():
    # 70,000 blocks of 64 KiB of codes: offsets pass 2^32; the table uses the first and the last blocks
    cfg = KvqConfig("far", lens=(200, 130), new=(3, 2), D=256, block_size=128, bits=8, seed=7)
    c = Cache(cfg).to_gpu()
    n_blocks = 70000
    t = lm.alloc_kvq_cache(c.shape, n_blocks)
    assert t["k_q"].numel() > 1 << 32
    table = torch.tensor([[n_blocks - 1, 0], [n_blocks - 2, 65536]], dtype=torch.int32, device="cuda")
    handle = lm.make_kvq_cache(t)
    lm.lily_kvq_append(c.shape, handle, c.d["k_all"], c.d["v_all"], c.d["cu_all"], c.d["zeros"], table, c.ws)
    ko, vo = torch.empty_like(c.d["k_all"]), torch.empty_like(c.d["v_all"])
    lm.lily_kvq_read(c.shape, handle, ko, vo, c.d["cu_all"], c.d["zeros"], table, c.ws)
    out = torch.empty((2, cfg.H_q, cfg.D), dtype=torch.bfloat16, device="cuda")
    lm.lily_kvq_attn_decode(c.shape, handle, c.d["q"][:2].contiguous(), table, c.d["seq_lens"], out, c.ws)
    out5 = torch.empty((5, cfg.H_q, cfg.D), dtype=torch.bfloat16, device="cuda")
    ws = lm.alloc_kvq_workspace(c.shape, 5)
    lm.lily_kvq_attn_prefill(c.shape, handle, c.d["q"], c.d["cu"], table, c.d["seq_lens"], out5, ws)
    assert c.status() == 0 and lm.lily_moe_device_status(ws) == 0
    q = rounded(c.a["q"])
    at = 0
    for b, L in enumerate(cfg.lens):
        kk, vv, km, vm = c.sequence(b)
        np.testing.assert_array_equal(raw(ko[at:at + L]), kvq.bf16_round(kk.astype(np.float32)))
        at += L
        ref, mags = kvq.attend_and_bound(q[b:b + 1], kk, vv, [L], None, km, vm)
        check(rounded(out[b:b + 1]), ref, mags)
        m, n0 = cfg.news[b], int(c.a["cu"][b])
        ref, mags = kvq.attend_and_bound(q[n0:n0 + m], kk, vv, L - m + 1 + np.arange(m), None, km, vm)
        check(rounded(out5[n0:n0 + m]), ref, mags)


# ------------------------------------------------------------------ decode attention
def _decode(c, q=None, scale=None, lens=None):
    cfg = c.cfg
    out = torch.full((cfg.B, cfg.H_q, cfg.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lm.lily_kvq_attn_decode(c.shape, c.handle, c.d["q"] if q is None else q, c.d["block_table"],
                            c.d["seq_lens"] if lens is None else lens, out, c.ws, scale=scale)
    return out


def _check_decode(cfg, scale=None, poison=False, q_gain=1.0):
    c = Cache(cfg, poison=poison)
    c.a["q"] = (c.a["q"].float() * q_gain).to(torch.bfloat16)
    c.to_gpu()
    out = _decode(c, scale=scale)
    assert c.status() == 0
    q, got = rounded(c.a["q"]), rounded(out)
    for b in range(cfg.B):
        kk, vv, km, vm = c.sequence(b)
        ref, mags = kvq.attend_and_bound(q[b:b + 1], kk, vv, [cfg.lens[b]], scale, km, vm)
        check(got[b:b + 1], ref, mags, operand=0.0)
    return c, out


def _cfg(lens, **kw):
    return KvqConfig("decode", lens=tuple(lens), new=(1,) * len(lens), **kw)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D,bs", [(64, 32), (64, 128), (128, 64), (256, 32), (256, 64), (256, 128)])
def test_decode_head_dims_and_block_sizes(bits, D, bs):
    _check_decode(_cfg((1, bs, bs + 1, 3 * bs + 5, 1000), D=D, block_size=bs, bits=bits, seed=D + bs))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("H_q,H_kv", [(16, 2), (8, 2), (4, 4), (2, 1), (6, 3), (1, 1), (14, 2)])
def test_decode_group_sizes(bits, H_q, H_kv):
    _check_decode(_cfg((257, 15), H_q=H_q, H_kv=H_kv, D=128, bits=bits, seed=30 + H_q))


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 4095, 4097])
def test_decode_lengths(L):
    # poison: rows behind the sequence hold parameters of NaN and infinity
    _check_decode(_cfg((L,), seed=L), poison=True)


@pytest.mark.parametrize("D,H_q,H_kv", [(64, 4, 4), (128, 8, 4), (256, 16, 2)])
@pytest.mark.parametrize("lens", [(640,), (1024,), (1088,), (1, 1024, 30), (1100,) * 9 + (1, 2000, 64, 0), (1000, 60) * 19, (1100, 3, 64) * 27])
def test_decode_of_short_and_middle_caches(lens, D, H_q, H_kv):
    # a CTA for each segment and shares of the list, joins of few and of many segments
    _check_decode(_cfg(lens, D=D, H_q=H_q, H_kv=H_kv, block_size=32, seed=49 + len(lens)), poison=True)


def test_decode_empty_sequences_give_zeros():
    c, out = _check_decode(_cfg((0, 70, 0), D=64, seed=40), poison=True)
    assert (out[0] == 0).all() and (out[2] == 0).all()


def test_decode_scales_and_large_scores():
    _check_decode(_cfg((500, 90), D=128, seed=41), scale=0.2)
    _check_decode(_cfg((500, 90), D=128, seed=41), scale=-0.05)
    _check_decode(_cfg((500, 90), D=128, seed=42), scale=0.0)
    _check_decode(_cfg((700, 33), D=256, seed=43), q_gain=6.0)     # a sharp softmax
    _check_decode(_cfg((700, 33), D=256, seed=43), q_gain=1e-30, scale=1e28)   # queries far below the fp16 range
    _check_decode(_cfg((700, 33), D=256, seed=43), q_gain=1e30, scale=1e-32)


@pytest.mark.parametrize("gain", [1e-12, 1e-4, 300.0, 1e12])
def test_decode_values_of_any_size(gain):
    # the codes and parameters have no range limit: values from 1e-12 to 1e12, and growing along the sequence
    cfg = _cfg((300, 1000), D=128, seed=44)
    c = Cache(cfg)
    ramp = torch.logspace(0, 3, 1300).view(-1, 1, 1)
    for n, f in (("k", 1.0), ("v", gain)):
        x = (c.a[n + "_all"].float() * f * (ramp if n == "v" else 1.0)).to(torch.bfloat16)
        for b, (at, L) in enumerate(((0, 300), (300, 1000))):
            code, sb = kvq.quantise(raw(x[at:at + L]), cfg.bits)
            kvq.write_rows(c.h[n + "_q"], c.table[b], 0, kvq.pack(code, cfg.bits))
            kvq.write_rows(c.h[n + "_sb"], c.table[b], 0, sb)
    c.to_gpu()
    got, q = rounded(_decode(c)), rounded(c.a["q"])
    assert c.status() == 0
    for b in range(2):
        kk, vv, km, vm = c.sequence(b)
        ref, mags = kvq.attend_and_bound(q[b:b + 1], kk, vv, [cfg.lens[b]], None, km, vm)
        check(got[b:b + 1], ref, mags, operand=0.0)


def test_decode_many_sequences():
    lens = tuple(int(x) for x in np.random.default_rng(5).integers(0, 1500, 40))
    _check_decode(_cfg(lens, D=128, seed=45))
    lens = tuple(int(x) for x in np.random.default_rng(6).integers(0, 90, 400))
    _check_decode(_cfg(lens, D=64, H_q=4, H_kv=4, block_size=32, bits=8, seed=46))


@pytest.mark.parametrize("name", ["kvq_32k", "kvq_128k"])
def test_decode_long_contexts(name):
    c, out = _check_decode(KVQ_CONFIGS[name])
    first = out.clone()
    for _ in range(5):
        assert torch.equal(first, _decode(c))


def test_decode_strided_queries():
    cfg = _cfg((100, 50, 7), D=128, seed=47)
    c = Cache(cfg).to_gpu()
    want = _decode(c)
    assert torch.equal(want, _decode(c, q=_strided(c.d["q"], 48)))


def test_attention_reports_bad_tables_and_lengths():
    cfg = _cfg((100, 50), D=64, seed=48)
    for what in ("table", "negative", "long", "below"):
        c = Cache(cfg, n_query=2).to_gpu()
        lens = c.d["seq_lens"].clone()
        if what == "table":
            c.d["block_table"][0, 1] = c.a["n_blocks"] + 3
        elif what == "negative":
            c.d["block_table"][0, 0] = -5
        else:
            lens[1] = cfg.max_blocks * cfg.block_size + 1 if what == "long" else -4
            c.d["block_table"][1].clamp_(min=0)   # the clamped length reads the whole table
        ref = _decode(c, lens=lens)
        assert c.status() == INDEX_ERR, what
        lm.lily_moe_clear_status(c.ws)
        out = torch.full_like(ref, float("nan"))
        lm.lily_kvq_attn_prefill(c.shape, c.handle, c.d["q"], c.d["cu"], c.d["block_table"], lens, out, c.ws)
        assert c.status() == INDEX_ERR, what
        assert torch.isfinite(out).all()


# ------------------------------------------------------------------ prefill attention
def _prefill(c, scale=None, q=None):
    cfg = c.cfg
    q = c.d["q"] if q is None else q
    out = torch.full((q.shape[0], cfg.H_q, cfg.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lm.lily_kvq_attn_prefill(c.shape, c.handle, q, c.d["cu"], c.d["block_table"], c.d["seq_lens"], out, c.ws, scale=scale)
    return out


def _check_prefill(cfg, scale=None, poison=False, rows=None):
    c = Cache(cfg, poison=poison, n_query=cfg.N).to_gpu()
    out = _prefill(c, scale)
    assert c.status() == 0
    q, got = rounded(c.a["q"]), rounded(out)
    for b, m in enumerate(cfg.news):
        if m == 0:
            continue
        n0, L = int(c.a["cu"][b]), cfg.lens[b]
        kk, vv, km, vm = c.sequence(b)
        pick = np.arange(m) if rows is None else np.unique(np.clip(rows, 0, m - 1))
        ref, mags = kvq.attend_and_bound(q[n0 + pick], kk, vv, L - m + 1 + pick, scale, km, vm)
        check(got[n0 + pick], ref, mags)
    return c, out


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D,bs", [(64, 32), (64, 128), (128, 64), (256, 32), (256, 64), (256, 128)])
def test_prefill_head_dims_and_block_sizes(bits, D, bs):
    cfg = KvqConfig("prefill", lens=(1, bs + 1, 300, 500), new=(1, bs + 1, 40, 3), D=D, block_size=bs, bits=bits, seed=D + bs)
    _check_prefill(cfg, poison=True)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("H_q,H_kv", [(16, 2), (8, 2), (4, 4), (2, 1), (6, 3), (1, 1), (14, 2)])
def test_prefill_group_sizes(bits, H_q, H_kv):
    cfg = KvqConfig("groups", lens=(257, 200), new=(150, 17), H_q=H_q, H_kv=H_kv, D=128, bits=bits, seed=H_q)
    _check_prefill(cfg)


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 300])
@pytest.mark.parametrize("ctx", [0, 1, 127, 1000])
def test_prefill_lengths(m, ctx):
    _check_prefill(KvqConfig("lengths", lens=(ctx + m,), new=(m,), D=64, seed=m + ctx), poison=True)


def test_prefill_ragged_batch_with_idle_sequences():
    lens = (700, 0, 64, 5, 1300, 90, 333)
    new = (700, 0, 0, 5, 4, 1, 129)
    _check_prefill(KvqConfig("ragged", lens=lens, new=new, D=256, seed=50), poison=True)


def test_prefill_more_queries_than_cached_tokens():
    # a sequence shorter than its chunk: the queries before its first position see nothing and give zeros
    cfg = KvqConfig("short", lens=(40, 10), new=(40, 10), D=128, seed=51)
    c = Cache(cfg, poison=True, n_query=cfg.N).to_gpu()
    c.d["seq_lens"] = torch.tensor([25, 0], dtype=torch.int32, device="cuda")
    out = _prefill(c)
    assert c.status() == 0
    assert (out[:15] == 0).all() and (out[40:] == 0).all()
    q = rounded(c.a["q"])
    kk, vv, km, vm = c.sequence(0, 25)
    ref, mags = kvq.attend_and_bound(q[15:40], kk, vv, 1 + np.arange(25), None, km, vm)
    check(rounded(out[15:40]), ref, mags)


def test_prefill_padding_rows_are_left_as_they_were():
    cfg = KvqConfig("padding", lens=(50, 300), new=(20, 130), D=128, seed=52)
    c = Cache(cfg, n_query=cfg.N + 200).to_gpu()
    want = _prefill(c)
    q = torch.full((cfg.N + 200, cfg.H_q, cfg.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    q[:cfg.N] = c.d["q"]
    out = torch.full_like(q, 3.0)
    lm.lily_kvq_attn_prefill(c.shape, c.handle, q, c.d["cu"], c.d["block_table"], c.d["seq_lens"], out, c.ws)
    assert torch.isfinite(out).all() and (out[cfg.N:] == 3).all()
    check(rounded(out[:cfg.N]), rounded(want), {"score": np.zeros((cfg.N, cfg.H_q)), "value": np.abs(rounded(want)) * 2})
    assert c.status() == 0


def test_prefill_scales_and_strided_queries():
    cfg = KvqConfig("scales", lens=(300, 77), new=(60, 77), D=128, seed=53)
    for s in (0.2, -0.05, 0.0):
        _check_prefill(cfg, scale=s)
    c = Cache(cfg, n_query=cfg.N).to_gpu()
    assert torch.equal(_prefill(c), _prefill(c, q=_strided(c.d["q"], 24)))


def test_prefill_long_context_and_repeats():
    # a chunk at the end of a long context, and a long prompt (a sample of its rows against the oracle)
    c, out = _check_prefill(KvqConfig("long", lens=(20000,), new=(96,), seed=54))
    for _ in range(3):
        assert torch.equal(out, _prefill(c))
    _check_prefill(KvqConfig("prompt", lens=(3000,), seed=55), rows=np.arange(0, 3000, 97))
    # draft tokens of several sequences
    _check_prefill(KvqConfig("draft", lens=(4096, 5000, 2049, 17), new=(4, 4, 4, 4), seed=56))


@pytest.mark.parametrize("D,bits", [(64, 8), (128, 4), (256, 4)])
@pytest.mark.parametrize("lens,new", [((20000,), (3,)), ((9000, 40, 0, 5000), (16, 1, 0, 7)), ((2000, 3000) * 10, (1, 2) * 10)])
def test_prefill_of_few_tokens_on_long_contexts(lens, new, D, bits):
    # items with more and with fewer parts than a join's loads in flight
    c, out = _check_prefill(KvqConfig("few", lens=lens, new=new, D=D, bits=bits, seed=58 + D), poison=True)
    assert torch.equal(out, _prefill(c))


@pytest.mark.parametrize("D,H_q,H_kv", [(64, 8, 2), (128, 16, 4), (256, 16, 2)])
@pytest.mark.parametrize("lens,new", [((1000,), None), ((1700,), None), ((700, 300, 0, 61), None), ((2500, 900), (300, 40)), ((40,) * 33, None)])
def test_prefill_of_short_prompts(lens, new, D, H_q, H_kv):
    # items that are whole for a share, and cut ones; more sequences than a warp has lanes
    cfg = KvqConfig("short", lens=lens, new=new, D=D, H_q=H_q, H_kv=H_kv, block_size=32, seed=74 + D)
    c, out = _check_prefill(cfg, poison=True, rows=np.arange(0, 2500, 23))
    assert torch.equal(out, _prefill(c))


def test_prefill_of_one_token_equals_decode():
    cfg = KvqConfig("one", lens=(800, 90, 1), new=(1, 1, 1), seed=57)
    c = Cache(cfg, n_query=3).to_gpu()
    a, b = rounded(_prefill(c)), rounded(_decode(c))
    q = rounded(c.a["q"])
    for i, L in enumerate(cfg.lens):
        kk, vv, km, vm = c.sequence(i)
        _, mags = kvq.attend_and_bound(q[i:i + 1], kk, vv, [L], None, km, vm)
        check(a[i:i + 1], b[i:i + 1], {k: 2 * v for k, v in mags.items()})


# ------------------------------------------------------------------ together, captured, on another stream
def test_prompt_then_decode_steps():
    # two sequences: prompts in two chunks (append, prefill), then token by token (append, decode), the cache and
    # every output against the oracle
    cfg = KvqConfig("serve", lens=(150, 90), D=128, block_size=32, seed=60)
    c = Cache(cfg, n_query=140).to_gpu()
    t, handle = _fresh(c)
    steps = [((0, 0), (100, 33)), ((100, 33), (140, 33))] + [((140 + i, 33 + i), (141 + i, 34 + i)) for i in range(8)]
    first = c.a["cu_all"].numpy()
    i32 = dict(dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(61)
    for lo, hi in steps:
        m = [h - l for l, h in zip(lo, hi)]
        cu = torch.tensor([0, m[0], m[0] + m[1]], **i32)
        pick = torch.cat([torch.arange(first[b] + lo[b], first[b] + hi[b]) for b in range(2)]).cuda()
        lm.lily_kvq_append(c.shape, handle, c.d["k_all"][pick], c.d["v_all"][pick], cu, torch.tensor(lo, **i32),
                           c.d["block_table"], c.ws)
        q = torch.randn((sum(m), cfg.H_q, cfg.D), generator=g).to(torch.bfloat16)
        out = torch.empty_like(q, device="cuda")
        lens = torch.tensor(hi, **i32)
        if m == [1, 1]:
            lm.lily_kvq_attn_decode(c.shape, handle, q.cuda(), c.d["block_table"], lens, out, c.ws)
        else:
            lm.lily_kvq_attn_prefill(c.shape, handle, q.cuda(), cu, c.d["block_table"], lens, out, c.ws)
        assert c.status() == 0
        at = 0
        for b in range(2):
            if m[b] == 0:
                continue
            kk, vv, km, vm = c.sequence(b, hi[b])
            ref, mags = kvq.attend_and_bound(rounded(q[at:at + m[b]]), kk, vv, lo[b] + 1 + np.arange(m[b]), None, km, vm)
            check(rounded(out[at:at + m[b]]), ref, mags)
            at += m[b]


def _captured(c, fn, outs):
    """fn(stream) captured on a side stream: capture runs nothing, two replays equal the direct call."""
    fn(torch.cuda.current_stream())
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    for o in outs:
        o.zero_()
    with torch.cuda.graph(g, stream=side):
        fn(side)
    torch.cuda.synchronize()
    assert all(bool((o == 0).all()) for o in outs)
    for _ in range(2):
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs))
    return g, want


def test_capture_and_two_graphs_on_one_workspace():
    cfg = KvqConfig("capture", lens=(300, 90), new=(20, 3), D=128, seed=62)
    c = Cache(cfg, n_query=cfg.N).to_gpu()
    d = c.d
    outs = [torch.empty((2, cfg.H_q, cfg.D), dtype=torch.bfloat16, device="cuda"),
            torch.empty((cfg.N, cfg.H_q, cfg.D), dtype=torch.bfloat16, device="cuda")]
    ko, vo = (torch.empty((cfg.N, cfg.H_kv, cfg.D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    kn, vn = (torch.randn_like(ko) for _ in "kv")

    def step(st):
        lm.lily_kvq_append(c.shape, c.handle, kn, vn, d["cu"], d["starts"], d["block_table"], c.ws, stream=st)
        lm.lily_kvq_attn_prefill(c.shape, c.handle, d["q"], d["cu"], d["block_table"], d["seq_lens"], outs[1], c.ws, stream=st)
        lm.lily_kvq_read(c.shape, c.handle, ko, vo, d["cu"], d["starts"], d["block_table"], c.ws, stream=st)

    def token(st):
        lm.lily_kvq_attn_decode(c.shape, c.handle, d["q"][:2], d["block_table"], d["seq_lens"], outs[0], c.ws, stream=st)

    g1, w1 = _captured(c, step, [outs[1], ko, vo])
    g2, w2 = _captured(c, token, [outs[0]])
    for _ in range(3):   # replayed in turn on one stream: the workspace is shared
        g1.replay()
        g2.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(w1 + w2, [outs[1], ko, vo, outs[0]]))
    assert c.status() == 0


def test_two_streams_with_their_own_workspaces():
    cfgs = [_cfg((900, 200), D=128, seed=63), _cfg((1500,), D=256, bits=8, seed=64)]
    cs = [Cache(x).to_gpu() for x in cfgs]
    want = [_decode(c).clone() for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [torch.empty_like(w) for w in want]
    for _ in range(10):
        for c, st, o in zip(cs, streams, outs):
            lm.lily_kvq_attn_decode(c.shape, c.handle, c.d["q"], c.d["block_table"], c.d["seq_lens"], o, c.ws, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


def _scaled(cfg, k_gain, v_gain):
    """A cache whose K and V are the workload's times a gain, the bf16 values quantised as usual."""
    c = Cache(cfg, n_query=cfg.N)
    first = c.a["cu_all"].numpy()
    for n, g in (("k", k_gain), ("v", v_gain)):
        x = raw((c.a[n + "_all"].float() * g).to(torch.bfloat16))
        for b, L in enumerate(cfg.lens):
            code, sb = kvq.quantise(x[first[b]:first[b] + L], cfg.bits)
            kvq.write_rows(c.h[n + "_q"], c.table[b], 0, kvq.pack(code, cfg.bits))
            kvq.write_rows(c.h[n + "_sb"], c.table[b], 0, sb)
    return c.to_gpu()


@pytest.mark.parametrize("bits", [4, 8])
def test_prefill_values_beyond_fp16_are_reported(bits):
    # K and V are rebuilt in fp16: a value of 65520 or more would become infinite and is reported; decode has no limit
    cfg = KvqConfig("range", lens=(200,), new=(30,), D=128, bits=bits, seed=70)
    for k_gain, v_gain in ((1.0, 1e6), (1e6, 1.0)):
        c = _scaled(cfg, k_gain, v_gain)
        _prefill(c, scale=1e-8)
        assert c.status() == -9   # LILY_ERR_DEVICE_RANGE
    # large but within the range: exact to the usual bound
    c = _scaled(cfg, 1000.0, 1000.0)
    out = _prefill(c, scale=1e-4)
    assert c.status() == 0
    kk, vv, km, vm = c.sequence(0)
    ref, mags = kvq.attend_and_bound(rounded(c.a["q"]), kk, vv, 171 + np.arange(30), 1e-4, km, vm)
    check(rounded(out), ref, mags)


def test_prefill_queries_of_any_size():
    # q is scaled per row by a power of two before it becomes fp16
    cfg = KvqConfig("qsize", lens=(200,), new=(30,), D=128, seed=71)
    for gain in (1e-30, 1e30):
        c = Cache(cfg, n_query=cfg.N)
        c.a["q"] = (c.a["q"].float() * gain).to(torch.bfloat16)
        c.to_gpu()
        out = _prefill(c, scale=0.1 / gain)
        assert c.status() == 0
        kk, vv, km, vm = c.sequence(0)
        ref, mags = kvq.attend_and_bound(rounded(c.a["q"]), kk, vv, 171 + np.arange(30), 0.1 / gain, km, vm)
        check(rounded(out), ref, mags)


def test_prefill_sharp_softmax():
    # scores that grow along the sequence: the running maximum moves many times, O is rescaled each time
    cfg = KvqConfig("sharp", lens=(1500,), new=(64,), D=256, seed=72)
    c = Cache(cfg, n_query=cfg.N)
    ramp = torch.linspace(0.0, 8.0, 1500).view(-1, 1, 1)
    x = raw((c.a["k_all"].float() + ramp * torch.sign(c.a["q"][0].float().view(2, 8, 256).mean(1, keepdim=True)).view(1, 2, 256)).to(torch.bfloat16))
    code, sb = kvq.quantise(x, cfg.bits)
    kvq.write_rows(c.h["k_q"], c.table[0], 0, kvq.pack(code, cfg.bits))
    kvq.write_rows(c.h["k_sb"], c.table[0], 0, sb)
    c.to_gpu()
    for scale in (None, 0.5):
        out = _prefill(c, scale=scale)
        assert c.status() == 0
        kk, vv, km, vm = c.sequence(0)
        ref, mags = kvq.attend_and_bound(rounded(c.a["q"]), kk, vv, 1437 + np.arange(64), scale, km, vm)
        check(rounded(out), ref, mags)


@pytest.mark.parametrize("D,bits", [(64, 8), (128, 4), (256, 4), (256, 8)])
def test_cold_caches_change_nothing(D, bits):
    # with the inputs out of L2 the warps of a CTA meet in another order: the results are the same bits
    cfg = KvqConfig("cold", lens=(1, 33, 300, 500), new=(1, 33, 40, 3), D=D, block_size=32, bits=bits, seed=73)
    c, want = _check_prefill(cfg, poison=True)
    one = Cache(cfg.with_(new=(1, 1, 1, 1))).to_gpu()
    want_one = _decode(one)
    flush = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")
    for i in range(8):
        flush.fill_(i)
        assert torch.equal(want, _prefill(c)), i
        flush.fill_(i)
        assert torch.equal(want_one, _decode(one)), i


@pytest.mark.parametrize("B", [255, 256, 700])
def test_append_and_read_of_many_sequences(B):
    # around the number of sequences whose bounds a CTA keeps at hand; every third one idle
    lens = tuple((b * 7) % 23 + 1 for b in range(B))
    new = tuple(0 if b % 3 == 0 else (b * 5) % L + 1 for b, L in enumerate(lens))
    cfg = KvqConfig("many", lens=lens, new=new, H_q=2, H_kv=1, D=64, block_size=32, seed=74)
    c = Cache(cfg).to_gpu()
    first = c.a["cu_all"].numpy()
    pick = np.concatenate([np.arange(first[b] + L - m, first[b] + L) for b, (L, m) in enumerate(zip(lens, new)) if m])
    k, v = (c.d[n][torch.from_numpy(pick).cuda()] for n in ("k_all", "v_all"))
    t, handle = _fresh(c)
    lm.lily_kvq_append(c.shape, handle, k, v, c.d["cu"], c.d["starts"], c.d["block_table"], c.ws)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    lm.lily_kvq_read(c.shape, handle, ko, vo, c.d["cu"], c.d["starts"], c.d["block_table"], c.ws)
    assert c.status() == 0
    kk = np.concatenate([c.sequence(b)[0][L - m:] for b, (L, m) in enumerate(zip(lens, new)) if m])
    np.testing.assert_array_equal(raw(ko), kvq.bf16_round(kk.astype(np.float32)))
    out = torch.empty((B, cfg.H_q, cfg.D), dtype=torch.bfloat16, device="cuda")
    q = torch.randn((B, cfg.H_q, cfg.D), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    lm.lily_kvq_attn_decode(c.shape, c.handle, q.cuda(), c.d["block_table"], c.d["seq_lens"], out, c.ws)
    ws = lm.alloc_kvq_workspace(c.shape, cfg.N)
    chunk = torch.empty((cfg.N, cfg.H_q, cfg.D), dtype=torch.bfloat16, device="cuda")
    lm.lily_kvq_attn_prefill(c.shape, c.handle, c.d["q"], c.d["cu"], c.d["block_table"], c.d["seq_lens"], chunk, ws)
    assert c.status() == 0 and lm.lily_moe_device_status(ws) == 0
    for b in list(range(0, B, 37)) + [B - 1]:
        kk, vv, km, vm = c.sequence(b)
        ref, mags = kvq.attend_and_bound(rounded(q[b:b + 1]), kk, vv, [lens[b]], None, km, vm)
        check(rounded(out[b:b + 1]), ref, mags, operand=0.0)
        m, n0 = new[b], int(c.a["cu"][b])
        if m:
            ref, mags = kvq.attend_and_bound(rounded(c.a["q"][n0:n0 + m]), kk, vv, lens[b] - m + 1 + np.arange(m), None, km, vm)
            check(rounded(chunk[n0:n0 + m]), ref, mags)


def test_prefill_on_two_streams():
    # two calls at once, each with its own workspace: tensor memory and CTA pairs are taken by one after the other
    cs = [Cache(KvqConfig("streams", lens=(900, 300), new=(400, 300), D=D, bits=bits, seed=75 + D), n_query=700).to_gpu()
          for D, bits in ((256, 4), (128, 8))]
    want = [_prefill(c).clone() for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [torch.empty_like(w) for w in want]
    for _ in range(6):
        for c, st, o in zip(cs, streams, outs):
            lm.lily_kvq_attn_prefill(c.shape, c.handle, c.d["q"], c.d["cu"], c.d["block_table"], c.d["seq_lens"], o, c.ws, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))
    assert all(c.status() == 0 for c in cs)


def test_binding_refuses_tensors_of_other_shapes():
    c = Cache(_cfg((100, 50), D=64, seed=66)).to_gpu()
    t, q, n = c.d["block_table"], c.d["q"], c.d["seq_lens"]
    out = torch.empty_like(q)

    def refused(what, **kw):
        a = {"q": q, "block_table": t, "seq_lens": n, "out": out, "ws": c.ws, **kw}
        with pytest.raises(ValueError, match=what):
            lm.lily_kvq_attn_decode(c.shape, c.handle, a["q"], a["block_table"], a["seq_lens"], a["out"], a["ws"])

    refused("block_table", block_table=torch.cat([t, t], 1))   # a wider table
    refused("block_table", block_table=t.flatten())
    refused("block_table", block_table=t.long())
    refused("block_table", block_table=torch.cat([t, t], 1)[:, :t.shape[1]])   # its rows are not contiguous
    refused("seq_lens", seq_lens=n[:1])
    refused("out", out=out[:1])
    refused("sequences", q=q[:1])
    refused("ws", ws=c.ws.to(torch.int8))
    assert c.status() == 0


def test_attention_of_more_sequences_than_threads():
    rng = np.random.default_rng(67)
    lens = tuple(int(x) for x in rng.integers(0, 70, 1300))
    new = tuple(int(min(L, x)) for L, x in zip(lens, rng.integers(0, 4, 1300)))
    _check_decode(_cfg(lens, D=64, H_q=2, H_kv=1, block_size=32, seed=67), poison=True)
    _check_prefill(KvqConfig("many", lens=lens, new=new, D=64, H_q=2, H_kv=1, block_size=32, seed=68), poison=True)
    _check_prefill(KvqConfig("many", lens=lens, new=lens, D=128, H_q=2, H_kv=2, block_size=32, seed=69), poison=True)


def test_calls_with_nothing_to_do():
    # every sequence empty or idle: zeros from decode, untouched rows from prefill
    cfg = KvqConfig("idle", lens=(0, 0, 90), new=(0, 0, 0), D=128, seed=70)
    c = Cache(cfg, n_query=8).to_gpu()
    q = torch.randn((8, cfg.H_q, cfg.D), device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, 5.0)
    lm.lily_kvq_attn_prefill(c.shape, c.handle, q, c.d["cu"], c.d["block_table"], c.d["seq_lens"], out, c.ws)
    assert (out == 5).all()
    none = torch.zeros_like(c.d["seq_lens"])
    lm.lily_kvq_attn_decode(c.shape, c.handle, q[:3], c.d["block_table"], none, out[:3], c.ws)
    assert (out[:3] == 0).all() and (out[3:] == 5).all()
    assert c.status() == 0


def test_attention_over_a_cache_beyond_four_gigabytes():
    # the same blocks at the end of arrays of 4.9 GB: the same bits
    cfg = KvqConfig("far", lens=(300, 77), new=(40, 3), seed=71)
    c = Cache(cfg, n_query=cfg.N).to_gpu()
    n, far = c.a["n_blocks"], 300000
    want = [_prefill(c), _decode(c, q=c.d["q"][:2])]
    big = {}
    for k, t in c.t.items():
        big[k] = torch.empty((far + n,) + t.shape[1:], dtype=t.dtype, device="cuda")
        big[k][far:] = t
    assert big["k_q"].numel() > 1 << 32
    c.handle = lm.make_kvq_cache(big)
    c.d["block_table"] = torch.where(c.d["block_table"] >= 0, c.d["block_table"] + far, -1).to(torch.int32)
    assert torch.equal(_prefill(c), want[0]) and torch.equal(_decode(c, q=c.d["q"][:2]), want[1])
    assert c.status() == 0


def test_sequences_that_share_blocks():
    # a common prefix held once: both tables name the same blocks
    cfg = _cfg((200, 200), D=128, seed=72)
    c = Cache(cfg, n_query=2).to_gpu()
    alone = _decode(c)
    c.d["block_table"][1] = c.d["block_table"][0]
    q = c.d["q"][:1].expand(2, -1, -1).contiguous()
    both = _decode(c, q=q)
    assert torch.equal(both[0], both[1]) and torch.equal(both[0], alone[0])
    assert c.status() == 0


@pytest.mark.parametrize("D,bits,bs", [(256, 8, 64), (256, 8, 128), (256, 4, 64), (128, 8, 128), (128, 4, 64)])
def test_decode_of_fresh_memory(D, bits, bs):
    # blocks of memory that the GPU has not touched lately arrive in any order: every call gives the same bits
    cfg = _cfg((20000, 9000), D=D, bits=bits, block_size=bs, seed=73)
    c = Cache(cfg).to_gpu()
    want = _decode(c)
    host = {k: t.cpu() for k, t in c.t.items()}
    for i in range(6):
        c.t = c.handle = None
        torch.cuda.empty_cache()
        pad = torch.empty((i + 1) << 22, dtype=torch.uint8, device="cuda")
        c.t = {k: t.cuda() for k, t in host.items()}
        c.handle = lm.make_kvq_cache(c.t)
        torch.cuda.synchronize()
        assert torch.equal(_decode(c), want)
        del pad
    assert c.status() == 0
