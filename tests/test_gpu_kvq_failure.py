"""Failure detection of the quantised-cache attention without a GPU fault.

Every wait of the kernels is bounded: when one runs out, LILY_ERR_DEVICE_TIMEOUT is recorded in the workspace, every role
gives up, copies and tensor-core work in flight drain, and the kernel returns, so that the context stays usable.  The
test-only build variant (waits of 1 ms; with 77 sequences or query tokens, one that nothing completes) makes one run out;
the product library then runs the same call and is checked against the oracle."""
import ctypes

import numpy as np
import pytest
import torch

import bit_grouped_expert_top_gb300 as lm
from bit_grouped_expert_top_gb300 import _abi
from bit_grouped_expert_top_gb300.build import STALL_TEST_T
from bit_grouped_expert_top_gb300.kvq_inputs import KvqConfig
from kvq_util import Cache, check, rounded
from oracle import kvq

pytestmark = pytest.mark.gpu
TIMEOUT = -6  # LILY_ERR_DEVICE_TIMEOUT


def _call(L, c, decode):
    q, s = c.d["q"], c.shape
    out = torch.zeros_like(q)
    head = (ctypes.byref(s), ctypes.byref(c.handle), q.data_ptr(), s.H_q * s.D)
    tail = (c.d["block_table"].data_ptr(), c.d["seq_lens"].data_ptr(), s.D ** -0.5, out.data_ptr(), c.ws.data_ptr(), c.ws.numel(),
            torch.cuda.current_stream().cuda_stream)
    if decode:
        rc = L.lily_kvq_attn_decode(*head, *tail)
    else:
        rc = L.lily_kvq_attn_prefill(*head, q.shape[0], c.d["cu"].data_ptr(), *tail)
    assert rc == 0
    return out


def _check(c, out):
    q, got = rounded(c.a["q"]), rounded(out)
    for b, m in enumerate(c.cfg.news):
        rows = slice(int(c.a["cu"][b]), int(c.a["cu"][b + 1]))
        kk, vv, km, vm = c.sequence(b)
        ref, mags = kvq.attend_and_bound(q[rows], kk, vv, c.cfg.lens[b] - m + 1 + np.arange(m), None, km, vm)
        check(got[rows], ref, mags)


def _both(cfg, decode):
    """Two calls of the variant: one that stalls (and the product library's after it), one of another size."""
    variant = _abi.load_variant("stalltest")
    c = Cache(cfg, n_query=cfg.N).to_gpu()
    _call(variant, c, decode)
    assert c.status() == TIMEOUT
    torch.cuda.synchronize()
    lm.lily_moe_clear_status(c.ws)
    out = _call(_abi.load(), c, decode)
    assert c.status() == 0
    _check(c, out)
    return variant


@pytest.mark.parametrize("D,bits", [(64, 8), (128, 4), (256, 4)])
@pytest.mark.parametrize("L", [200, 3000])
def test_decode_wait_that_runs_out(L, D, bits):
    lens = (L,) + (150,) * (STALL_TEST_T - 1)
    cfg = KvqConfig("stall", lens=lens, new=(1,) * len(lens), H_q=4, D=D, bits=bits, seed=90)
    variant = _both(cfg, True)
    c = Cache(cfg.with_(lens=lens[1:], new=(1,) * (len(lens) - 1))).to_gpu()   # one fewer: the product's path
    assert torch.equal(_call(variant, c, True), _call(_abi.load(), c, True)) and c.status() == 0


# pairs of CTAs (D = 256, 128), single CTAs of 128 rows (D = 64) and of 32 rows
@pytest.mark.parametrize("kw", [dict(D=256), dict(D=128, bits=8), dict(D=64), dict(D=256, H_q=2, lens=(500, 900, 300), new=(30, 30, 17))])
@pytest.mark.parametrize("ctx", [0, 2000])
def test_prefill_wait_that_runs_out(ctx, kw):
    cfg = KvqConfig("stall", **{"lens": (ctx + STALL_TEST_T,), "new": (STALL_TEST_T,), "seed": 91, **kw})
    assert cfg.N == STALL_TEST_T
    variant = _both(cfg, False)
    fewer = cfg.new[:-1] + (cfg.new[-1] - 1,)
    c = Cache(cfg.with_(new=fewer), n_query=cfg.N).to_gpu()
    assert torch.equal(_call(variant, c, False), _call(_abi.load(), c, False)) and c.status() == 0
