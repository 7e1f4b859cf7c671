"""Helpers of the quantised-cache tests: a cache filled by the oracle, the
library's calls on it, and the error bound of the attention."""
from __future__ import annotations

import numpy as np
import torch

import bit_grouped_expert_top_gb300 as lm
from bit_grouped_expert_top_gb300.kvq_inputs import KvqConfig, make_kvq
from helpers import bits as raw
from oracle import kvq


class Cache:
    """One workload: host copies (numpy) filled by the oracle, device copies for the library."""

    def __init__(self, cfg: KvqConfig, poison: bool = False, n_query: int = 0):
        self.cfg, self.a = cfg, make_kvq(cfg)
        lead = (self.a["n_blocks"], cfg.H_kv, cfg.D // 64, cfg.block_size)
        self.h = {}
        self.table = self.a["block_table"].numpy()
        first = self.a["cu_all"].numpy()
        for n in "kv":
            # rows that no token owns: bytes 0xA5, or (poison) parameters of NaN and infinity
            self.h[n + "_q"] = np.full(lead + (8 * cfg.bits,), 0xA5, np.uint8)
            self.h[n + "_sb"] = np.full(lead + (2,), 0xA5A5, np.uint16)
            if poison:
                self.h[n + "_sb"][..., 0], self.h[n + "_sb"][..., 1] = 0x7FC0, 0xFF80
            x = raw(self.a[n + "_all"])
            for b, L in enumerate(cfg.lens):
                code, sb = kvq.quantise(x[first[b]:first[b] + L], cfg.bits)
                kvq.write_rows(self.h[n + "_q"], self.table[b], 0, kvq.pack(code, cfg.bits))
                kvq.write_rows(self.h[n + "_sb"], self.table[b], 0, sb)
        self.shape = lm.make_kvq_shape(cfg.B, cfg.H_q, cfg.H_kv, cfg.D, cfg.block_size, cfg.max_blocks, cfg.bits)
        self.n_query = n_query

    def to_gpu(self):
        self.t = {k: torch.from_numpy(v.view(np.int16) if v.dtype == np.uint16 else v).cuda() for k, v in self.h.items()}
        for n in "kv":
            self.t[n + "_sb"] = self.t[n + "_sb"].view(torch.bfloat16)
        self.d = {k: v.cuda() for k, v in self.a.items() if isinstance(v, torch.Tensor)}
        self.handle = lm.make_kvq_cache(self.t)
        self.ws = lm.alloc_kvq_workspace(self.shape, self.n_query)
        return self

    def status(self) -> int:
        return lm.lily_moe_device_status(self.ws)

    def sequence(self, b: int, count=None):
        """K, V and their magnitudes of one sequence, fp64 [L][H_kv][D]."""
        L = self.cfg.lens[b] if count is None else count
        got = []
        for f in (kvq.values, kvq.magnitudes):
            for n in "kv":
                got.append(f(kvq.rows_of(self.h[n + "_q"], self.table[b], 0, L),
                             kvq.rows_of(self.h[n + "_sb"], self.table[b], 0, L), self.cfg.bits))
        return got


def rounded(o: np.ndarray) -> np.ndarray:
    return kvq.bf16_value(raw(o) if isinstance(o, torch.Tensor) else o).astype(np.float64)


def error_bound(ref: np.ndarray, mags, operand: float) -> np.ndarray:
    """|o_gpu - o| per element, first order.

    The output is rounded to bf16: 2^-8 |o|.  A score is off by at most
    delta = score * (operand + 2^-18): `operand` is the relative rounding of a
    rebuilt key (0 where the codes themselves are multiplied), 2^-18 covers the
    fp32 sum over D <= 256 channels (64 sequential additions of 2^-24).  A weight is
    then off by a factor of at most e^(2 delta) (its own score and the
    normaliser's).  The weights are rounded to fp16 before they multiply the values
    (2^-11, and 2^-11 again in the normaliser where that is not rounded with them),
    and a rebuilt value by `operand`.
    """
    delta = mags["score"] * (operand + 2.0 ** -18)
    rel = np.expm1(2 * delta)[..., None] + 2 * 2.0 ** -11 + operand
    return (2.0 ** -8) * np.abs(ref) + rel * mags["value"] * (1 + 2.0 ** -8) + 1e-30


def check(got: np.ndarray, ref: np.ndarray, mags, operand: float = 2.0 ** -11):
    assert np.isfinite(got).all()
    err, bound = np.abs(got - ref), error_bound(ref, mags, operand)
    assert (err <= bound).all(), f"max err {err.max():.3e}, worst ratio {(err / bound).max():.3f}"
    # the 2-norm goes by the rounding of the output alone, up to a factor
    n = np.linalg.norm(ref)
    assert np.linalg.norm(got - ref) <= 5e-3 * n + 1e-30, np.linalg.norm(got - ref) / n
