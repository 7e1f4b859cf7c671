"""Oracle of the quantised KV cache and of the attention over it (numpy).

TEST INFRASTRUCTURE ONLY, like the rest of this package.  The codes and
parameters are defined with fp32 arithmetic, so `quantise` is fp32 and its
results are compared bit for bit; everything after it is fp64.
"""
from __future__ import annotations

from typing import Dict, Optional, Tuple

import numpy as np

GROUP = 64


def bf16_round(x: np.ndarray) -> np.ndarray:
    """bf16 bit patterns of finite fp32 values, round to nearest even."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def bf16_value(bits: np.ndarray) -> np.ndarray:
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32)


def quantise(x_bits: np.ndarray, bits: int) -> Tuple[np.ndarray, np.ndarray]:
    """Codes uint8 [..., D/64, 64] and (scale, bias) bf16 bits [..., D/64, 2] of
    bf16 bits [..., D].  Halves of the values, so that no range overflows."""
    x = bf16_value(x_bits)
    x = x.reshape(x.shape[:-1] + (x.shape[-1] // GROUP, GROUP)) * np.float32(0.5)
    L = np.float32(2 ** bits - 1)
    lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
    scale = bf16_value(bf16_round((hi - lo) / (L * np.float32(0.5))))
    scale = np.where(scale < np.float32(2.0 ** -126), np.float32(0), scale)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.rint((x - lo) / (scale * np.float32(0.5)))
    c = np.where(scale > 0, np.minimum(c, L), 0).astype(np.uint8)
    sb = np.concatenate([bf16_round(scale), bf16_round(lo * np.float32(2))], -1)
    return c, sb


def pack(codes: np.ndarray, bits: int) -> np.ndarray:
    """Stored bytes [..., 8 bits] of codes [..., 64]: at 4 bits the even channel
    of each pair is the low nibble."""
    return codes if bits == 8 else (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(q: np.ndarray, bits: int) -> np.ndarray:
    if bits == 8:
        return q
    out = np.empty(q.shape[:-1] + (GROUP,), np.uint8)
    out[..., 0::2], out[..., 1::2] = q & 15, q >> 4
    return out


def values(q: np.ndarray, sb: np.ndarray, bits: int) -> np.ndarray:
    """code * scale + bias in fp64, [..., D], of stored bytes [..., D/64, 8 bits]."""
    p = bf16_value(sb).astype(np.float64)
    v = unpack(q, bits).astype(np.float64) * p[..., :1] + p[..., 1:]
    return v.reshape(v.shape[:-2] + (v.shape[-2] * GROUP,))


def magnitudes(q: np.ndarray, sb: np.ndarray, bits: int) -> np.ndarray:
    """code * |scale| + |bias|: what the rounding errors of a value go by."""
    p = np.abs(bf16_value(sb).astype(np.float64))
    v = unpack(q, bits).astype(np.float64) * p[..., :1] + p[..., 1:]
    return v.reshape(v.shape[:-2] + (v.shape[-2] * GROUP,))


def rows_of(cache: np.ndarray, table_row: np.ndarray, start: int, count: int) -> np.ndarray:
    """Rows [start, start + count) of one sequence: [count][H_kv][D/64][...]."""
    bs = cache.shape[3]
    pos = np.arange(start, start + count)
    return cache[table_row[pos // bs], :, :, pos % bs]


def write_rows(cache: np.ndarray, table_row: np.ndarray, start: int, rows: np.ndarray) -> None:
    bs = cache.shape[3]
    pos = np.arange(start, start + rows.shape[0])
    cache[table_row[pos // bs], :, :, pos % bs] = rows


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, limits: np.ndarray, scale: Optional[float] = None) -> np.ndarray:
    """o[n][h] = sum_{t < limits[n]} softmax_t(scale q[n][h] . k[t][g]) v[t][g], fp64:
    q [n][H_q][D], k and v [L][H_kv][D]; rows with no tokens give zeros."""
    return attend_and_bound(q, k, v, limits, scale)[0]


def attend_and_bound(q, k, v, limits, scale=None, k_mag=None, v_mag=None) -> Tuple[np.ndarray, Dict[str, np.ndarray]]:
    """attend(), and what error bounds go by, per query token and head: the largest
    scale * sum_d |q_d| k_mag_d over the tokens seen ("score"), and per output
    element sum_t w_t v_mag_t ("value")."""
    n, H_q, D = q.shape
    L, H_kv, _ = k.shape
    G = H_q // H_kv
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    out, val, sc = np.zeros((n, H_q, D)), np.zeros((n, H_q, D)), np.zeros((n, H_q))
    q = q.astype(np.float64)
    seen = np.arange(L)[None] < np.asarray(limits)[:, None]
    some = seen.any(1)
    if not some.any():
        return out, {"score": sc, "value": val}
    for h in range(H_q):
        g = h // G
        s = np.where(seen, scale * (q[:, h] @ k[:, g].T), -np.inf)
        m = np.where(some, s.max(1), 0.0)
        w = np.exp(s - m[:, None])
        w /= np.where(some, w.sum(1), 1.0)[:, None]
        out[:, h] = w @ v[:, g]
        if v_mag is not None:
            val[:, h] = w @ v_mag[:, g]
            sc[:, h] = np.where(seen, abs(scale) * (np.abs(q[:, h]) @ k_mag[:, g].T), 0.0).max(1)
    return out, {"score": sc, "value": val}
