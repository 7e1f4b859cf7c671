"""Seeded synthetic inputs for the quantised KV cache and the attention over it.

Like `attn_inputs.py`, this module only draws random numbers and lays them out:
it holds none of the quantisation or attention arithmetic.

Workload recipe: the full-attention layers of `attn_inputs.py` (16 query heads
over two KV heads, head size 256, blocks of 64 tokens, 32K to 128K tokens of
context), with K and V drawn N(0, 1) times a per-channel gain exp(N(0, 1/4)), as
the channels of rotated keys are of unlike size; q is N(0, 1).  The physical
blocks of a sequence are a seeded random permutation.
"""
from __future__ import annotations

from dataclasses import dataclass, replace
from typing import Dict, Optional, Tuple

import torch


@dataclass(frozen=True)
class KvqConfig:
    """Shape and seed of one workload: `lens` cached tokens per sequence, the last
    `new` of them written, read back or querying in the call (None: all)."""

    name: str
    lens: Tuple[int, ...]
    new: Optional[Tuple[int, ...]] = None
    H_q: int = 16
    H_kv: int = 2
    D: int = 256
    block_size: int = 64
    bits: int = 4
    seed: int = 0

    @property
    def B(self) -> int:
        return len(self.lens)

    @property
    def news(self) -> Tuple[int, ...]:
        return self.lens if self.new is None else self.new

    @property
    def N(self) -> int:
        return sum(self.news)

    @property
    def max_blocks(self) -> int:
        return max(max((L + self.block_size - 1) // self.block_size for L in self.lens), 1)

    def with_(self, **kw) -> "KvqConfig":
        return replace(self, **kw)


KVQ_CONFIGS: Dict[str, KvqConfig] = {
    # one token, a ragged block, several blocks: the oracle is instant
    "kvq_tiny": KvqConfig("kvq_tiny", lens=(1, 100, 777), new=(1, 1, 1), D=128, seed=21),
    # batch-1 decode at the context lengths of attn_inputs.py, and prompt chunks
    "kvq_32k": KvqConfig("kvq_32k", lens=(32768,), new=(1,), seed=22),
    "kvq_128k": KvqConfig("kvq_128k", lens=(131072,), new=(1,), seed=23),
    "kvq_prompt_8k": KvqConfig("kvq_prompt_8k", lens=(8192,), seed=24),
    "kvq_chunk_2k_32k": KvqConfig("kvq_chunk_2k_32k", lens=(32768,), new=(2048,), seed=25),
}


def make_kvq(cfg: KvqConfig, device="cpu", extra_blocks: int = 3) -> Dict[str, torch.Tensor]:
    """k_all / v_all [sum(lens)][H_kv][D] (bf16, the whole contexts, sequence by
    sequence), q [N][H_q][D], block_table [B][max_blocks] (-1 where unused),
    seq_lens, starts [B], cu [B+1] of the `new` tokens and cu_all [B+1] of all
    (int32), and n_blocks."""
    g = torch.Generator(device=device)
    g.manual_seed(7919 * (cfg.seed + 1))
    total, bs = sum(cfg.lens), cfg.block_size
    gain = torch.randn((2, cfg.H_kv, cfg.D), generator=g, device=device).mul_(0.5).exp_()
    out = {n: (torch.randn((total, cfg.H_kv, cfg.D), generator=g, device=device) * gain[i]).to(torch.bfloat16)
           for i, n in enumerate(("k_all", "v_all"))}
    out["q"] = torch.randn((cfg.N, cfg.H_q, cfg.D), generator=g, device=device).to(torch.bfloat16)
    need = [(L + bs - 1) // bs for L in cfg.lens]
    n_blocks = sum(need) + extra_blocks
    phys = torch.randperm(n_blocks, generator=g, device=device).to(torch.int32)
    table = torch.full((cfg.B, cfg.max_blocks), -1, dtype=torch.int32, device=device)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = phys[at:at + n]
        at += n

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=device)

    def ascending(v):
        return ints([sum(v[:b]) for b in range(len(v) + 1)])

    out.update(block_table=table, seq_lens=ints(cfg.lens), starts=ints([L - m for L, m in zip(cfg.lens, cfg.news)]),
               cu=ascending(cfg.news), cu_all=ascending(cfg.lens), zeros=ints([0] * cfg.B))
    out["n_blocks"] = n_blocks
    return out
