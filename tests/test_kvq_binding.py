"""The quantised-cache binding's check that a cache is of the shape that a call names: other heads, blocks or bits can have as
many bytes of codes, and fewer parameters than the kernels would read."""
import pytest
import torch

import bit_grouped_expert_top_gb300 as lm
from bit_grouped_expert_top_gb300 import _abi

FAKE = 0x10000000  # an aligned address that is never dereferenced
SHAPE = dict(B=2, H_q=4, H_kv=2, D=128, block_size=64, max_blocks=4, bits=4)
# as many bytes of codes a block
OTHERS = [dict(block_size=32, bits=8), dict(H_kv=4, block_size=32), dict(D=64, block_size=128), dict(D=64, bits=8), dict(H_kv=1, D=256)]


def _calls(s, cache, device):
    def t(*size, dtype=torch.bfloat16):
        return torch.zeros(size, dtype=dtype, device=device)

    n = t(4, dtype=torch.int32)
    table, ws = t(s.B, s.max_blocks, dtype=torch.int32), t(4096, dtype=torch.uint8)
    k, q = t(3, s.H_kv, s.D), t(s.B, s.H_q, s.D)
    return [lambda: lm.lily_kvq_append(s, cache, k, k, n, n, table, ws), lambda: lm.lily_kvq_read(s, cache, k, k, n, n, table, ws),
            lambda: lm.lily_kvq_attn_decode(s, cache, q, table, n, q, ws),
            lambda: lm.lily_kvq_attn_prefill(s, cache, q, n, table, n, q, ws)]


@pytest.mark.parametrize("kw", OTHERS)
def test_cache_of_another_layout_is_refused(kw):
    s, other = lm.make_kvq_shape(**SHAPE), lm.make_kvq_shape(**{**SHAPE, **kw})
    n_bytes = 10 * other.H_kv * other.D * other.block_size * other.bits // 8
    assert n_bytes == 10 * s.H_kv * s.D * s.block_size * s.bits // 8
    cache = _abi.lily_kvq_cache(FAKE, FAKE, FAKE, FAKE, 10, n_bytes)
    cache.block = (other.H_kv, other.D // 64, other.block_size, 8 * other.bits)
    for call in _calls(s, cache, "cpu"):
        with pytest.raises(ValueError, match="cache: blocks of"):
            call()
    cache.block = None   # a struct made by hand: nothing is known, the next check answers
    for call in _calls(s, cache, "cpu"):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("kw", OTHERS)
def test_cache_handle_knows_its_layout(kw):
    s, other = lm.make_kvq_shape(**SHAPE), lm.make_kvq_shape(**{**SHAPE, **kw})
    cache = lm.make_kvq_cache(lm.alloc_kvq_cache(other, 10))
    for call in _calls(s, cache, "cuda"):
        with pytest.raises(ValueError, match="cache: blocks of"):
            call()
