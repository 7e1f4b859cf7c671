"""The ends of the documented ranges of the calls between the layers: what is inside is not refused, what is outside is, also from Python,
where sizes have more than 32 bits.  Nothing here touches a GPU: calls that pass the check of sizes are refused for a missing
array, and the library is a stand-in where a call would go through."""
import pytest
import torch

import bit_grouped_expert_top_gb300 as lm
from bit_grouped_expert_top_gb300 import _abi

FAKE = 0x10000000  # an aligned address that is never dereferenced


@pytest.mark.parametrize("D", [16, 48, 64, 80, 112, 256, 272, 496, 512])
def test_rope_takes_all_of_its_documented_range(D):
    """N * (H_q + H_k) * D < 2^34, with D that divides it and D that does not."""
    def call(N, H_q, H_k):
        return lm.load().lily_rope(_abi.lily_rope_shape(N, H_q, H_k, D, 16, 0), None, H_q * D, FAKE, H_k * D, FAKE, FAKE, 1.0, FAKE,
                                   H_q * D, FAKE, H_k * D, None)

    for heads in (1, 3, 16, 1000):
        most = (2 ** 34 - 1) // (D * heads)   # the largest N inside
        H_q, H_k = (heads + 1) // 2, heads // 2
        if most < 2 ** 31:
            assert call(most, H_q, H_k) == -1, (D, heads)       # goes on to q, which is missing
            assert call(most + 1, H_q, H_k) == -2, (D, heads)
    assert call(1, 2 ** 20 - 1, 0) == (-1 if (2 ** 20 - 1) * D < 2 ** 34 else -2)


# ------------------------------------------------------------------ sizes of more than 32 bits, from Python
class Array:
    """What the binding asks of a dense tensor, without its memory."""

    def __init__(self, *shape, dtype=torch.bfloat16):
        self.shape, self.dtype, self.device, self.is_cuda = torch.Size(shape), dtype, "cuda:0", True

    def stride(self, i=None):
        st = [1]
        for n in reversed(self.shape[1:]):
            st.insert(0, st[0] * n)
        return tuple(st) if i is None else st[i]

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return FAKE


class Library:
    """Takes the calls and keeps their shapes."""

    def __init__(self):
        self.shapes = []

    def __getattr__(self, name):
        def call(shape, *args):
            self.shapes.append(shape)
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(_abi, "_lib", lib)
    monkeypatch.setattr(_abi, "_current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(_abi, "_launch_stream", lambda stream, dev: None)
    return lib


BIG = 2 ** 32
I32, F32 = torch.int32, torch.float32


def _norm(N, H, d):
    x = Array(N, H, d)
    return lm.lily_rms_norm(x, None, y=x)


def _matvec(T, rows, K):
    w = lm.make_q4(Array(rows, K // 2, dtype=torch.uint8), Array(rows, K // 64), Array(rows, K // 64))
    return lm.lily_q4_matvec(w, Array(T, K), Array(T, rows))


def _rope(N, H_q, H_k, D, n):
    return lm.lily_rope(Array(N, H_q, D), Array(N, H_k, D), Array(N, dtype=I32), Array(n, dtype=torch.int64))


def _verify(B, N, V):
    return lm.lily_draft_verify(Array(N + B, V, dtype=F32), Array(N, V, dtype=F32), Array(N, dtype=I32), Array(B + 1, dtype=I32), Array(N, dtype=F32),
                                Array(B, dtype=F32), Array(B, dtype=I32), Array(N + B, dtype=I32), Array(256, dtype=torch.uint8))


CALLS = [(_norm, (4, 2, 64)), (_matvec, (4, 8, 128)), (_rope, (4, 2, 1, 64, 16)), (_verify, (3, 5, 100))]


@pytest.mark.parametrize("call,sizes", CALLS)
def test_the_stand_in_takes_calls(library, call, sizes):
    assert call(*sizes) == 0 and len(library.shapes) == 1


@pytest.mark.parametrize("call,sizes,at", [(c, s, i) for c, s in CALLS for i in range(len(s))])
@pytest.mark.parametrize("more", [-BIG // 2, 0, BIG * 7])
def test_sizes_beyond_32_bits_are_refused(library, call, sizes, at, more):
    """They would come out as other, smaller ones on the way into the library."""
    sizes = list(sizes)
    sizes[at] += BIG + more
    with pytest.raises(ValueError, match="32 bits"):
        call(*sizes)
    assert not library.shapes


def test_numbers_of_pairs_beyond_32_bits_are_refused():
    with pytest.raises(ValueError, match="32 bits"):
        lm.rope_frequencies(BIG + 64)
