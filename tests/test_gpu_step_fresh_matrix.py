"""A 4-bit product whose matrix a kernel of the same stream has just written, with a call of the library between them that lets
the product's kernel start early."""
import pytest
import torch

import bit_grouped_expert_top_gb300 as lm
import step_util as su

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


class Chain:
    """A writer of the codes, scales and biases, a norm of the tokens, the product of both."""

    def __init__(self, rows, K, T, by_library):
        g = torch.Generator().manual_seed(rows + K + T)
        self.by_library, half = by_library, K // 2
        self.source = torch.randn((rows, half // 2), generator=g).to(BF).cuda()
        self.params = torch.randn((rows, K // 64 * 8), generator=g).to(BF).cuda()
        self.x = torch.randn((T, K), generator=g).to(BF).cuda()
        self.q = torch.empty((rows, half), dtype=torch.uint8, device="cuda")
        self.scale, self.bias = (torch.empty((rows, K // 64), dtype=BF, device="cuda") for _ in "sb")
        self.y, self.out = torch.empty((T, K), dtype=BF, device="cuda"), torch.empty((T, rows), device="cuda")
        self.w = lm.make_q4(self.q, self.scale, self.bias)

    def write(self):
        if not self.by_library:
            self.q.copy_((self.source.abs() * 61).to(torch.uint8).repeat(1, 2))
        n = self.scale.shape[1]
        self.scale.copy_(self.params[:, :n] * 0.01)
        self.bias.copy_(self.params[:, n:2 * n] * 0.05)
        if self.by_library:   # any byte is two codes: a norm's output will do, and its kernel lets the next start at once
            lm.lily_rms_norm(self.source, None, y=self.q.view(BF), weight_offset=1.0)

    def norm(self):
        lm.lily_rms_norm(self.x, None, y=self.y, weight_offset=1.0)

    def product(self):
        lm.lily_q4_matvec(self.w, self.y, self.out)

    def change(self):
        self.source.mul_(-1.25).clamp_(-4, 4)
        self.params.neg_()
        self.x.mul_(-1)

    def run(self, wait=False):
        for f in (self.write, self.norm, self.product):
            f()
            if wait:
                torch.cuda.synchronize()


SIZES = [(4096, 2048, 1), (20000, 2048, 4), (2048, 4096, 12), (9000, 4224, 20), (3000, 2112, 32), (16384, 1024, 8)]


@pytest.mark.parametrize("by_library", [True, False])
@pytest.mark.parametrize("rows,K,T", SIZES)
def test_a_matrix_written_just_before(rows, K, T, by_library):
    c = Chain(rows, K, T, by_library)
    for _ in range(15):
        c.change()
        c.run(wait=True)
        want = c.out.clone()
        # another matrix, then the first again, with nothing between the writer and the product but the norm
        c.q.fill_(0x5A)
        c.scale.fill_(3.0)
        c.bias.fill_(-2.0)
        c.product()
        torch.cuda.synchronize()
        c.run()
        torch.cuda.synchronize()
        assert torch.equal(c.out, want)
    exact, bound = su.matvec(c.q, c.scale, c.bias, c.y)
    su.near(c.out, exact, bound * 2 + exact.abs() * 2.0 ** -20)


@pytest.mark.parametrize("rows,K,T", SIZES)
def test_a_matrix_written_in_a_graph(rows, K, T):
    c = Chain(rows, K, T, True)
    c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
        c.product()
    for _ in range(10):
        c.change()
        graph.replay()
        torch.cuda.synchronize()
        got = c.out.clone()
        c.run(wait=True)
        assert torch.equal(c.out, got)
