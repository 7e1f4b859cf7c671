"""One serving step of drafted tokens, as a program makes it of the library's calls: norm, projection, norms of the heads, rotary
positions, quantised cache, attention, projection, norm, expert layer, norm, logits, verification.  Each of the operators
between the attention and the expert layer is checked on what the step really hands it."""
import numpy as np
import pytest
import torch

import bit_grouped_expert_top_gb300 as lm
import step_util as su
from bit_grouped_expert_top_gb300.inputs import CONFIGS
from gpu_util import Layer, shape_of

pytestmark = pytest.mark.gpu
BF, F32, F8, I32 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32


class Step:
    """Weights, cache and buffers of a step of B sequences with m drafts each (m + 1 tokens a sequence, 8 in all)."""

    H_q, H_kv, D, bs, rot, V = 4, 2, 128, 32, 64, 1003

    def __init__(self, drafts=(2, 3, 0), past=(100, 7, 33)):
        g = torch.Generator().manual_seed(11)
        cfg = CONFIGS["tiny"]
        self.d, self.drafts, self.past = cfg.d, drafts, past
        self.N, self.B = sum(drafts) + len(drafts), len(drafts)
        d, D, n, B = cfg.d, self.D, self.N, self.B

        def rand(*size, by=1.0, dtype=BF):
            return (torch.randn(size, generator=g) * by).to(dtype).cuda()

        def ints(v):
            return torch.tensor(v, dtype=I32, device="cuda")

        self.layer = Layer(cfg)
        self.moe, self.moe_ws = shape_of(cfg, n), None
        self.moe_ws = lm.alloc_workspace(self.moe, n_layers_decode=1)
        self.parts = {"qkv": su.make_matrix((self.H_q + 2 * self.H_kv) * D, d, seed=1), "o": su.make_matrix(d, self.H_q * D, seed=2),
                      "head": su.make_matrix(self.V, d, seed=3)}
        self.w = {k: lm.make_q4(*v) for k, v in self.parts.items()}
        self.norms = {k: rand(s, by=0.2) for k, s in (("in", d), ("q", D), ("k", D), ("moe", d), ("out", d))}
        self.table_f = lm.rope_frequencies(self.rot, 1e6)
        self.table = lm.make_rope_table(self.table_f)
        news = [m + 1 for m in drafts]
        blocks = [(p + m + self.bs - 1) // self.bs for p, m in zip(past, news)]
        self.kvq = lm.make_kvq_shape(B, self.H_q, self.H_kv, D, self.bs, max(blocks), 8)
        self.cache_t = lm.alloc_kvq_cache(self.kvq, sum(blocks))
        self.cache, self.kvq_ws = lm.make_kvq_cache(self.cache_t), lm.alloc_kvq_workspace(self.kvq, n)
        table = torch.zeros((B, max(blocks)), dtype=I32)
        for b in range(B):
            table[b, :blocks[b]] = torch.arange(blocks[b]) + sum(blocks[:b])
        self.blocks = table.cuda()
        # the past: random keys and values
        old = sum(past)
        lm.lily_kvq_append(self.kvq, self.cache, rand(old, self.H_kv, D), rand(old, self.H_kv, D), ints([sum(past[:b]) for b in range(B + 1)]),
                           ints([0] * B), self.blocks, self.kvq_ws)
        self.cu = ints([sum(news[:b]) for b in range(B + 1)])
        self.starts, self.lens = ints(list(past)), ints([p + m for p, m in zip(past, news)])
        self.positions = ints([p + i for p, m in zip(past, news) for i in range(m)])
        self.cu_drafts = ints([sum(drafts[:b]) for b in range(B + 1)])
        self.hidden = rand(n, d, by=2.0)
        self.tokens = torch.randint(0, self.V, (sum(drafts),), generator=g).to(I32).cuda()
        self.u, self.r = torch.rand(sum(drafts), generator=g).cuda(), torch.rand(B, generator=g).cuda()
        e = lambda *s, dtype=BF: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        self.o = {"y8": e(n, d, dtype=F8), "s8": e(n, d // 64, dtype=F32), "qkv": e(n, (self.H_q + 2 * self.H_kv) * D), "qn": e(n, self.H_q, D),
                  "kn": e(n, self.H_kv, D), "q": e(n, self.H_q, D), "k": e(n, self.H_kv, D), "att": e(n, self.H_q, D), "proj": e(n, d),
                  "h1": e(n, d), "x": e(n, d), "moe": e(1, n, d, dtype=F32), "h2": e(n, d), "y": e(n, d), "logits": e(n, self.V, dtype=F32),
                  "p": e(n, self.V, dtype=F32), "acc": e(B, dtype=I32), "tok": e(n, dtype=I32)}
        self.ver_ws = lm.alloc_draft_workspace()

    def run(self):
        o, D, H, K = self.o, self.D, self.H_q, self.H_kv
        lm.lily_rms_norm(self.hidden, self.norms["in"], y8=o["y8"], y8_scale=o["s8"], weight_offset=1.0)
        lm.lily_q4_matvec(self.w["qkv"], o["y8"], o["qkv"], x_scale=o["s8"])
        q, k, v = (t.unflatten(-1, (-1, D)) for t in o["qkv"].split([H * D, K * D, K * D], -1))
        lm.lily_rms_norm(q, self.norms["q"], y=o["qn"], weight_offset=1.0)
        lm.lily_rms_norm(k, self.norms["k"], y=o["kn"], weight_offset=1.0)
        lm.lily_rope(o["qn"], o["kn"], self.positions, self.table, o["q"], o["k"])
        lm.lily_kvq_append(self.kvq, self.cache, o["k"], v, self.cu, self.starts, self.blocks, self.kvq_ws)
        lm.lily_kvq_attn_prefill(self.kvq, self.cache, o["q"], self.cu, self.blocks, self.lens, o["att"], self.kvq_ws)
        lm.lily_q4_matvec(self.w["o"], o["att"].flatten(1), o["proj"])
        lm.lily_rms_norm(o["proj"], self.norms["moe"], y=o["x"], residual=self.hidden, h=o["h1"], weight_offset=1.0)
        lm.lily_moe_decode(self.moe, [self.layer.w], o["x"], o["moe"], self.moe_ws)
        lm.lily_rms_norm(o["moe"][0], self.norms["out"], y=o["y"], residual=o["h1"], h=o["h2"], weight_offset=1.0)
        lm.lily_q4_matvec(self.w["head"], o["y"], o["logits"])
        torch.softmax(o["logits"], -1, out=o["p"])
        lm.lily_draft_verify(o["p"], None, self.tokens, self.cu_drafts, self.u, self.r, o["acc"], o["tok"], self.ver_ws)

    def status(self):
        return [lm.lily_moe_device_status(ws) for ws in (self.moe_ws, self.kvq_ws, self.ver_ws)]


def _matvec(got, parts, x, scale=None):
    want, bound = su.matvec(*parts, x, scale)
    su.near(got, want, bound + (want.abs() + bound) * su.U[got.dtype] + su.TINY[got.dtype])


def test_a_serving_step():
    s = Step()
    s.run()
    o, D, H, K = s.o, s.D, s.H_q, s.H_kv
    assert s.status() == [0, 0, 0]
    w = s.norms
    su.check_norm(su.norm(s.hidden, w["in"], 1.0, 1e-6), y8=o["y8"], y8_scale=o["s8"])
    _matvec(o["qkv"], s.parts["qkv"], o["y8"], o["s8"])
    q, k, _ = (t.unflatten(-1, (-1, D)) for t in o["qkv"].split([H * D, K * D, K * D], -1))
    su.check_norm(su.norm(q, w["q"], 1.0, 1e-6), y=o["qn"])
    su.check_norm(su.norm(k, w["k"], 1.0, 1e-6), y=o["kn"])
    for n in "qk":
        su.near(o[n].cpu(), *su.rope(o[n + "n"], s.positions, s.table_f, False))
    _matvec(o["proj"], s.parts["o"], o["att"].flatten(1))
    su.check_norm(su.norm(o["proj"], w["moe"], 1.0, 1e-6, s.hidden), h=o["h1"], y=o["x"])
    su.check_norm(su.norm(o["moe"][0], w["out"], 1.0, 1e-6, o["h1"]), h=o["h2"], y=o["y"])
    _matvec(o["logits"], s.parts["head"], o["y"])
    acc, tok = su.verify(*(t.cpu().numpy() if t is not None else None for t in (o["p"], None, s.tokens, s.cu_drafts, s.u, s.r)))
    assert np.array_equal(o["acc"].cpu().numpy(), acc) and np.array_equal(o["tok"].cpu().numpy(), tok)
    assert all(bool(torch.isfinite(t.float()).all()) for t in o.values())


def test_the_whole_step_in_a_graph():
    s = Step(drafts=(1, 1, 1, 1), past=(64, 1, 95, 31))
    s.run()
    torch.cuda.synchronize()
    want = {n: t.clone() for n, t in s.o.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for _ in range(2):
        for t in s.o.values():
            t.view(torch.uint8).zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t.view(torch.uint8), want[n].view(torch.uint8)) for n, t in s.o.items())
    # other inputs of the same sizes, the same graph
    s.hidden.copy_(torch.randn_like(s.hidden))
    graph.replay()
    torch.cuda.synchronize()
    got = {n: t.clone() for n, t in s.o.items()}
    s.run()
    torch.cuda.synchronize()
    assert s.status() == [0, 0, 0]
    assert not torch.equal(got["logits"], want["logits"])
    assert all(torch.equal(t.view(torch.uint8), got[n].view(torch.uint8)) for n, t in s.o.items())
