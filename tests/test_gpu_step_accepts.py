"""The serving step with drafts of which some are accepted: the target's likeliest tokens, with random numbers on both sides of their
probability."""
import numpy as np
import pytest
import torch

import step_util as su
from test_gpu_serving_step import Step

pytestmark = pytest.mark.gpu


def likely_drafts(s, refused):
    """Drafts of a step that has run: the target's likeliest tokens, of which `refused` (by number) just fail."""
    rows = torch.tensor([sum(s.drafts[:b]) + b + i for b, m in enumerate(s.drafts) for i in range(m)], device="cuda")
    p, token = s.o["p"][rows].max(-1)
    s.tokens.copy_(token)
    s.u.copy_(p * 0.999)
    at = torch.tensor(refused, dtype=torch.long, device="cuda")
    s.u[at] = p[at]   # u = p is a refusal


def expected(s):
    return su.verify(*(t.cpu().numpy() if t is not None else None for t in (s.o["p"], None, s.tokens, s.cu_drafts, s.u, s.r)))


@pytest.mark.parametrize("drafts,past,refused,accepted", [
    ((2, 3, 0), (100, 7, 33), [], [2, 3, 0]), ((2, 3, 0), (100, 7, 33), [3], [2, 1, 0]), ((1, 1, 1, 1), (64, 1, 95, 31), [0, 2], [0, 1, 0, 1]),
    ((7,), (200,), [5], [5]), ((7,), (31,), [0, 1, 2, 3, 4, 5, 6], [0])])
def test_a_step_accepts_likely_drafts(drafts, past, refused, accepted):
    s = Step(drafts=drafts, past=past)
    s.run()
    likely_drafts(s, refused)
    p = s.o["p"].clone()
    s.run()
    assert s.status() == [0, 0, 0] and torch.equal(s.o["p"], p)   # the drafts' own rows do not go by the drafts here
    acc, tok = expected(s)
    assert acc.tolist() == accepted
    assert np.array_equal(s.o["acc"].cpu().numpy(), acc) and np.array_equal(s.o["tok"].cpu().numpy(), tok)


def test_a_graph_accepts_other_drafts_at_each_replay():
    s = Step()
    s.run()
    likely_drafts(s, [])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for refused, accepted in (([0], [0, 3, 0]), ([2, 4], [2, 0, 0]), ([4], [2, 2, 0]), ([], [2, 3, 0])):
        likely_drafts(s, refused)
        graph.replay()
        torch.cuda.synchronize()
        acc, tok = expected(s)
        assert acc.tolist() == accepted
        assert np.array_equal(s.o["acc"].cpu().numpy(), acc) and np.array_equal(s.o["tok"].cpu().numpy(), tok)
