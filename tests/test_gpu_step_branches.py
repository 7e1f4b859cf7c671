"""Branches of the rotary positions and of the verification that are chosen by size: several heads a thread, clusters of one, two, four
and eight CTAs a sequence, CTAs of 512 and of 1,024 threads."""
import math

import numpy as np
import pytest
import torch

import bit_grouped_expert_top_gb300 as lm
import step_util as su

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


# ------------------------------------------------------------------ rotary positions
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("N,H_q,H_k,D,rot", [(8192, 16, 2, 256, 64), (8191, 5, 4, 128, 128), (20011, 3, 7, 64, 32)])
def test_rope_of_several_heads_a_thread(N, H_q, H_k, D, rot, interleaved):
    """More than three heads a thread, the last of the queries and the first of the keys among one thread's; each compared
    on a sample of the tokens, the rest against the same tokens alone (few heads a thread)."""
    g = torch.Generator().manual_seed(N)
    width = (H_q + 2 * H_k) * D
    fused = torch.randn((N, width), generator=g).to(BF).cuda()
    q, k = fused[:, :H_q * D].unflatten(-1, (H_q, D)), fused[:, H_q * D:(H_q + H_k) * D].unflatten(-1, (H_k, D))
    before, f = fused.clone(), lm.rope_frequencies(rot, 10000.0)
    table, pos = lm.make_rope_table(f), torch.randint(-1000000, 1000000, (N,), generator=g).to(torch.int32).cuda()
    qo, ko = torch.empty((N, H_q, D), dtype=BF, device="cuda"), torch.empty((N, H_k, D), dtype=BF, device="cuda")
    lm.lily_rope(q, k, pos, table, qo, ko, interleaved=interleaved)
    at = torch.cat([torch.arange(5), torch.arange(N - 5, N), torch.randint(0, N, (150,), generator=g)]).cuda()
    su.near(qo[at].cpu(), *su.rope(q[at], pos[at], f, interleaved))
    su.near(ko[at].cpu(), *su.rope(k[at], pos[at], f, interleaved))
    for n0 in range(0, N, 600):
        part = slice(n0, min(N, n0 + 600))
        few_q, few_k = torch.empty_like(qo[part]), torch.empty_like(ko[part])
        lm.lily_rope(q[part], k[part], pos[part].clone(), table, few_q, few_k, interleaved=interleaved)
        assert torch.equal(few_q, qo[part]) and torch.equal(few_k, ko[part])
    lm.lily_rope(q, k, pos, table, interleaved=interleaved)   # in place, in the slices
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(fused[:, (H_q + H_k) * D:], before[:, (H_q + H_k) * D:])


# ------------------------------------------------------------------ drafts
def _units(p):
    """p in units of 2^-62, rounded down: at most 2^62, and exact in fp64 (24 bits)."""
    p = np.nan_to_num(np.clip(p.astype(np.float64), 0.0, 1.0), nan=0.0)
    return np.floor(np.ldexp(p, 62)).astype(np.uint64)


def _expected(p, q, drafts, cu, u, r):
    """As step_util.verify, on whole rows at once: rows sum to about 2^62, so 64 bits hold the sums."""
    accepted, tokens = [], []
    for b in range(len(r)):
        c0, m = int(cu[b]), int(cu[b + 1] - cu[b])
        n = 0
        while n < m and float(u[c0 + n]) * (1.0 if q is None else float(q[c0 + n, drafts[c0 + n]])) < float(p[c0 + b + n, drafts[c0 + n]]):
            n += 1
        whole = _units(p[c0 + b + n])
        w = whole.copy()
        if n < m and q is None:
            w[drafts[c0 + n]] = 0
        elif n < m:
            other = _units(q[c0 + n])
            w = np.where(w > other, w - np.minimum(other, w), np.uint64(0))
        w = w if w.any() else whole
        upto = np.cumsum(w)
        below = int(upto[-1]) * int(math.ldexp(float(r[b]), 64)) >> 64
        accepted.append(n)
        tokens += [int(t) for t in drafts[c0:c0 + n]] + [int(np.searchsorted(upto, np.uint64(below), side="right"))] + [-1] * (m - n)
    return np.array(accepted, np.int32), np.array(tokens, np.int32)


def _case(lens, V, seed, draft):
    N, B = sum(lens), len(lens)
    g = torch.Generator(device="cuda").manual_seed(seed)
    p = torch.softmax(2.0 * torch.randn((N + B, V), generator=g, device="cuda"), -1)
    rows = torch.tensor([sum(lens[:b]) + b + i for b in range(B) for i in range(lens[b])], dtype=torch.long, device="cuda")
    q = torch.softmax((p[rows] + 1e-30).log() + 0.5 * torch.randn((N, V), generator=g, device="cuda"), -1) if draft else None
    x = torch.multinomial(q if draft else p[rows], 1, generator=g)[:, 0].to(torch.int32) if N else torch.zeros(0, dtype=torch.int32, device="cuda")
    cu = torch.tensor([sum(lens[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
    u = torch.rand(N, generator=g, device="cuda")
    if not draft:
        u[::2] *= 0.5 * p[rows, x.long()][::2]  # some that are accepted
    return p, q, x, cu, u, torch.rand(B, generator=g, device="cuda")


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("B,V", [
    # 8, 4, 2 and 1 CTAs a sequence, on both sides of each change, few tokens and many
    (19, 130), (20, 131), (24, 1001), (38, 257), (39, 5003), (64, 999), (76, 33), (77, 1500), (100, 515), (152, 64), (153, 2003),
    # 1,024 threads: 8, 4, 2 and 1 CTAs a sequence with 32,768 tokens each, and one less
    (1, 262147), (2, 262143), (9, 300007), (24, 131075), (24, 131071), (40, 65539), (64, 131072), (40, 65535), (80, 32771), (80, 32767), (160, 40009)])
def test_verify_of_each_number_of_ctas(B, V, draft):
    lens = [(3 * b + b // 4) % 5 for b in range(B)] if B > 1 else [3]
    case = _case(lens, V, B + V, draft)
    want = _expected(*(None if t is None else t.cpu().numpy() for t in case))
    acc, tok = (torch.full((n + 8,), -77, dtype=torch.int32, device="cuda") for n in (B, sum(lens) + B))
    ws = lm.alloc_draft_workspace()
    lm.lily_draft_verify(*case, acc[:B], tok[:sum(lens) + B], ws)
    assert lm.lily_moe_device_status(ws) == 0
    acc, tok = acc.cpu().numpy(), tok.cpu().numpy()
    assert (acc[B:] == -77).all() and (tok[sum(lens) + B:] == -77).all()
    assert np.array_equal(acc[:B], want[0]) and np.array_equal(tok[:sum(lens) + B], want[1])
    if B > 20:
        assert 0 < want[0].sum() < sum(lens)  # accepted and refused ones


def test_the_oracles_of_the_verification_agree():
    for draft in (True, False):
        case = [None if t is None else t.cpu().numpy() for t in _case([2, 0, 3, 1], 203, 5, draft)]
        for a, b in zip(_expected(*case), su.verify(*case)):
            assert np.array_equal(a, b)
