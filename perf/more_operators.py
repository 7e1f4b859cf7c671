"""What lies between the attention and the expert layers in a serving step of drafted tokens: what a call does, in plain
torch operations and through the library, on the sizes that serving meets.

"norm": root-mean-square norm of a hidden state with the residual's addition; output in bf16, in e4m3 codes with a scale for
each group of 64 channels, or both.  "matvec": a few tokens times a matrix of 4-bit codes with (scale, bias) for each group
of 64; tokens in bf16 or in the norm's 8-bit form.  "rope": rotary positions on queries and keys, half and interleaved
pairs, on a part of the head or all of it, frequencies scaled for long contexts.  "verify": drafted tokens accepted or refused against the target's
probabilities from given random numbers, and the token that follows them.
"""
import math

import torch

own = False

GROUP = 64
EPS = 1e-6


def listed():
    return [
        # one step of eight tokens: the expert layer's fp32 output joins the residual, the next projection reads 8 bits
        {"name": "norm_step", "op": "norm", "N": 8, "H": 1, "d": 2048, "x": "f32", "h": "bf16", "out": "codes", "pad": 0},
        # a whole prompt between two layers, both outputs (the expert layer reads bf16)
        {"name": "norm_prompt", "op": "norm", "N": 8192, "H": 1, "d": 2048, "x": "f32", "h": "bf16", "out": "both", "pad": 0},
        # the query heads of a chunk, normalised one by one as they lie in a fused projection's output
        {"name": "norm_heads", "op": "norm", "N": 2049, "H": 16, "d": 256, "x": "bf16", "h": "none", "out": "y", "pad": 1024},
        # the fused query/key/value projection of one token
        {"name": "matvec_one", "op": "matvec", "T": 1, "rows": 5120, "K": 2048, "x": "bf16", "out": "bf16"},
        # the projection after attention, eight tokens in 8 bits
        {"name": "matvec_codes", "op": "matvec", "T": 8, "rows": 2048, "K": 4096, "x": "codes", "out": "bf16"},
        # a vocabulary's logits of four tokens, an odd number of rows
        {"name": "matvec_head", "op": "matvec", "T": 4, "rows": 130001, "K": 2048, "x": "bf16", "out": "f32"},
        # the same for eight sequences of four tokens
        {"name": "matvec_drafts", "op": "matvec", "T": 32, "rows": 65536, "K": 2048, "x": "bf16", "out": "f32"},
        # one step of eight tokens: a quarter of the head turns
        {"name": "rope_step", "op": "rope", "N": 8, "H_q": 16, "H_k": 2, "D": 256, "rot": 64, "pairs": "half", "scaling": "none", "far": 32768},
        # a whole prompt
        {"name": "rope_prompt", "op": "rope", "N": 8192, "H_q": 16, "H_k": 2, "D": 256, "rot": 64, "pairs": "half", "scaling": "none", "far": 8192},
        # a ragged chunk at the far end of a scaled context, the whole head, neighbouring pairs
        {"name": "rope_far", "op": "rope", "N": 1001, "H_q": 8, "H_k": 8, "D": 128, "rot": 128, "pairs": "next", "scaling": "parts", "far": 1000000},
        # eight conversations with up to five drafts each, an odd vocabulary
        {"name": "verify_step", "op": "verify", "drafts": "4,4,0,5,1,4,3,4", "V": 100003, "q": True},
        # a batch whose drafts were looked up in the text, so that no draft distribution exists
        {"name": "verify_lookup", "op": "verify", "drafts": ",".join(["3"] * 64), "V": 131072, "q": False},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "matvec", "rope", "verify"])
    if op == "norm":
        out = rng.choice(["y", "codes", "both"])
        step = 64 if out != "y" else 8
        d = min(16384, step * log(1 if step == 64 else 4, 16384 // step))
        H = rng.choice([1, 1, 1, 2, 5, 16]) if d <= 512 else 1
        N = log(1, max(1, 8192 * 2048 // (H * d)))
        h = "none" if H > 1 else rng.choice(["bf16", "f32", "none"])
        return {"op": op, "N": N, "H": H, "d": d, "x": rng.choice(["f32", "bf16"]), "h": h, "out": out, "pad": rng.choice([0, 0, 8, 1024])}
    if op == "matvec":
        T, K = log(1, 32), 64 * log(1, 256)
        rows = log(1, max(1, min(262144, 65536 * 2048 // K)))
        return {"op": op, "T": T, "rows": rows, "K": K, "x": rng.choice(["bf16", "codes"]), "out": rng.choice(["bf16", "f32"])}
    if op == "rope":
        D = rng.choice([64, 128, 256])
        H_q, H_k = rng.choice([(16, 2), (8, 8), (6, 3), (1, 1), (4, 0), (5, 1)])
        return {"op": op, "N": log(1, 8192 * 18 * 256 // ((H_q + H_k) * D)), "H_q": H_q, "H_k": H_k, "D": D,
                "rot": rng.choice([D, D // 2, D // 4, 16 * rng.randint(1, D // 16)]), "pairs": rng.choice(["half", "next"]),
                "scaling": rng.choice(["none", "linear", "base", "parts"]), "far": log(1, 1000000)}
    B = log(1, 64)
    drafts = [rng.randint(0, 8) for _ in range(B)]
    V = log(2, min(200000, 131072 * 64 // (2 * B)))
    return {"op": op, "drafts": ",".join(map(str, drafts)), "V": V, "q": rng.random() < 0.7}


def _ints(text):
    return [int(x) for x in text.split(",")]


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the plain form
def _codes(y):
    """e4m3 codes [..., d] and fp32 scales [..., d / 64] of y [..., d] in fp32."""
    g = y.unflatten(-1, (-1, GROUP))
    most = g.abs().amax(-1, keepdim=True)
    some = most >= 2.0 ** -100
    inverse = torch.where(some, 448.0 / torch.where(some, most, 1.0), 0.0)
    scale = torch.where(some, most * (1.0 / 448.0), 0.0)
    return (g * inverse).flatten(-2).to(torch.float8_e4m3fn), scale.squeeze(-1)


def _norm(s):
    h = s["x"].float()
    outs = []
    if s["residual"] is not None:
        h = h + s["residual"].float()
        outs.append(h.to(s["residual"].dtype))
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * (s["weight"].float() + 1.0)
    if s["out"] != "codes":
        outs.append(y.to(torch.bfloat16))
    if s["out"] != "y":
        outs.extend(_codes(y))
    return tuple(outs)


def _matrix(s):
    code = torch.stack([s["w_q"] & 15, s["w_q"] >> 4], -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    return (code * s["w_scale"].float()[..., None] + s["w_bias"].float()[..., None]).flatten(-2)


def _matvec(s):
    x = s["x"].float()
    if s["x_scale"] is not None:
        x = (x.unflatten(-1, (-1, GROUP)) * s["x_scale"][..., None]).flatten(-2)
    return (x @ _matrix(s).T).to(_TYPES[s["out"]])


def _frequencies(rot, theta, scaling, factor, original):
    """Angle of each pair a position, in 64 bits."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    if scaling == "base":
        theta = theta * factor ** (rot / (rot - 2)) if rot > 2 else theta
    f = theta ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "parts":  # turns over the original context: few are stretched, many are left
        keep = ((original * f / (2.0 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / factor)
    return f


def _turned(x, cos, sin, pairs):
    n = 2 * cos.shape[-1]
    a, b = (x[..., :n // 2], x[..., n // 2:n]) if pairs == "half" else (x[..., 0:n:2], x[..., 1:n:2])
    a, b = a.float(), b.float()
    a, b = a * cos - b * sin, a * sin + b * cos
    head = torch.cat([a, b], -1) if pairs == "half" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([head.to(x.dtype), x[..., n:]], -1)


def _rope(s):
    f = _frequencies(s["rot"], *s["rule"])
    angle = s["positions"].double()[:, None, None] * f
    cos, sin = (angle.cos() * s["amplitude"]).float(), (angle.sin() * s["amplitude"]).float()
    return tuple(_turned(s[n], cos, sin, s["pairs"]) for n in ("q", "k") if s[n] is not None)


def _verify(s):
    p, q, cu, B, N = s["p"], s["q"], s["cu"].long(), s["B"], s["N"]
    b = torch.searchsorted(cu[1:], torch.arange(N, device="cuda"), right=True)  # sequence of each draft
    i = torch.arange(N, device="cuda") - cu[b]
    x = s["drafts"].long()
    px = p[cu[b] + b + i, x].double()
    qx = torch.ones_like(px) if q is None else q[torch.arange(N, device="cuda"), x].double()
    refused = ~(s["u"].double() * qx < px)
    m = cu[1:] - cu[:-1]
    n = m.scatter_reduce(0, b, torch.where(refused, i, m[b]), "amin")
    # the token that follows: from what the target has beyond the draft, or, all accepted, from the target
    seq = torch.arange(B, device="cuda")
    w = p[cu[:-1] + seq + n].double()
    more = n < m
    at = torch.where(more, cu[:-1] + n, 0).clamp_max(max(N - 1, 0))
    if N and q is None:
        w[seq, x[at]] = torch.where(more, 0.0, w[seq, x[at]])
    elif N:
        rest = (w - q[at].double()).clamp_min(0.0)
        w = torch.where((more & (rest.sum(-1) > 0))[:, None], rest, w)
    upto = w.cumsum(-1)
    token = (upto <= (s["r"].double() * upto[:, -1])[:, None]).sum(-1)
    out = torch.full((N + B,), -1, dtype=torch.int32, device="cuda")
    out[cu[b] + b + i] = torch.where(i < n[b], s["drafts"], -1)
    out[cu[:-1] + seq + n] = token.to(torch.int32)
    return n.to(torch.int32), out


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    c = {k: v for k, v in case.items() if k != "name"}
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*size):
        return torch.randn(size, generator=g, device="cuda")

    if c["op"] == "norm":
        N, H, d = c["N"], c["H"], c["d"]
        # hidden states have a few channels far larger than the rest
        gain = normal(d).mul_(0.7).exp_()
        x = torch.empty((N, H * d + c["pad"]), dtype=_TYPES[c["x"]], device="cuda")
        x.copy_(normal(N, H * d + c["pad"]))
        x = x[:, :H * d].unflatten(-1, (H, d))
        x.mul_(gain.to(x.dtype))
        x = x[:, 0] if H == 1 else x
        weight = normal(d).mul_(0.2).to(torch.bfloat16)  # around zero: the channel's factor is 1 + weight
        residual = None if c["h"] == "none" else (3 * normal(N, d)).to(_TYPES[c["h"]])
        s = {**c, "x": x, "weight": weight, "residual": residual}
        if residual is not None:
            s["h_out"] = torch.empty_like(residual)
        if c["out"] != "codes":
            s["y"] = torch.empty(x.shape, dtype=torch.bfloat16, device="cuda")
        if c["out"] != "y":
            s["y8"] = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda")
            s["y8_scale"] = torch.empty(x.shape[:-1] + (d // GROUP,), dtype=torch.float32, device="cuda")
        return s
    if c["op"] == "matvec":
        T, rows, K = c["T"], c["rows"], c["K"]
        w_q = torch.randint(0, 256, (rows, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        w_scale = (0.01 + 0.01 * torch.rand((rows, K // GROUP), generator=g, device="cuda")).to(torch.bfloat16)
        w_bias = (-7.5 * w_scale.float() + 0.01 * normal(rows, K // GROUP)).to(torch.bfloat16)
        x, x_scale = normal(T, K) * normal(K).mul_(0.5).exp_(), None
        x, x_scale = _codes(x) if c["x"] == "codes" else (x.to(torch.bfloat16), None)
        return {**c, "w_q": w_q, "w_scale": w_scale, "w_bias": w_bias, "x": x, "x_scale": x_scale,
                "y": torch.empty((T, rows), dtype=_TYPES[c["out"]], device="cuda")}
    if c["op"] == "rope":
        N, H_q, H_k, D = c["N"], c["H_q"], c["H_k"], c["D"]
        # slices of a fused projection's output
        fused = normal(N, (H_q + 2 * H_k) * D).to(torch.bfloat16)
        q = fused[:, :H_q * D].unflatten(-1, (H_q, D))
        k = fused[:, H_q * D:(H_q + H_k) * D].unflatten(-1, (H_k, D)) if H_k else None
        positions = (torch.arange(N, device="cuda") + max(0, c["far"] - N)).to(torch.int32)
        return {**c, "q": q, "k": k, "positions": positions, "amplitude": 1.2 if c["scaling"] == "parts" else 1.0,
                "rule": (1000000.0, c["scaling"], 8.0, 32768.0),
                "q_out": torch.empty((N, H_q, D), dtype=torch.bfloat16, device="cuda"),
                "k_out": torch.empty((N, H_k, D), dtype=torch.bfloat16, device="cuda") if H_k else None}
    drafts, V = _ints(c["drafts"]), c["V"]
    B, N = len(drafts), sum(drafts)
    cu = torch.tensor([sum(drafts[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
    # distributions with a few likely tokens; a draft model that is near the target
    logits = 2.5 * normal(N + B, V)
    p = torch.softmax(logits, -1)
    b = torch.searchsorted(cu[1:].long(), torch.arange(N, device="cuda"), right=True)
    q = torch.softmax(logits[torch.arange(N, device="cuda") + b] + 0.5 * normal(N, V), -1)
    del logits
    x = ((q if c["q"] else p[torch.arange(N, device="cuda") + b]).cumsum(-1) < torch.rand((N, 1), generator=g, device="cuda")).sum(-1)
    return {**c, "B": B, "N": N, "cu": cu, "p": p, "q": q if c["q"] else None, "drafts": x.clamp_max(V - 1).to(torch.int32),
            "u": torch.rand(N, generator=g, device="cuda"), "r": torch.rand(B, generator=g, device="cuda"),
            "accepted": torch.empty(B, dtype=torch.int32, device="cuda"),
            "tokens": torch.empty(N + B, dtype=torch.int32, device="cuda")}


# ---------------------------------------------------------------- the calls
def _through_the_library(s):
    import bit_grouped_expert_top_gb300 as lm

    op = s["op"]
    if op == "norm":
        lm.lily_rms_norm(s["x"], s["weight"], y=s.get("y"), y8=s.get("y8"), y8_scale=s.get("y8_scale"), residual=s["residual"],
                         h=s.get("h_out"), eps=EPS, weight_offset=1.0)
        return tuple(s[n] for n in ("h_out", "y", "y8", "y8_scale") if n in s)
    if op == "matvec":
        if "matrix" not in s:  # what a program sets up once
            s["matrix"] = lm.make_q4(s["w_q"], s["w_scale"], s["w_bias"])
        lm.lily_q4_matvec(s["matrix"], s["x"], s["y"], x_scale=s["x_scale"])
        return s["y"]
    if op == "rope":
        if "table" not in s:
            theta, scaling, factor, original = s["rule"]
            f = lm.rope_frequencies(s["rot"], theta, scaling, factor=factor, original=original, low=1.0, high=32.0)
            s["table"] = lm.make_rope_table(f)
        lm.lily_rope(s["q"], s["k"], s["positions"], s["table"], s["q_out"], s["k_out"], interleaved=s["pairs"] == "next",
                     amplitude=s["amplitude"])
        return (s["q_out"],) if s["k"] is None else (s["q_out"], s["k_out"])
    if "ws" not in s:
        s["ws"] = lm.alloc_draft_workspace()
    lm.lily_draft_verify(s["p"], s["q"], s["drafts"], s["cu"], s["u"], s["r"], s["accepted"], s["tokens"], s["ws"])
    return s["accepted"], s["tokens"]


def run(state):
    return _through_the_library(state) if own else {"norm": _norm, "matvec": _matvec, "rope": _rope, "verify": _verify}[state["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "norm":
        n, d = case["N"] * case["H"] * case["d"], case["d"]
        size = {"bf16": 2, "f32": 4, "none": 0}
        outs = {"y": 2.0, "codes": 1 + 4 / GROUP, "both": 3 + 4 / GROUP}[case["out"]]
        return {"bytes": int(n * (size[case["x"]] + 2 * size[case["h"]] + outs)) + 2 * d, "flops": 6 * n}
    if case["op"] == "matvec":
        T, rows, K = case["T"], case["rows"], case["K"]
        x = T * K * 2 if case["x"] == "bf16" else T * (K + K // GROUP * 4)
        return {"bytes": rows * (K // 2 + K // GROUP * 4) + x + T * rows * (2 if case["out"] == "bf16" else 4), "flops": 2 * T * rows * K}
    if case["op"] == "rope":
        n = case["N"] * (case["H_q"] + case["H_k"])
        return {"bytes": n * case["D"] * 4 + case["N"] * 4, "flops": 3 * n * case["rot"]}
    drafts, V = _ints(case["drafts"]), case["V"]
    rows = len(drafts) + (sum(m > 0 for m in drafts) if case["q"] else 0)
    return {"bytes": rows * V * 4 + sum(drafts) * 20 + len(drafts) * 16, "flops": 2 * rows * V}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "norm":
        h = s["x"].double()
        outs = []
        if s["residual"] is not None:
            h = h + s["residual"].double()
            outs.append(h)
        y = h / torch.sqrt((h * h).sum(-1, keepdim=True) / s["d"] + EPS) * (1 + s["weight"].double())
        if s["out"] != "codes":
            outs.append(y)
        if s["out"] != "y":
            by_group = y.reshape(*y.shape[:-1], -1, GROUP)
            scale = by_group.abs().max(-1).values / 448
            outs += [(by_group / scale[..., None]).reshape(y.shape), scale]
        return tuple(outs)
    if s["op"] == "matvec":
        x = s["x"].double()
        if s["x_scale"] is not None:
            x = x * s["x_scale"].double().repeat_interleave(GROUP, -1)
        out = torch.empty((s["T"], s["rows"]), dtype=torch.float64, device="cuda")
        for a in range(0, s["rows"], 16384):
            q = s["w_q"][a:a + 16384].to(torch.int64)
            w = torch.empty((len(q), s["K"]), dtype=torch.float64, device="cuda")
            w[:, 0::2], w[:, 1::2] = q % 16, q // 16
            w *= s["w_scale"][a:a + 16384].double().repeat_interleave(GROUP, -1)
            w += s["w_bias"][a:a + 16384].double().repeat_interleave(GROUP, -1)
            out[:, a:a + 16384] = x @ w.T
        return out
    if s["op"] == "rope":
        rot, (theta, scaling, factor, original) = s["rot"], s["rule"]
        angles = []
        for i in range(rot // 2):
            f = theta ** (-2 * i / rot)
            if scaling == "linear":
                f /= factor
            if scaling == "base" and rot > 2:
                f = (theta * factor ** (rot / (rot - 2))) ** (-2 * i / rot)
            if scaling == "parts":
                turns = original * f / (2 * math.pi)
                part = min(1.0, max(0.0, (turns - 1) / 31))
                f = (1 - part) * f / factor + part * f
            angles.append(s["positions"].double() * f)
        spin = torch.polar(torch.full((s["N"], 1, rot // 2), s["amplitude"], dtype=torch.float64, device="cuda"), torch.stack(angles, -1)[:, None])
        outs = []
        for x in (s["q"], s["k"]):
            if x is None:
                continue
            o = x.double()
            at = (slice(0, rot // 2), slice(rot // 2, rot)) if s["pairs"] == "half" else (slice(0, rot, 2), slice(1, rot, 2))
            z = torch.complex(o[..., at[0]].contiguous(), o[..., at[1]].contiguous()) * spin
            o[..., at[0]], o[..., at[1]] = z.real, z.imag
            outs.append(o)
        return tuple(outs)
    drafts, first = _ints(case["drafts"]), 0
    accepted, tokens = [], []
    for b, m in enumerate(drafts):
        x, n = s["drafts"][first:first + m].tolist(), 0
        while n < m and float(s["u"][first + n]) * (float(s["q"][first + n, x[n]]) if s["q"] is not None else 1.0) < float(s["p"][first + b + n, x[n]]):
            n += 1
        w = s["p"][first + b + n].double()
        if n < m and s["q"] is None:
            w[x[n]] = 0
        elif n < m and bool((w > s["q"][first + n].double()).any()):
            w = torch.relu(w - s["q"][first + n].double())
        total = torch.cumsum(w, 0)
        accepted.append(n)
        tokens += x[:n] + [int(torch.searchsorted(total, total[-1:] * float(s["r"][b]), right=True))] + [-1] * (m - n)
        first += m
    return torch.tensor(accepted, dtype=torch.int32, device="cuda"), torch.tensor(tokens, dtype=torch.int32, device="cuda")
