"""The quantised key/value cache and the attention over it: what a call does, in plain torch operations and through
the library, on the sizes that serving meets.

A cache holds, for each token, KV head and group of 64 channels, 64 codes of 4 or 8 bits and a (scale, bias) pair in
bf16; a value is code * scale + bias.  Four operators: "write" (quantise new keys and values into the cache, and read
them back), "read" (a span of the cache as bf16), "decode" (attention of one query token per sequence) and "prefill"
(attention of a chunk of query tokens per sequence, causal).

A case gives the cache length of each sequence after the call (`lens`, new tokens included) and the tokens the call
deals with (`new`: written, read back from the end, or querying; decode: one each).
"""
import math

import torch

own = False

GROUP = 64

MODEL = {"H_q": 16, "H_kv": 2, "D": 256, "bs": 64}  # the repository's full-attention layers


def listed():
    def case(name, op, lens, new=None, bits=4, **kw):
        return {"name": name, "op": op, "bits": bits, **{**MODEL, **kw}, "lens": lens, "new": lens if new is None else new}

    return [
        # one decode step of four conversations: latency
        case("write_step", "write", "1,100,777,5000", "1,1,1,1"),
        # continuous batching: a long prompt, a single token, a chunk on a long context, an idle slot
        case("write_prompts", "write", "8192,100,2049,64,33281", "8192,1,2049,0,513"),
        # a batch of documents read in at 8 bits, as many KV heads as query heads, small blocks
        case("write_8bit", "write", "16384,12001,9000,8191,7777,6000,4097,1", bits=8, H_q=4, H_kv=4, D=128, bs=32),
        # a 64K-token context taken out of the cache (to move it or to hand it to a bf16 path)
        case("read_64k", "read", "65536"),
        # a ragged batch at the edges of 128-token blocks, an empty sequence, 8 bits, small heads
        case("read_ragged", "read", "1,127,128,129,4000,0", bits=8, H_q=6, H_kv=3, D=64, bs=128),
        # the smallest batch: one token, a ragged block, several blocks
        case("decode_tiny", "decode", "1,100,777", "1,1,1", D=128),
        # one conversation at the context lengths that the repository's benchmark has
        case("decode_32k", "decode", "32768", "1"),
        case("decode_128k", "decode", "131072", "1"),
        # a decode batch of 24 sequences of mixed lengths at 8 bits
        case("decode_batch", "decode", "2011,37,2900,1500,801,2222,64,1,1203,2741,999,130,2503,417,1777,65,2816,640,1333,2999,290,1024,2107,555",
             ",".join(["1"] * 24), bits=8, D=128),
        # eight sequences, four draft tokens each, checked at once
        case("prefill_draft", "prefill", "8192,4100,12000,333,7001,9999,2048,5555", "4,4,4,4,4,4,4,4"),
        # a whole prompt
        case("prefill_8k", "prefill", "8192"),
        # a chunk of a long prompt
        case("prefill_chunk", "prefill", "32768", "2048"),
    ]


def draw(rng):
    op = rng.choice(["write", "read", "decode", "prefill"])
    H_q, H_kv = rng.choice([(16, 2), (8, 2), (4, 4), (2, 1), (6, 3)])
    D, bs, bits = rng.choice([64, 128, 256]), rng.choice([32, 64, 128]), rng.choice([4, 4, 8])

    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    B = log(1, 32)
    total = log(64, 131072 * 512 // (H_kv * D) // 2) // B  # cached tokens a sequence, about
    if op == "prefill":
        total = min(total, 16384)
    lens = [0 if rng.random() < 0.05 else max(1, log(max(1, total // 4), max(2, total * 2))) for _ in range(B)]
    if op == "decode":
        new = [1] * B
    elif op == "prefill":
        # padded to the longest chunk and the longest context, a pass costs no more than the largest listed one
        most = max(1, min(4096, (2048 * 32768 * 16 * 256) // (B * max(lens + [1]) * H_q * D)))
        new = [min(n, log(1, most)) for n in lens]
    else:
        new = [n if rng.random() < 0.5 else min(n, log(1, 4096)) for n in lens]
    lens, new = (lens, new) if sum(new) else ([5] + lens[1:], [1] + new[1:])
    return {"op": op, "bits": bits, "H_q": H_q, "H_kv": H_kv, "D": D, "bs": bs,
            "lens": ",".join(map(str, lens)), "new": ",".join(map(str, new))}


def _ints(text):
    return [int(x) for x in text.split(",")]


# ---------------------------------------------------------------- the plain form
def _quantise(x, bits):
    """Codes (uint8) [..., D/64, 64] and (scale, bias) bf16 [..., D/64, 2] of x [..., D]."""
    x = x.float().unflatten(-1, (-1, GROUP))
    levels = torch.tensor(float(2 ** bits - 1), device=x.device)
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale = ((hi - lo) / levels).to(torch.bfloat16)
    scale = torch.where(scale.float() < 2.0 ** -126, torch.zeros_like(scale), scale)
    s = scale.float()
    code = torch.where(s > 0, torch.round((x - lo) / s), torch.zeros_like(x)).clamp(0, 2 ** bits - 1).to(torch.uint8)
    return code, torch.cat([scale, lo.to(torch.bfloat16)], -1)


def _pack(code, bits):
    return code if bits == 8 else code[..., 0::2] | (code[..., 1::2] << 4)


def _values(q, sb, bits):
    """Values in fp32 [..., D] of packed codes [..., D/64, 64 bits / 8] and parameters [..., D/64, 2]."""
    code = q if bits == 8 else torch.stack([q & 15, q >> 4], -1).flatten(-2)
    sb = sb.float()
    return (code.float() * sb[..., :1] + sb[..., 1:]).flatten(-2)


def _rows(s):
    """Sequence and position of each of the call's tokens."""
    n = torch.arange(s["N"], device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), n, right=True)
    return b, s["starts"][b].long() + n - s["cu"][b].long()


def _place(s, b, pos):
    return s["table"][b, pos // s["bs"]].long(), pos % s["bs"]


def _padded(s):
    """Keys and values of all sequences, [B, H_kv, longest, D] in fp32, and the lengths [B, 1]."""
    pos = torch.arange(s["longest"], device="cuda")[None]
    lens = s["lens"].long()[:, None]
    pos = torch.where(pos < lens, pos, 0)
    phys = torch.where(lens > 0, s["table"].long().gather(1, pos // s["bs"]), 0)
    c = s["cache"]
    k, v = (_values(c[n + "_q"][phys, :, :, pos % s["bs"]], c[n + "_sb"][phys, :, :, pos % s["bs"]], s["bits"]) for n in "kv")
    return k.transpose(1, 2), v.transpose(1, 2), lens


def _attend(q, k, v, seen, scale):
    """q [B, H_kv, R, D] on k, v [B, H_kv, L, D]; seen [B, 1, R, L]."""
    w = (q @ k.transpose(-1, -2)).mul_(scale).masked_fill_(~seen, -math.inf)
    m = w.amax(-1, keepdim=True)
    w = w.sub_(torch.where(m > -math.inf, m, 0)).exp_()
    return (w @ v) / w.sum(-1, keepdim=True).clamp_min(1e-30)


def _plain(s):
    op, H_kv, D, bits, c = s["op"], s["H_kv"], s["D"], s["bits"], s["cache"]
    if op in ("write", "read"):
        phys, row = _place(s, *_rows(s))
        if op == "write":
            (k, k_sb), (v, v_sb) = _quantise(s["k"], bits), _quantise(s["v"], bits)
            c["k_q"][phys, :, :, row], c["k_sb"][phys, :, :, row] = _pack(k, bits), k_sb
            c["v_q"][phys, :, :, row], c["v_sb"][phys, :, :, row] = _pack(v, bits), v_sb
        return tuple(_values(c[n + "_q"][phys, :, :, row], c[n + "_sb"][phys, :, :, row], bits).to(torch.bfloat16) for n in "kv")
    k, v, lens = _padded(s)
    B, G = s["B"], s["H_q"] // H_kv
    at = torch.arange(s["longest"], device="cuda")
    if op == "decode":
        q = s["q"].float().view(B, H_kv, G, D)
        return _attend(q, k, v, (at < lens)[:, None, None], D ** -0.5).view(B, s["H_q"], D).to(torch.bfloat16)
    b, pos = _rows(s)
    i = pos - s["starts"][b].long()
    q = torch.zeros((B, s["most"], H_kv, G, D), device="cuda")
    q[b, i] = s["q"].float().view(-1, H_kv, G, D)
    upto = s["starts"].long()[:, None] + torch.arange(s["most"], device="cuda")
    seen = ((at <= upto[..., None]) & (at < lens[..., None]))[:, None, :, None].expand(-1, -1, -1, G, -1).flatten(2, 3)
    o = _attend(q.permute(0, 2, 1, 3, 4).flatten(2, 3), k, v, seen, D ** -0.5)
    o = o.view(B, H_kv, s["most"], G, D).permute(0, 2, 1, 3, 4)
    return o[b, i].reshape(-1, s["H_q"], D).to(torch.bfloat16)


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    c = {k: v for k, v in case.items() if k != "name"}
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    lens, new = _ints(c["lens"]), _ints(c["new"])
    H_q, H_kv, D, bs, bits = c["H_q"], c["H_kv"], c["D"], c["bs"], c["bits"]
    need = [(n + bs - 1) // bs for n in lens]
    blocks, width, N = sum(need) + 3, max(max(need), 1), sum(new)
    # keys with channels of unlike size, as rotated and normalised keys have
    gain = torch.randn((2, H_kv, D), generator=g, device="cuda").mul_(0.5).exp_()

    def values(n, which):
        return (torch.randn((n, H_kv, D), generator=g, device="cuda") * gain[which]).to(torch.bfloat16)

    cache = {}
    for which, n in enumerate("kv"):
        code, sb = _quantise(values(blocks * bs, which), bits)
        cache[n + "_q"] = _pack(code, bits).unflatten(0, (blocks, bs)).permute(0, 2, 3, 1, 4).contiguous()
        cache[n + "_sb"] = sb.unflatten(0, (blocks, bs)).permute(0, 2, 3, 1, 4).contiguous()
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    first = [sum(need[:b]) for b in range(len(lens))]
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(first[b], first[b] + n, dtype=torch.int32)
    table = table.to("cuda")
    table = torch.where(table >= 0, order[table.clamp_min(0).long()], table)
    s = {**c, "B": len(lens), "N": N, "longest": max(max(lens), 1), "most": max(new), "cache": cache, "table": table.contiguous(),
         "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
         "starts": torch.tensor([n - m for n, m in zip(lens, new)], dtype=torch.int32, device="cuda"),
         "cu": torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32, device="cuda")}
    if c["op"] == "write":
        # slices of a fused projection's output: the rows are further apart than they are wide
        s["fused"] = torch.randn((N, (H_q + 2 * H_kv) * D), generator=g, device="cuda").to(torch.bfloat16)
        kv = s["fused"][:, H_q * D:].unflatten(-1, (2, H_kv, D))
        kv.mul_(gain)
        s["k"], s["v"] = kv[:, 0], kv[:, 1]
    if c["op"] in ("write", "read"):
        s["k_out"], s["v_out"] = (torch.empty((N, H_kv, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    else:
        n = len(lens) if c["op"] == "decode" else N
        s["q"] = torch.randn((n, H_q, D), generator=g, device="cuda").to(torch.bfloat16)
        s["out"] = torch.empty((n, H_q, D), dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------- the calls
def _through_the_library(s):
    import bit_grouped_expert_top_gb300 as lm

    if "ws" not in s:  # what a program sets up once
        s["shape"] = lm.make_kvq_shape(s["B"], s["H_q"], s["H_kv"], s["D"], s["bs"], s["table"].shape[1], s["bits"])
        s["handle"] = lm.make_kvq_cache(s["cache"])
        s["ws"] = lm.alloc_kvq_workspace(s["shape"], s["N"] if s["op"] == "prefill" else 0)
    shape, cache, ws = s["shape"], s["handle"], s["ws"]
    if s["op"] == "decode":
        lm.lily_kvq_attn_decode(shape, cache, s["q"], s["table"], s["lens"], s["out"], ws)
        return s["out"]
    if s["op"] == "prefill":
        lm.lily_kvq_attn_prefill(shape, cache, s["q"], s["cu"], s["table"], s["lens"], s["out"], ws)
        return s["out"]
    if s["op"] == "write":
        lm.lily_kvq_append(shape, cache, s["k"], s["v"], s["cu"], s["starts"], s["table"], ws)
    lm.lily_kvq_read(shape, cache, s["k_out"], s["v_out"], s["cu"], s["starts"], s["table"], ws)
    return s["k_out"], s["v_out"]


def run(state):
    return _through_the_library(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    lens, new = _ints(case["lens"]), _ints(case["new"])
    H_q, H_kv, D, bits = case["H_q"], case["H_kv"], case["D"], case["bits"]
    token = 2 * H_kv * (D * bits // 8 + D // GROUP * 4)  # codes and parameters of K and V
    plain = 2 * H_kv * D * 2
    N = sum(new)
    if case["op"] == "write":
        return {"bytes": N * (2 * plain + 2 * token), "flops": 10 * N * 2 * H_kv * D}
    if case["op"] == "read":
        return {"bytes": N * (plain + token), "flops": 2 * N * 2 * H_kv * D}
    rows = len(lens) if case["op"] == "decode" else N
    used = [n for n, m in zip(lens, new) if m]
    pairs = sum(lens) if case["op"] == "decode" else sum(m * (n - m) + m * (m + 1) // 2 for n, m in zip(lens, new))
    return {"bytes": sum(used) * token + rows * H_q * D * 4, "flops": 4 * H_q * D * pairs}


# ---------------------------------------------------------------- the definition in 64 bits
def _decoded(q, sb, bits):
    """One sequence's rows [n][H_kv][D/64][bytes] as 64-bit values [n][H_kv][D]."""
    whole = q.to(torch.int64)
    n, H_kv, groups, _ = q.shape
    code = torch.empty((n, H_kv, groups, GROUP), dtype=torch.float64, device=q.device)
    if bits == 8:
        code[:] = whole
    else:
        code[..., 0::2] = whole % 16
        code[..., 1::2] = whole // 16
    sb = sb.double()
    return (code * sb[..., 0, None] + sb[..., 1, None]).reshape(n, H_kv, groups * GROUP)


def _rounded(x, bits):
    """x [n][H_kv][D] as the 64-bit values that its codes stand for."""
    x = x.double().reshape(*x.shape[:2], -1, GROUP)
    low, high = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    step = ((high - low) / (2 ** bits - 1)).float().to(torch.bfloat16).double()
    step[step < 2.0 ** -126] = 0
    code = torch.nan_to_num((x - low) / step).round().clamp(0, 2 ** bits - 1)
    return (code * step + low).flatten(-2)


def exact(case, seed):
    lens, new = _ints(case["lens"]), _ints(case["new"])
    s = prepare(case, seed)
    op, bits, bs, D, H_kv = s["op"], s["bits"], s["bs"], s["D"], s["H_kv"]
    G = s["H_q"] // H_kv
    if op == "write":
        return tuple(_rounded(s[n], bits) for n in "kv")
    first = [sum(new[:b]) for b in range(len(new))]
    outs = []
    for b, (L, m) in enumerate(zip(lens, new)):
        if op != "decode" and m == 0:
            continue
        if L == 0:
            outs.append(torch.zeros((1, s["H_q"], D), dtype=torch.float64, device="cuda"))
            continue
        used = s["table"][b, :(L + bs - 1) // bs].long()
        k, v = (_decoded(s["cache"][n + "_q"][used].permute(0, 3, 1, 2, 4).flatten(0, 1)[:L],
                         s["cache"][n + "_sb"][used].permute(0, 3, 1, 2, 4).flatten(0, 1)[:L], bits) for n in "kv")
        if op == "read":
            outs.append((k[L - m:], v[L - m:]))
            continue
        q = s["q"][b:b + 1] if op == "decode" else s["q"][first[b]:first[b] + m]
        o = torch.empty(q.shape, dtype=torch.float64, device="cuda")
        hidden = torch.arange(L, device="cuda")[None] > torch.arange(L - len(q), L, device="cuda")[:, None]
        for h in range(s["H_q"]):
            score = q[:, h].double() @ k[:, h // G].T / math.sqrt(D)
            score[hidden] = -math.inf
            o[:, h] = torch.softmax(score, -1) @ v[:, h // G]
        outs.append(o)
    if op == "read":
        return tuple(torch.cat([o[n] for o in outs]) for n in range(2))
    return torch.cat(outs)
