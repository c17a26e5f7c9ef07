"""What the building blocks of a packed transformer layer cost, and what they compute.

Three operators, each through the package's public call and in a plain form of elementary
torch operations:

  linear     y = act(x W^T + b) + r                                     (linear_fused)
  attention  softmax(q k^T scale) v over packed sequences, grouped heads (attention_packed)
  rotary     positions turned into rotations of feature pairs            (Rotary.apply)

`own` selects the package's kernels; otherwise the plain forms run.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one token through the first feed-forward matrix of the XL width: latency, weights read once
        dict(name="linear_one_token", op="linear", m=1, k=1152, n=4608, dtype="bf16", act="gelu_tanh", bias=True,
             residual="none", out="bf16"),
        # condition rows of a guided batch to the six modulation vectors of one XL block
        dict(name="linear_condition_rows", op="linear", m=32, k=1152, n=6912, dtype="bf16", act="none", bias=True,
             residual="none", out="fp32"),
        # patches of 14 x 14 x 3 values (rows of 588, not whole 16-byte groups) to an odd width
        dict(name="linear_odd_patches", op="linear", m=1111, k=588, n=1153, dtype="fp16", act="silu", bias=True,
             residual="fp16", out="fp16"),
        # second feed-forward matrix of the XL width into the float32 residual stream, 32 rows of 256 tokens
        dict(name="linear_into_stream", op="linear", m=8192, k=4608, n=1152, dtype="bf16", act="none", bias=True,
             residual="fp32", out="fp32"),
        # first feed-forward matrix with its activation, 16 rows of 1024 tokens
        dict(name="linear_hidden", op="linear", m=16384, k=1152, n=4608, dtype="bf16", act="gelu_tanh", bias=True,
             residual="none", out="bf16"),
        # one new token in each of eight sequences over what they hold so far
        dict(name="attention_single_tokens", op="attention", q="1,1,1,1,1,1,1,1",
             k="1,77,700,1025,2048,3333,5000,8192", heads=32, kv_heads=8, dim=128, dtype="bf16", causal=True, lse=False),
        # pieces of prompts behind what was read before: empty, one-token, and longer than their keys
        dict(name="attention_prompt_pieces", op="attention", q="256,0,1,130,511,300,64", k="1024,40,513,130,2000,129,64",
             heads=12, kv_heads=4, dim=64, dtype="fp16", causal=True, lse=True),
        # latents of different sizes packed into one batch of 8192 tokens, every token sees its own latent
        dict(name="attention_packed_latents", op="attention", q="1024,256,576,784,1024,400,225,1023,640,256,960,1024",
             k="1024,256,576,784,1024,400,225,1023,640,256,960,1024", heads=16, kv_heads=16, dim=72, dtype="bf16",
             causal=False, lse=False),
        # one long prompt
        dict(name="attention_long_prompt", op="attention", q="8192", k="8192", heads=16, kv_heads=4, dim=128,
             dtype="bf16", causal=True, lse=False),
        # one token far behind the trained length, queries and keys together
        dict(name="rotary_one_token", op="rotary", tokens=1, heads=40, dim=128, part=128, interleaved=False, axes=1,
             dtype="bf16", scaling="yarn", factor=16.0, first=100000),
        # video latents of 2 x 4096 tokens: frame, row and column turn a third of the head each
        dict(name="rotary_video_latents", op="rotary", tokens=8192, heads=16, dim=72, part=72, interleaved=True, axes=3,
             dtype="fp32", scaling="none", factor=1.0, first=0),
        # a long prompt, half of every head turned, positions interpolated
        dict(name="rotary_long_prompt", op="rotary", tokens=32768, heads=20, dim=128, part=64, interleaved=False, axes=1,
             dtype="bf16", scaling="linear", factor=4.0, first=0),
    ]


def _between(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["linear", "attention", "rotary"])
    if op == "linear":
        m, n = _between(rng, 1, 8192), _between(rng, 64, 8192)
        k = _between(rng, 32, 8192)
        if rng.random() < 0.7:
            k = -(-k // 8) * 8
        most = 16384 * 1152 * 4608
        while m * n * k > most:
            m = max(1, m // 2)
        dtype = rng.choice(["bf16", "fp16"])
        out = rng.choice([dtype, dtype, "fp32"])
        return dict(op=op, m=m, k=k, n=n, dtype=dtype, act=rng.choice(["none", "relu", "gelu_tanh", "gelu", "silu"]),
                    bias=rng.random() < 0.7, residual=rng.choice(["none", out]), out=out)
    if op == "attention":
        count = _between(rng, 1, 12)
        longest = _between(rng, 16, 8192)
        kv_heads = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 3, 4, 8])
        while group * kv_heads > 32:
            group = max(1, group // 2)
        kind = rng.choice(["single", "piece", "whole"])
        k = [rng.randint(1, longest) for _ in range(count)]
        if kind == "single":
            q = [1] * count
        elif kind == "whole":
            q = list(k)
        else:
            q = [rng.randint(0, min(n, 512)) for n in k]
        heads = group * kv_heads
        # the plain form holds a padded score matrix: keep it, and the work, below the long prompt's
        while heads * count * max(max(q), 1) * max(k) > 16 * 8192 * 8192:
            q, k = [-(-n // 2) for n in q], [-(-n // 2) for n in k]
        if not sum(q):
            q[0] = 1
        return dict(op=op, q=",".join(map(str, q)), k=",".join(map(str, k)), heads=heads, kv_heads=kv_heads,
                    dim=rng.choice([64, 72, 80, 96, 128]), dtype=rng.choice(["bf16", "fp16"]),
                    causal=rng.random() < 0.7, lse=rng.random() < 0.5)
    dim = rng.choice([64, 72, 96, 128])
    axes = rng.choice([1, 1, 1, 2, 3])
    part = dim if rng.random() < 0.5 else dim // 2
    part -= part % (2 * axes)
    scaling = rng.choice(["none", "linear", "ntk", "yarn"])
    return dict(op=op, tokens=_between(rng, 1, 16384), heads=rng.randint(1, 40), dim=dim, part=part,
                interleaved=rng.random() < 0.5, axes=axes, dtype=rng.choice(["bf16", "fp16", "fp32"]), scaling=scaling,
                factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 16.0]),
                first=rng.choice([0, _between(rng, 1, 1000000)]))


def _lengths(text):
    return [int(n) for n in text.split(",")]


def _offsets(lengths):
    return torch.tensor([0] + lengths, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()


ORIGINAL = 4096  # positions that the scaled rotations were trained on


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, device="cuda", generator=g) * std).to(dtype)

    t = DTYPES[case["dtype"]]
    if case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        s = dict(case=case, x=normal(m, k, dtype=t), w=normal(n, k, std=k ** -0.5, dtype=t), bias=None, residual=None)
        if case["bias"]:
            s["bias"] = normal(n, std=0.5)
        if case["residual"] != "none":
            s["residual"] = normal(m, n, dtype=DTYPES[case["residual"]])
        return s
    if case["op"] == "attention":
        q, k = _lengths(case["q"]), _lengths(case["k"])
        h, hk, d = case["heads"], case["kv_heads"], case["dim"]
        return dict(case=case, q=normal(sum(q), h, d, dtype=t), k=normal(sum(k), hk, d, dtype=t),
                    v=normal(sum(k), hk, d, dtype=t), cu_q=_offsets(q), cu_k=_offsets(k), max_q=max(q), max_k=max(k))
    n, a = case["tokens"], case["axes"]
    x = normal(n, case["heads"], case["dim"], dtype=t)
    if a == 1:
        # one run of positions, the start moved with the seed
        pos = (torch.arange(n, device="cuda") + case["first"] + seed % 97).to(torch.int32)
    else:
        pos = torch.randint(0, 64, (n, a), device="cuda", generator=g).to(torch.int32) + case["first"]
    s = dict(case=case, x=x, positions=pos)
    if own:
        from diffusion_transformer_denoiser_dit_b200 import Rotary
        s["rotary"] = Rotary(case["dim"], rotary_dim=case["part"], interleaved=case["interleaved"], axes=a,
                             scaling=case["scaling"], factor=case["factor"], original_length=ORIGINAL)
    return s


def run(state):
    case = state["case"]
    if own:
        return _kernel(case, state)
    return {"linear": _plain_linear, "attention": _plain_attention, "rotary": _plain_rotary}[case["op"]](case, state)


def _kernel(case, s):
    from diffusion_transformer_denoiser_dit_b200 import attention_packed, linear_fused
    if case["op"] == "linear":
        return linear_fused(s["x"], s["w"], s["bias"], act=case["act"], residual=s["residual"],
                            out_dtype=DTYPES[case["out"]])
    if case["op"] == "attention":
        return attention_packed(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["max_q"], s["max_k"],
                                causal=case["causal"], return_lse=case["lse"])
    return s["rotary"].apply(s["x"], s["positions"])


# ---------------------------------------------------------------- plain forms


def _plain_linear(case, s):
    y = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        y = y + s["bias"]
    if case["act"] == "relu":
        y = y * (y > 0)
    elif case["act"] == "gelu_tanh":
        y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    elif case["act"] == "gelu":
        y = 0.5 * y * torch.erfc(y * -math.sqrt(0.5))
    elif case["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(DTYPES[case["out"]])


def _plain_attention(case, s):
    """Every sequence padded to the longest: scores [sequences, heads, queries, keys] in 32 bits."""
    group = case["heads"] // case["kv_heads"]
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    nq, nk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    i, j = torch.arange(s["max_q"], device="cuda"), torch.arange(s["max_k"], device="cuda")
    has_q, has_k = i < nq[:, None], j < nk[:, None]
    row_q = (cu_q[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    row_k = (cu_k[:-1, None] + j).clamp(max=s["k"].shape[0] - 1)
    q = s["q"][row_q].float().transpose(1, 2)                                       # [b, h, i, d]
    k = s["k"][row_k].float().repeat_interleave(group, 2).permute(0, 2, 3, 1)       # [b, h, d, j]
    v = s["v"][row_k].float().repeat_interleave(group, 2).transpose(1, 2)           # [b, h, j, d]
    seen = has_q[:, None, :, None] & has_k[:, None, None, :]
    if case["causal"]:
        seen = seen & (j[None, None, None, :] <= i[None, None, :, None] + (nk - nq)[:, None, None, None])
    scores = (q @ k) * case["dim"] ** -0.5
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0.0)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / total.masked_fill(total == 0, 1.0)
    out = o.transpose(1, 2)[has_q].to(s["q"].dtype)                                  # packed again
    if not case["lse"]:
        return out
    return out, (top + torch.log(total))[..., 0].transpose(1, 2)[has_q].t().contiguous()


def _frequencies(case):
    """Radians per position of each pair of one section, in 64 bits, and what multiplies cos and sin."""
    n = case["part"] // case["axes"]
    base, factor = 10000.0, case["factor"]
    e = torch.arange(0, n, 2, dtype=torch.float64, device="cuda") / n
    if case["scaling"] == "ntk":
        return (base * factor ** (n / (n - 2))) ** -e, 1.0
    f = base ** -e
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "yarn":
        keep = ((ORIGINAL * f / (2 * math.pi) - 1) / 31).clamp(0, 1)
        return f * keep + f / factor * (1 - keep), 0.1 * math.log(factor) + 1
    return f, 1.0


def _plain_rotary(case, s):
    f, mult = _frequencies(case)
    x, part = s["x"].float(), case["part"]
    angle = (s["positions"].double().reshape(-1, case["axes"], 1) * f).flatten(1)[:, None, :]
    cos, sin = (torch.cos(angle) * mult).float(), (torch.sin(angle) * mult).float()
    if case["interleaved"]:
        a, b = x[..., 0:part:2], x[..., 1:part:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :part // 2], x[..., part // 2:part]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., part:]), -1).to(s["x"].dtype)


# ---------------------------------------------------------------- what a pass cannot do without


def _pairs(q, k, causal):
    """Query-key pairs of one sequence that the mask lets through."""
    if not causal:
        return q * k
    rows = min(q, k)                 # the queries before these see nothing
    return rows * (k - rows + 1) + rows * (rows - 1) // 2


def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    e = size[case["dtype"]]
    if case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        moved = e * (m * k + n * k) + size[case["out"]] * m * n + (4 * n if case["bias"] else 0)
        if case["residual"] != "none":
            moved += size[case["residual"]] * m * n
        return {"bytes": moved, "flops": 2 * m * n * k}
    if case["op"] == "attention":
        q, k = _lengths(case["q"]), _lengths(case["k"])
        h, hk, d = case["heads"], case["kv_heads"], case["dim"]
        # keys that no query of their sequence sees need not be read
        read = sum(b for a, b in zip(q, k) if a)
        pairs = sum(_pairs(a, b, case["causal"]) for a, b in zip(q, k))
        moved = e * d * (2 * h * sum(q) + 2 * hk * read) + (4 * h * sum(q) if case["lse"] else 0)
        return {"bytes": moved, "flops": 4 * d * h * pairs}
    n = case["tokens"] * case["heads"]
    return {"bytes": 2 * e * n * case["dim"] + 4 * case["tokens"] * case["axes"], "flops": 3 * n * case["part"]}


# ---------------------------------------------------------------- the definitions, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        z = torch.einsum("mk,nk->mn", s["x"].double(), s["w"].double())
        if s["bias"] is not None:
            z += s["bias"].double()
        z = {"none": lambda a: a, "relu": lambda a: a.clamp(min=0),
             "gelu_tanh": lambda a: a * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (a + 0.044715 * a ** 3)),
             "gelu": lambda a: a * torch.special.ndtr(a), "silu": lambda a: a * torch.sigmoid(a)}[case["act"]](z)
        return z if s["residual"] is None else z + s["residual"].double()
    if case["op"] == "attention":
        h, hk, d = case["heads"], case["kv_heads"], case["dim"]
        outs, logs, a, b = [], [], 0, 0
        for nq, nk in zip(_lengths(case["q"]), _lengths(case["k"])):
            q, k, v = s["q"][a:a + nq].double(), s["k"][b:b + nk].double(), s["v"][b:b + nk].double()
            a, b = a + nq, b + nk
            o = torch.zeros(nq, h, d, dtype=torch.float64, device="cuda")
            z = torch.full((h, nq), -math.inf, dtype=torch.float64, device="cuda")
            for head in range(h):
                e = torch.einsum("id,jd->ij", q[:, head], k[:, head * hk // h]) / math.sqrt(d)
                if case["causal"]:
                    e += torch.full_like(e, -math.inf).triu(nk - nq + 1)
                z[head] = torch.logsumexp(e, 1) if nk else z[head]
                w = torch.exp(e - z[head][:, None])
                o[:, head] = torch.where(torch.isinf(z[head])[:, None], 0.0, w @ v[:, head * hk // h])
            outs.append(o)
            logs.append(z)
        return (torch.cat(outs), torch.cat(logs, 1)) if case["lse"] else torch.cat(outs)
    part, axes = case["part"], case["axes"]
    each = part // 2 // axes
    x = s["x"].double()
    pos = s["positions"].double().reshape(-1, axes)
    turned = []
    for pair in range(part // 2):
        axis, i = divmod(pair, each)
        theta = 10000.0 ** (-i / each)
        size = 1.0
        if case["scaling"] == "linear":
            theta /= case["factor"]
        elif case["scaling"] == "ntk":
            theta = (10000.0 * case["factor"] ** (each / (each - 1))) ** (-i / each)
        elif case["scaling"] == "yarn":
            share = min(1.0, max(0.0, (ORIGINAL / (2 * math.pi / theta) - 1.0) / (32.0 - 1.0)))
            theta = (1 - share) * theta / case["factor"] + share * theta
            size = 1.0 + 0.1 * math.log(case["factor"])
        u, w = (2 * pair, 2 * pair + 1) if case["interleaved"] else (pair, pair + part // 2)
        turn = torch.polar(torch.full_like(pos[:, axis], size), pos[:, axis] * theta)[:, None]
        turned.append((u, w, torch.complex(x[..., u], x[..., w]) * turn))
    y = x.clone()
    for u, w, z in turned:
        y[..., u], y[..., w] = z.real, z.imag
    return y
