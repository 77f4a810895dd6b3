"""Timed cases of the operators that a decoding program calls around the eviction step.

Three operators, in the order a serving loop runs them on one layer:

* ``qk_norm_rope``: RMS norm of every query and key head and the rotation to the token's position,
  in one pass over a projection's output; the keys land in the layout the cache takes.
* ``attend`` over cache rows: one query token per sequence against the sequence's own kept keys and
  values (grouped query heads, ragged lengths) and the token's own key and value.
* ``attend`` with a shared prefix: the same with a long prefix that the whole batch shares, whose
  keys and values are read once for all sequences; without own rows it is the prefix part of a
  prompt chunk.

``run`` computes a case with elementary torch operations, or with the library's calls where ``own``
is set. ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


def listed():
    def qk(name, batch, seq, heads, kv_heads, dim, dtype, theta, scattered):
        return {"name": name, "op": "qk", "batch": batch, "seq": seq, "heads": heads, "kv_heads": kv_heads,
                "dim": dim, "dtype": dtype, "theta": theta, "scattered": scattered}

    def at(name, batch, heads, kv_heads, dim, rows, prefix, dtype, new, ragged):
        return {"name": name, "op": "attend", "batch": batch, "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "rows": rows, "prefix": prefix, "dtype": dtype, "new": new, "ragged": ragged}

    return [
        # one token of the four-row cache: the smallest call, all latency
        qk("qk_one_token_small", 1, 1, 4, 4, 64, "fp16", 10000.0, False),
        # one decode step of 32 sequences, a bf16 model's projection
        qk("qk_step_batch32", 32, 1, 32, 8, 128, "bf16", 500000.0, False),
        # three prompts of an odd length at their own positions (continued conversations), fp32 activations
        qk("qk_prompt_odd_positions", 3, 1021, 24, 8, 128, "fp32", 500000.0, True),
        # one layer of the largest prompt: 32 sequences of 4096 tokens
        qk("qk_prompt_large", 32, 4096, 32, 8, 128, "bf16", 500000.0, False),
        # the 32-row budget of the smallest cache
        at("rows_small", 1, 4, 4, 64, 32, 0, "fp16", True, False),
        # one layer of a single sequence at budget 512, three query heads a key head
        at("rows_budget512", 1, 24, 8, 128, 512, 0, "fp16", True, False),
        # one layer of 32 sequences at the average budget of the large cache
        at("rows_budget2048_batch32", 32, 32, 8, 128, 2048, 0, "fp16", True, False),
        # unequal sequences that kept everything, an empty and a one-token one among them
        at("rows_long_ragged", 7, 40, 8, 128, 65521, 0, "bf16", False, True),
        # a short instruction in front of four short conversations
        at("prefix_short", 4, 24, 8, 128, 64, 333, "fp16", True, False),
        # a long document that 32 conversations ask about, budget 512 each
        at("prefix_decode_batch32", 32, 32, 8, 128, 512, 16384, "fp16", True, False),
        # prompt chunks against the shared prefix: 16 sequences of 256 tokens, bound by arithmetic
        at("prefix_chunk", 4096, 32, 8, 128, 0, 8192, "bf16", False, False),
        # sequences that share different lengths of the prefix, some none of it
        at("prefix_ragged", 48, 40, 8, 64, 0, 65521, "fp16", False, True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    op = rng.choice(["qk", "rows", "prefix", "chunk"])
    if op == "qk":
        tokens = log(1, 131072 * 40 // (kv_heads + heads) if kv_heads + heads > 40 else 131072)
        batch = min(tokens, log(1, 64))
        return {"op": "qk", "batch": batch, "seq": max(1, tokens // batch), "heads": heads, "kv_heads": kv_heads,
                "dim": dim, "dtype": rng.choice(["fp16", "bf16", "fp32"]), "theta": rng.choice([10000.0, 500000.0]),
                "scattered": rng.random() < 0.5}
    case = {"op": "attend", "heads": heads, "kv_heads": kv_heads, "dim": dim, "dtype": rng.choice(["fp16", "bf16"])}
    if op == "rows":
        # at most the listed ragged case's keys and values, over all sequences
        rows = log(1, 65521)
        batch = log(1, max(1, min(256, 3000000 // (rows * kv_heads))))
        case.update(batch=batch, rows=rows, prefix=0, new=rng.random() < 0.5, ragged=rng.random() < 0.5)
    elif op == "prefix":
        # decode steps: a few sequences to a full batch, with their own short rows or none
        prefix, batch = log(1, 65521), log(1, 64)
        rows = rng.choice([0, log(1, 1024)])
        case.update(batch=batch, rows=rows, prefix=prefix, new=rng.random() < 0.5, ragged=rng.random() < 0.5)
    else:
        # prompt chunks: at most the listed chunk's products
        prefix = log(64, 16384)
        most = 4096 * 32 * 8192 * 128 // (heads * prefix * dim)
        case.update(batch=log(min(64, most), max(64, min(8192, most))), rows=0, prefix=prefix, new=False,
                    ragged=rng.random() < 0.3)
    return case


def lengths(count, top):
    """Unequal lengths in 0 .. top, spread over it; the first is the whole, the next two are nothing and one row."""
    found = [int(top * ((0.6180339887 * i) % 1.0)) for i in range(count)]
    found[:3] = [top, 0, min(1, top)][:count]
    return found


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    B, H, G, D = case["batch"], case["kv_heads"], case["heads"], case["dim"]
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, to=dtype):
        return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32 if to is torch.float32 else torch.float16) * scale).to(to)

    if case["op"] == "qk":
        S = case["seq"]
        # the fused projection's output: queries, keys and values of a token side by side
        qkv = normal(B, S, G + 2 * H, D, scale=2.0)
        state = {"case": case, "q": qkv[:, :, :G], "k": qkv[:, :, G:G + H],
                 "q_weight": 1 + normal(D, scale=0.1), "k_weight": 1 + normal(D, scale=0.1),
                 "q_out": torch.empty(B, S, G, D, dtype=torch.float16, device="cuda"),
                 # the cache takes a layer's prompt keys as [batch, kv_heads, seq, dim]
                 "k_out": torch.empty(B, H, S, D, dtype=torch.float16, device="cuda").transpose(1, 2),
                 "positions": None, "pos0": 0 if S > 1 else 4096}
        if case["scattered"]:
            first = torch.randint(0, 100000, (B, 1), generator=gen, device="cuda", dtype=torch.int32)
            state["positions"] = first + torch.arange(S, device="cuda", dtype=torch.int32)
        return state
    state = {"case": case, "q": normal(B, G, D, scale=1.5),
             "out": torch.empty(B, G, D, dtype=dtype, device="cuda"),
             "lse": torch.empty(B, G, dtype=torch.float32, device="cuda"),
             "k": None, "v": None, "lens": None, "k_new": None, "v_new": None,
             "prefix_k": None, "prefix_v": None, "prefix_lens": None}
    if case["rows"]:
        state["k"], state["v"] = normal(B, H, case["rows"], D), normal(B, H, case["rows"], D)
        if case["ragged"]:
            state["lens"] = torch.tensor(lengths(B, case["rows"]), dtype=torch.int32, device="cuda")
    if case["new"]:
        state["k_new"], state["v_new"] = normal(B, H, D), normal(B, H, D)
    if case["prefix"]:
        state["prefix_k"], state["prefix_v"] = normal(H, case["prefix"], D), normal(H, case["prefix"], D)
        if case["ragged"]:
            state["prefix_lens"] = torch.tensor(lengths(B, case["prefix"]), dtype=torch.int32, device="cuda")
    return state


def run(state):
    if state["case"]["op"] == "qk":
        return run_qk(state)
    return run_attend(state)


def run_qk(s):
    if own:
        import kv_cache_attention_02_gb300 as kvx
        kvx.qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], rope_theta=s["case"]["theta"], q_weight=s["q_weight"],
                         k_weight=s["k_weight"], eps=EPS, positions=s["positions"], pos0=s["pos0"])
        return s["q_out"], s["k_out"]
    S, D = s["case"]["seq"], s["case"]["dim"]
    p = s["positions"]
    if p is None:
        p = torch.arange(s["pos0"], s["pos0"] + S, device="cuda")[None]
    w = s["case"]["theta"] ** (-2.0 * torch.arange(D // 2, device="cuda", dtype=torch.float64) / D)
    angle = p.double()[..., None] * w
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]

    def one(x, weight):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1).half()

    # the key's layout is the cache's: [batch, kv_heads, seq, dim], seen as [batch, seq, kv_heads, dim]
    return one(s["q"], s["q_weight"]), one(s["k"], s["k_weight"]).transpose(1, 2).contiguous().transpose(1, 2)


def run_attend(s):
    if own:
        import kv_cache_attention_02_gb300 as kvx
        kvx.attend(s["q"], s["out"], k=s["k"], v=s["v"], lens=s["lens"], k_new=s["k_new"], v_new=s["v_new"],
                   prefix_k=s["prefix_k"], prefix_v=s["prefix_v"], prefix_lens=s["prefix_lens"], lse=s["lse"])
        return s["out"], s["lse"]
    c = s["case"]
    B, H, D = c["batch"], c["kv_heads"], c["dim"]
    N, G = c["heads"] // H, c["heads"]
    q = s["q"].float().view(B, H, N, D) / math.sqrt(D)
    parts = []
    if s["k"] is not None:
        part = q @ s["k"].float().transpose(2, 3)
        if s["lens"] is not None:
            part.masked_fill_(torch.arange(c["rows"], device="cuda") >= s["lens"][:, None, None, None], -math.inf)
        parts.append(part)
    if s["k_new"] is not None:
        parts.append((q * s["k_new"].float()[:, :, None]).sum(-1, keepdim=True))
    if s["prefix_k"] is not None:
        folded = q.transpose(0, 1).reshape(H, B * N, D) @ s["prefix_k"].float().transpose(1, 2)
        part = folded.view(H, B, N, -1).transpose(0, 1)
        if s["prefix_lens"] is not None:
            part = part.masked_fill(torch.arange(c["prefix"], device="cuda") >= s["prefix_lens"][:, None, None, None], -math.inf)
        parts.append(part)
    # a sequence with nothing to attend to answers with zeros
    top = torch.stack([x.amax(-1) for x in parts]).amax(0)[..., None]
    top = torch.where(top == -math.inf, 0.0, top)
    parts = [torch.exp(x - top) for x in parts]
    total = torch.stack([x.sum(-1) for x in parts]).sum(0)
    out = torch.zeros(B, H, N, D, device="cuda")
    if s["prefix_k"] is not None:
        folded = parts.pop().transpose(0, 1).reshape(H, B * N, -1) @ s["prefix_v"].float()
        out += folded.view(H, B, N, D).transpose(0, 1)
    if s["k_new"] is not None:
        out += parts.pop() * s["v_new"].float()[:, :, None]
    if s["k"] is not None:
        out += parts.pop() @ s["v"].float()
    out = out / torch.where(total == 0, 1.0, total)[..., None]
    lse = top[..., 0] + torch.log(total)
    return out.to(s["out"].dtype).view(B, G, D), lse.view(B, G)


def work(case):
    B, H, G, D = case["batch"], case["kv_heads"], case["heads"], case["dim"]
    width = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "qk":
        heads = B * case["seq"] * (G + H)
        positions = 4 * B * case["seq"] if case["scattered"] else 0
        # a square and its sum, the norm and the weight, and four products and two sums a pair
        return {"bytes": heads * D * (width + 2) + 2 * D * width + positions, "flops": heads * D * 7}
    own_rows = sum(lengths(B, case["rows"])) if case["ragged"] else B * case["rows"]
    shared = lengths(B, case["prefix"]) if case["ragged"] else [case["prefix"]] * B
    own_rows += B if case["new"] else 0
    keys = own_rows + max(shared)                    # rows read: the shared ones once
    pairs = own_rows + sum(shared)                   # rows that queries meet
    lens = 4 * B * (bool(case["rows"]) + bool(case["prefix"])) if case["ragged"] else 0
    return {"bytes": keys * H * D * 2 * width + 2 * B * G * D * width + 4 * B * G + lens,
            "flops": 4 * pairs * G * D}


def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence and key head by key head."""
    s = prepare(case, seed)
    if case["op"] == "qk":
        B, S, D = case["batch"], case["seq"], case["dim"]
        half = D // 2
        outs = [torch.empty(x.shape, dtype=torch.float64, device="cuda") for x in (s["q"], s["k"])]
        freq = torch.tensor([case["theta"] ** (-2.0 * i / D) for i in range(half)], dtype=torch.float64, device="cuda")
        for b in range(B):
            at = torch.arange(S, device="cuda") + s["pos0"] if s["positions"] is None else s["positions"][b]
            turn = torch.polar(torch.ones(S, half, dtype=torch.float64, device="cuda"), torch.outer(at.double(), freq))
            for x, weight, out in zip((s["q"], s["k"]), (s["q_weight"], s["k_weight"]), outs):
                y = x[b].double()
                y = y / torch.sqrt(torch.linalg.vector_norm(y, dim=-1, keepdim=True) ** 2 / D + EPS) * weight.double()
                z = torch.complex(y[..., :half], y[..., half:]) * turn[:, None]
                out[b] = torch.cat([z.real, z.imag], -1)
        return tuple(outs)
    B, H, G, D = case["batch"], case["kv_heads"], case["heads"], case["dim"]
    N = G // H
    out = torch.zeros(B, G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, G), -math.inf, dtype=torch.float64, device="cuda")
    if not case["rows"] and not case["new"]:
        # the prefix alone: all sequences at once, some hundred MB of logits at a time
        step = max(1, 2 ** 26 // (N * case["prefix"]))
        for h in range(H):
            keys, values = s["prefix_k"][h].double(), s["prefix_v"][h].double()
            for b in range(0, B, step):
                q = s["q"][b:b + step, h * N:h * N + N].double()
                logits = torch.mm(q.reshape(-1, D), keys.T).div_(D ** 0.5).view(-1, N, case["prefix"])
                if s["prefix_lens"] is not None:
                    past = torch.arange(case["prefix"], device="cuda") >= s["prefix_lens"][b:b + step, None]
                    logits.masked_fill_(past[:, None], -math.inf)
                total = torch.logsumexp(logits, -1, keepdim=True)
                weights = logits.sub_(total).exp_().nan_to_num_(nan=0.0)
                out[b:b + step, h * N:h * N + N] = torch.mm(weights.view(-1, case["prefix"]), values).view(-1, N, D)
                lse[b:b + step, h * N:h * N + N] = total[..., 0]
        return out, lse
    for h in range(H):
        for b in range(B):
            q = s["q"][b, h * N:h * N + N].double()
            keys, values = [], []
            if s["prefix_k"] is not None:
                n = case["prefix"] if s["prefix_lens"] is None else int(s["prefix_lens"][b])
                keys.append(s["prefix_k"][h, :n]), values.append(s["prefix_v"][h, :n])
            if s["k"] is not None:
                n = case["rows"] if s["lens"] is None else int(s["lens"][b])
                keys.append(s["k"][b, h, :n]), values.append(s["v"][b, h, :n])
            if s["k_new"] is not None:
                keys.append(s["k_new"][b, h, None]), values.append(s["v_new"][b, h, None])
            keys, values = torch.cat(keys).double(), torch.cat(values).double()
            if len(keys):
                logits = q @ keys.T / D ** 0.5
                lse[b, h * N:h * N + N] = torch.logsumexp(logits, -1)
                out[b, h * N:h * N + N] = torch.softmax(logits, -1) @ values
    return out, lse
