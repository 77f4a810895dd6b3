"""Timed cases of attention with several query tokens a sequence, around the eviction cache.

Three operators, as a serving loop uses them on one layer:

* ``attend_prompt``: causal attention of whole prompts, packed one behind another or a padded batch,
  grouped heads; also a chunk of a prompt behind rows that the sequence already has.
* ``attend_tree``: a tree of drafted tokens per sequence; each token sees the sequence's rows, itself
  and its ancestors.
* ``attend_join``: joins the results of attention over disjoint rows (a shared prefix's part and the
  rest) by their log sums.

``run`` computes a case with elementary torch operations, or with the library's calls where ``own``
is set. ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    def prompt(name, batch, seq, heads, kv_heads, dim, dtype, packed=False, ragged=False, rows=0):
        return {"name": name, "op": "prompt", "batch": batch, "seq": seq, "heads": heads, "kv_heads": kv_heads,
                "dim": dim, "dtype": dtype, "packed": packed, "ragged": ragged, "rows": rows}

    def tree(name, batch, tokens, heads, kv_heads, dim, rows, dtype, ragged=False):
        return {"name": name, "op": "tree", "batch": batch, "tokens": tokens, "heads": heads, "kv_heads": kv_heads,
                "dim": dim, "rows": rows, "dtype": dtype, "ragged": ragged}

    def join(name, tokens, heads, dim, parts, dtype):
        return {"name": name, "op": "join", "tokens": tokens, "heads": heads, "dim": dim, "parts": parts, "dtype": dtype}

    return [
        # a question of a few words on the smallest heads: all latency
        prompt("prompt_short", 1, 37, 4, 4, 64, "fp16"),
        # one prompt as long as its budget, three query heads a key head
        prompt("prompt_512", 1, 512, 24, 8, 128, "fp16"),
        # prompts of very unequal lengths packed one behind another, an empty and a one-token one among them
        prompt("prompt_packed", 11, 5003, 40, 8, 128, "bf16", packed=True, ragged=True),
        # a batch of equal prompts of the large cache: bound by arithmetic
        prompt("prompt_large", 8, 4096, 32, 8, 128, "bf16"),
        # chunks of long prompts behind the rows that earlier chunks left
        prompt("prompt_chunk", 3, 1000, 32, 8, 128, "fp16", ragged=True, rows=16384),
        # small heads, many short prompts in a padded batch
        prompt("prompt_batch_dim64", 48, 700, 16, 4, 64, "fp16", ragged=True),
        # eight drafted tokens on the 32 rows of the smallest cache
        tree("tree_small", 1, 8, 4, 4, 64, 32, "fp16"),
        # a single conversation at budget 512, sixteen drafted tokens
        tree("tree_budget512", 1, 16, 24, 8, 128, 512, "fp16"),
        # one layer of 32 sequences at the average budget of the large cache
        tree("tree_budget2048_batch32", 32, 16, 32, 8, 128, 2048, "fp16"),
        # unequal sequences that kept everything, wide trees
        tree("tree_long_ragged", 7, 63, 40, 8, 128, 65521, "bf16", ragged=True),
        # a decode step's shared and own parts of 32 sequences
        join("join_step", 32, 32, 128, 2, "fp16"),
        # a prompt chunk's three parts
        join("join_chunk", 16384, 32, 128, 3, "bf16"),
    ]


MOST = 4 * 128 * 32 * 8 * 4096 * 4097 // 2      # the largest listed case's products


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))

    dim, dtype = rng.choice([64, 128, 128]), rng.choice(["fp16", "bf16"])
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    op = rng.choice(["prompt", "prompt", "tree", "tree", "join"])
    if op == "prompt":
        case = {"op": op, "heads": heads, "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "packed": rng.random() < 0.5,
                "ragged": rng.random() < 0.6, "rows": rng.choice([0, 0, log(1, 32768)])}
        case["seq"] = log(1, 8192)
        fits = MOST // (4 * dim * heads * case["seq"] * (case["rows"] + (case["seq"] + 1) // 2))
        case["batch"] = log(1, max(1, min(64, fits, 65536 // case["seq"], 3000000 // (kv_heads * (case["rows"] + 1)))))
        while work(case)["flops"] > MOST:
            case["seq"] = case["seq"] * 7 // 8
        return case
    if op == "tree":
        case = {"op": op, "heads": heads, "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "rows": log(1, 65521),
                "tokens": log(1, 64), "ragged": rng.random() < 0.5}
        case["batch"] = log(1, max(1, min(128, 3000000 // (case["rows"] * kv_heads))))
        return case
    tokens, parts = log(1, 32768), rng.choice([2, 2, 3, 4])
    return {"op": op, "tokens": max(1, min(tokens, 2 ** 31 // (8 * heads * dim * parts))), "heads": heads, "dim": dim, "parts": parts,
            "dtype": dtype}


def lengths(count, top):
    """Unequal lengths in 0 .. top, spread over it; the first is the whole, the next two are nothing and one."""
    found = [int(top * ((0.6180339887 * i) % 1.0)) for i in range(count)]
    found[:3] = [top, 0, min(1, top)][:count]
    return found


def sizes(case):
    """Tokens and rows of each sequence."""
    B = case["batch"]
    most = case["seq"] if case["op"] == "prompt" else case["tokens"]
    # a tree has its full count, but for a batch's last sequence, which drafted fewer
    tokens = [most] * B
    if case["ragged"]:
        tokens = lengths(B, most) if case["op"] == "prompt" else [most] * (B - 1) + [(most + 1) // 2]
    rows = [case["rows"]] * B
    if case["ragged"] and case["rows"]:
        # the longest, then unequal ones, an empty one among them, in another order than the tokens'
        rows = lengths(B, case["rows"])
        rows = rows[:1] + rows[:0:-1]
    return tokens, rows


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16) * scale).to(dtype)

    D, G = case["dim"], case["heads"]
    if case["op"] == "join":
        T = case["tokens"]
        parts = []
        for _ in range(case["parts"]):
            lse = torch.randn((T, G), generator=gen, device="cuda") * 2 + 6
            # some tokens have no rows in a part
            lse.masked_fill_(torch.rand((T, G), generator=gen, device="cuda") < 0.05, -math.inf)
            part = normal(T, G, D, scale=0.3)
            part.masked_fill_((lse == -math.inf)[..., None], 0.0)
            parts.append((part, lse))
        return {"case": case, "parts": parts, "out": torch.empty(T, G, D, dtype=dtype, device="cuda"),
                "lse": torch.empty(T, G, device="cuda")}
    B, H = case["batch"], case["kv_heads"]
    tokens, rows = sizes(case)
    state = {"case": case, "k": None, "v": None, "lens": None, "new_lens": None, "starts": None, "parents": None}

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    if case["op"] == "prompt" and case["packed"]:
        total = sum(tokens)
        state["q"] = normal(total, G, D, scale=1.5)
        state["k_new"] = normal(total, H, D)
        # values as the fused projection left them, behind a token's queries and keys
        state["v_new"] = normal(total, G + 2 * H, D)[:, G + H:]
        state["starts"] = ints([sum(tokens[:b]) for b in range(B + 1)])
    else:
        S = case["seq"] if case["op"] == "prompt" else case["tokens"]
        state["q"] = normal(B, S, G, D, scale=1.5)
        # keys in the layout that the cache takes a layer's prompt in, or a step's keys
        state["k_new"] = normal(B, H, S, D).transpose(1, 2)
        state["v_new"] = normal(B, H, S, D).transpose(1, 2)
        if case["ragged"]:
            state["new_lens"] = ints(tokens)
    if case["op"] == "tree":
        # every token continues one of those before it, or the sequence itself
        before = torch.arange(case["tokens"] + 0.0, device="cuda") + 1
        state["parents"] = (torch.rand((B, case["tokens"]), generator=gen, device="cuda") * before).int().clamp(max=before.int() - 1) - 1
    if case["rows"]:
        state["k"], state["v"] = normal(B, H, case["rows"], D), normal(B, H, case["rows"], D)
        if case["ragged"]:
            state["lens"] = ints(rows)
    # tokens past a sequence's length stay as they are
    state["out"] = torch.zeros_like(state["q"])
    state["lse"] = torch.zeros(state["q"].shape[:-1], device="cuda")
    return state


def run(state):
    op = state["case"]["op"]
    if own:
        import kv_cache_attention_02_gb300 as kvx
        if op == "join":
            kvx.attend_join(state["out"], state["parts"], lse=state["lse"])
        elif op == "prompt":
            kvx.attend_prompt(state["q"], state["out"], k_new=state["k_new"], v_new=state["v_new"], starts=state["starts"],
                              new_lens=state["new_lens"], k=state["k"], v=state["v"], lens=state["lens"], lse=state["lse"])
        else:
            kvx.attend_tree(state["q"], state["out"], k_new=state["k_new"], v_new=state["v_new"], parents=state["parents"],
                            new_lens=state["new_lens"], k=state["k"], v=state["v"], lens=state["lens"], lse=state["lse"])
        return state["out"], state["lse"]
    return run_join(state) if op == "join" else run_tokens(state)


def run_join(s):
    lses = torch.stack([lse for _, lse in s["parts"]])
    top = lses.amax(0)
    top = torch.where(top == -math.inf, 0.0, top)
    weights = torch.exp(lses - top)
    total = weights.sum(0)
    out = sum(part.float() * w[..., None] for (part, _), w in zip(s["parts"], weights))
    return (out / torch.where(total == 0, 1.0, total)[..., None]).to(s["out"].dtype), top + torch.log(total)


def run_tokens(s):
    c = s["case"]
    B, H, G, D = c["batch"], c["kv_heads"], c["heads"], c["dim"]
    N = G // H
    tokens, rows = sizes(c)
    out, lse = torch.zeros_like(s["q"]), torch.zeros_like(s["lse"])
    seen = None
    if c["op"] == "tree":
        # who is before whom: powers of "itself or its parent", up to the deepest tree
        T = c["tokens"]
        index = torch.arange(T, device="cuda")
        seen = ((s["parents"][:, :, None] == index) | (index[:, None] == index)).float()
        for _ in range(max(1, (T - 1).bit_length())):
            seen = ((seen @ seen) > 0).float()
    begin = 0
    for b in range(B):
        n, m = tokens[b], rows[b]
        if s["starts"] is not None:
            here = slice(begin, begin + n)
            q, k, v, to, to_lse = s["q"][here], s["k_new"][here], s["v_new"][here], out[here], lse[here]
            begin += n
        else:
            q, k, v, to, to_lse = s["q"][b, :n], s["k_new"][b, :n], s["v_new"][b, :n], out[b, :n], lse[b, :n]
        if not n:
            continue
        q = q.float().view(n, H, N, D).permute(1, 2, 0, 3) / math.sqrt(D)
        k, v = k.float().transpose(0, 1), v.float().transpose(0, 1)
        if m:
            k, v = torch.cat([s["k"][b, :, :m].float(), k], 1), torch.cat([s["v"][b, :, :m].float(), v], 1)
        if seen is None:
            at = torch.arange(n, device="cuda")
            hidden = at[None] > at[:, None]
        else:
            hidden = seen[b, :n, :n] == 0
        # some GB of logits at a time
        step = max(1, min(H, 2 ** 30 // (N * n * (n + m))))
        for h in range(0, H, step):
            some = slice(h, h + step)
            logits = (q[some].reshape(-1, N * n, D) @ k[some].transpose(1, 2)).view(-1, N, n, n + m)
            logits[..., m:].masked_fill_(hidden, -math.inf)
            top = logits.amax(-1, keepdim=True)
            logits = logits.sub_(top).exp_()
            total = logits.sum(-1, keepdim=True)
            result = (logits.view(-1, N * n, n + m) @ v[some]).view(-1, N, n, D) / total
            to.view(n, H, N, D)[:, some] = result.permute(2, 0, 1, 3).to(out.dtype)
            to_lse.view(n, H, N)[:, some] = (top + torch.log(total))[..., 0].permute(2, 0, 1)
    return out, lse


def work(case):
    G, D = case["heads"], case["dim"]
    if case["op"] == "join":
        heads = case["tokens"] * G
        # a weight, its product and its sum for every part
        return {"bytes": heads * (2 * D + 4) * (case["parts"] + 1), "flops": heads * D * 2 * case["parts"]}
    H = case["kv_heads"]
    tokens, rows = sizes(case)
    pairs = 0
    for n, m in zip(tokens, rows):
        # a tree's tokens see some of the others: at least themselves
        pairs += n * m + (n * (n + 1) // 2 if case["op"] == "prompt" else n)
    data = 4 * D * H * (sum(tokens) + sum(m for n, m in zip(tokens, rows) if n)) + sum(tokens) * G * (4 * D + 4)
    ints = 4 * case["batch"] * (bool(case["ragged"] or case.get("packed")) + bool(case["ragged"] and case["rows"]))
    if case["op"] == "tree":
        ints += 4 * sum(tokens)
    return {"bytes": data + ints, "flops": 4 * pairs * G * D}


def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence and key head by key head."""
    s = prepare(case, seed)
    if case["op"] == "join":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        lse = torch.logsumexp(torch.stack([x.double() for _, x in s["parts"]]), 0)
        for part, x in s["parts"]:
            share = torch.exp(x.double() - lse).nan_to_num_(nan=0.0)       # (no rows at all: -inf less -inf)
            out.addcmul_(part.double(), share[..., None])
        return out, lse
    H, G, D = case["kv_heads"], case["heads"], case["dim"]
    N = G // H
    tokens, rows = sizes(case)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    parents = s["parents"].tolist() if s["parents"] is not None else None
    first = 0
    for b, (n, m) in enumerate(zip(tokens, rows)):
        if s["starts"] is None:
            pick = (b, slice(0, n))
        else:
            pick = (slice(first, first + n),)
            first += n
        if n == 0:
            continue
        if parents is None:
            allowed = torch.ones(n, n, dtype=torch.bool, device="cuda").tril_()
        else:
            allowed = [[False] * n for _ in range(n)]
            for i in range(n):
                j = i
                while j >= 0:
                    allowed[i][j] = True
                    j = parents[b][j]
            allowed = torch.tensor(allowed, device="cuda")
        block = max(1, 2 ** 27 // (N * (n + m)))        # query tokens at a time
        for h in range(H):
            keys, values = s["k_new"][pick][:, h].double(), s["v_new"][pick][:, h].double()
            if m:
                keys, values = torch.cat([s["k"][b, h, :m].double(), keys]), torch.cat([s["v"][b, h, :m].double(), values])
            for i in range(0, n, block):
                some = slice(i, min(n, i + block))
                q = s["q"][pick][some, h * N:h * N + N].double()
                logits = torch.einsum("tnd,kd->tnk", q, keys).div_(D ** 0.5)
                logits[..., m:].masked_fill_(~allowed[some, None], -math.inf)
                total = torch.logsumexp(logits, -1, keepdim=True)
                result = torch.einsum("tnk,kd->tnd", logits.sub_(total).exp_(), values)
                out[pick][some, h * N:h * N + N] = result
                lse[pick][some, h * N:h * N + N] = total[..., 0]
    return out, lse
