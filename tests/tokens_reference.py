"""Plain 64-bit forms of attention with several query tokens a sequence and of joins, with the error bounds their
16- and 32-bit computation is held to. Test infrastructure."""
import math

import torch

import attention_reference as ref


def attend(q, keys, values, visible, scale):
    """q [n, N, D], keys, values [m, D], visible [n, m] -> out [n, N, D], lse [n, N] and their bounds.

    The bounds are those of attention_reference.attend, row by row over the keys that the row sees: half a step for the
    output's rounding and one for the weights' 16 bits, the fp32 dot products' error in every weight, chains of sums.
    """
    dtype, (n, N, D) = q.dtype, q.shape
    q, keys, values = q.double(), keys.double(), values.double()
    s = torch.einsum("tnd,kd->tnk", q, keys) * scale
    hidden = ~visible[:, None, :]
    s = s.masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None]).masked_fill(hidden, 0.0)
    out = torch.einsum("tnk,kd->tnd", p, values)
    size = torch.einsum("tnk,kd->tnd", p, values.abs())
    sizes = torch.einsum("tnd,kd->tnk", q.abs(), keys.abs()) * scale
    delta = 2.0 ** -21 * sizes.masked_fill(hidden, 0.0).amax(-1)
    count = visible.sum(-1)[:, None].double()
    chain = (count / 16 + 64) * 2.0 ** -23
    half = ref.HALF_STEP[dtype]
    bound = half * (out.abs() + size) + size * (2 * delta + chain + 2.0 ** -20)[..., None]
    if dtype == torch.float16:
        largest = torch.exp(s.amax(-1) - lse)[..., None]
        bound = bound + 2.0 ** -25 + 2.0 ** -25 * largest * (visible.double() @ values.abs())[:, None]
    return out, lse, bound, delta + chain + 2.0 ** -21 * lse.abs() + 2.0 ** -21


def sequences(q, k_new, starts=None, new_lens=None):
    """(index of the batch, slice of tokens) of every sequence, as the library clamps them."""
    if q.dim() == 3:
        T = q.shape[0]
        at = [0, T] if starts is None else starts.tolist()
        out = []
        for x, y in zip(at, at[1:]):
            x = min(max(x, 0), T)
            out.append((slice(x, max(x, min(max(y, 0), T))),))
        return out
    B, S = q.shape[:2]
    return [(b, slice(0, S if new_lens is None else min(max(int(new_lens[b]), 0), S))) for b in range(B)]


def ancestors(parents, n):
    """[n, n]: whether token i sees token j."""
    seen = torch.zeros(n, n, dtype=torch.bool)
    for i in range(n):
        j = i
        while True:
            seen[i, j] = True
            p = int(parents[j])
            if p < 0 or p >= j:
                break
            j = p
    return seen


def attend_batch(q, *, k_new, v_new, starts=None, new_lens=None, parents=None, k=None, v=None, lens=None, scale=None):
    """The same for a batch; arguments as the library's attend_prompt and attend_tree. Also where tokens are."""
    G, D = q.shape[-2:]
    H = k_new.shape[-2]
    N = G // H
    scale = D ** -0.5 if scale is None else scale
    outs = [torch.zeros(q.shape, dtype=torch.float64, device=q.device) for _ in range(2)]
    lses = [torch.zeros(q.shape[:-1], dtype=torch.float64, device=q.device) for _ in range(2)]
    there = torch.zeros(q.shape[:-2], dtype=torch.bool, device=q.device)
    for b, at in enumerate(sequences(q, k_new, starts, new_lens)):
        there[at] = True
        n = q[at].shape[0]
        m = 0 if k is None else k.shape[2] if lens is None else min(max(int(lens[b]), 0), k.shape[2])
        if n == 0:
            continue
        if parents is None:
            seen = torch.ones(n, n, dtype=torch.bool).tril()
        else:
            seen = ancestors((parents if parents.dim() == 1 else parents[b]).tolist(), n)
        visible = torch.cat([torch.ones(n, m, dtype=torch.bool), seen], 1).to(q.device)
        for h in range(H):
            keys, values = k_new[at][:, h], v_new[at][:, h]
            if m:
                keys, values = torch.cat([k[b, h, :m], keys]), torch.cat([v[b, h, :m], values])
            some = slice(h * N, h * N + N)
            step = max(1, 2 ** 25 // (N * (n + m)))
            for i in range(0, n, step):
                part = slice(i, i + step)
                got = attend(q[at][part, some], keys, values, visible[part], scale)
                for to, x in zip((outs[0], lses[0], outs[1], lses[1]), got):
                    to[at][part, some] = x
    return outs[0], lses[0], outs[1], lses[1], there


def check(name, call, q, *, out=None, lse=None, **args):
    """Runs one of the library's calls and holds out and lse to the reference; what it must not write stays."""
    out = torch.full_like(q, 7.0) if out is None else out
    lse = torch.full(q.shape[:-1], 7.0, dtype=torch.float32, device=q.device) if lse is None else lse
    call(q, out, lse=lse, **args)
    torch.cuda.synchronize()
    want, wlse, bound, lbound, there = attend_batch(q, **args)
    assert (out[~there] == 7.0).all() and (lse[~there] == 7.0).all(), f"{name}: written behind a sequence"
    ref.check(name + " out", out[there], want[there], bound[there])
    ref.check(name + " lse", lse[there], wlse[there], lbound[there])
    return out, lse


def join(parts):
    """Parts (out [.., D], lse [..]) -> out, lse and their bounds: half a step for the output's rounding; weights within
    2^-21 and a sum of at most 8 terms, 2^-20 of the sizes that go in."""
    dtype = parts[0][0].dtype
    lses = torch.stack([x.double() for _, x in parts])
    lse = torch.logsumexp(lses, 0)
    out = torch.zeros(parts[0][0].shape, dtype=torch.float64, device=lse.device)
    size = torch.zeros_like(out)
    for part, x in parts:
        w = torch.exp(x.double() - lse).nan_to_num(nan=0.0)[..., None]
        part = part.double().masked_fill((x == -math.inf)[..., None], 0.0)
        out += w * part
        size += w * part.abs()
    # the difference of two log sums is within 2^-24 of the larger one's size
    spread = torch.where(lses.isfinite(), lses.abs(), 0.0).amax(0)[..., None] * 2.0 ** -22
    bound = ref.HALF_STEP[dtype] * out.abs() + size * (2.0 ** -20 + spread) + 2.0 ** -25
    return out, lse, bound, 2.0 ** -21 + 2.0 ** -22 * torch.where(lse.isfinite(), lse.abs(), 0.0)
