"""Plain 64-bit forms of the query/key norm with rotation and of attention, with
the error bounds their 16- and 32-bit computation is held to. Test infrastructure."""
import math

import torch

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def qk(x, weight, positions, theta, eps):
    """x [B, S, heads, D] of any type, positions [B, S] -> (result, size of the rotated pair), fp64."""
    D = x.shape[-1]
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * weight.double()
    w = torch.tensor([theta ** (-2.0 * i / D) for i in range(D // 2)], dtype=torch.float64, device=x.device)
    ang = positions.double()[..., None] * w
    c, s = ang.cos()[:, :, None], ang.sin()[:, :, None]
    a, b = y[..., : D // 2], y[..., D // 2:]
    size = a.abs() + b.abs()
    return torch.cat([a * c - b * s, a * s + b * c], -1), torch.cat([size, size], -1)


def qk_bound(ref, size, dtype):
    """Half a step of the output type; fp32 arithmetic: the norm's sum, root and two products and the rotation's
    three operations are 16 roundings at most with sin and cos within 2 steps, 2^-20 of the pair with room; an fp16
    result below 2^-14 is off by half its smallest step, 2^-25."""
    return HALF_STEP[dtype] * ref.abs() + 2.0 ** -20 * size + 2.0 ** -25


def attend(q, keys, values, scale):
    """q [N, D], keys, values [n, D] -> out [N, D], lse [N], bound of out as a share-free absolute error, bound of lse."""
    n, D = keys.shape
    dtype = q.dtype
    q, keys, values = q.double(), keys.double(), values.double()
    N = q.shape[0]
    if n == 0:
        z = torch.zeros(N, D, dtype=torch.float64, device=q.device)
        return z, torch.full((N,), -math.inf, dtype=torch.float64, device=q.device), z, torch.zeros_like(z[:, 0])
    s = q @ keys.T * scale
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[:, None])
    out = p @ values
    size = p @ values.abs()
    # fp32 dot product: within 2^-21 of the sum of the products' sizes (D <= 128 terms in groups of 16, each group and
    # the scaling rounded); it moves every weight by at most that much, and their sum too
    delta = (2.0 ** -21 * (q.abs() @ keys.abs().T) * scale).amax(-1)
    # sums of n terms in chains of at most n / 16 + 64 additions of 2^-24 each, numerator and denominator
    chain = (n / 16 + 64) * 2.0 ** -23
    # weights in 16 bits: half a step each, and below fp16's normal range 2^-25 of the largest weight
    low = 2.0 ** -25 * torch.exp(s.amax(-1) - lse)[:, None] * values.abs().sum(0) if dtype == torch.float16 else 0.0
    bound = HALF_STEP[dtype] * (out.abs() + size) + size * (2 * delta[:, None] + chain + 2.0 ** -20) + low
    if dtype == torch.float16:
        bound = bound + 2.0 ** -25
    return out, lse, bound, delta + chain + 2.0 ** -21 * lse.abs() + 2.0 ** -21


def check(name, got, ref, bound):
    got = got.double()
    assert got.shape == ref.shape, name
    same = torch.isinf(ref) | torch.isnan(ref)
    assert torch.equal(got[same].nan_to_num(nan=7.0), ref[same].nan_to_num(nan=7.0)), f"{name}: infinities differ"
    off = (got - ref).abs()[~same] - bound.expand_as(ref)[~same]
    assert not torch.isnan(got[~same]).any(), f"{name}: NaN"
    if off.numel():
        assert off.max() <= 0, f"{name}: over its bound by {off.max().item():.3g} (bound {bound.max().item():.3g})"


def attend_batch(q, scale=None, k=None, v=None, lens=None, k_new=None, v_new=None, prefix_k=None, prefix_v=None,
                 prefix_lens=None):
    """The same for a batch; arguments as the library's attend."""
    B, G, D = q.shape
    H = (k if k is not None else k_new).shape[1] if k is not None or k_new is not None else prefix_k.shape[0]
    N = G // H
    scale = D ** -0.5 if scale is None else scale
    outs = [torch.zeros(B, G, D, dtype=torch.float64, device=q.device) for _ in range(2)]
    lses = [torch.zeros(B, G, dtype=torch.float64, device=q.device) for _ in range(2)]
    for b in range(B):
        n = 0 if k is None else k.shape[2] if lens is None else min(max(int(lens[b]), 0), k.shape[2])
        P = 0 if prefix_k is None else prefix_k.shape[1] if prefix_lens is None else \
            min(max(int(prefix_lens[b]), 0), prefix_k.shape[1])
        for h in range(H):
            keys, values = [q.new_zeros(0, D)], [q.new_zeros(0, D)]
            if P:
                keys.append(prefix_k[h, :P]), values.append(prefix_v[h, :P])
            if n:
                keys.append(k[b, h, :n]), values.append(v[b, h, :n])
            if k_new is not None:
                keys.append(k_new[b, h, None]), values.append(v_new[b, h, None])
            some = slice(h * N, h * N + N)
            outs[0][b, some], lses[0][b, some], outs[1][b, some], lses[1][b, some] = \
                attend(q[b, some], torch.cat(keys), torch.cat(values), scale)
    return outs[0], lses[0], outs[1], lses[1]


def check_attend(kvx, q, *, scale=None, out=None, **rows):
    """Runs the library's attend and holds out and lse to the reference."""
    out = torch.full_like(q, float("nan")) if out is None else out
    lse = torch.full(q.shape[:2], float("nan"), dtype=torch.float32, device=q.device)
    kvx.attend(q, out, lse=lse, scale=scale, **rows)
    torch.cuda.synchronize()
    ref, rlse, bound, lbound = attend_batch(q, scale, **rows)
    check("out", out, ref, bound)
    check("lse", lse, rlse, lbound)
    return out, lse
