"""Weights far below the largest one: a dominant key in front of a long tail, and logits of any size."""
import math

import pytest

torch = pytest.importorskip("torch")
import attention_reference as ref  # noqa: E402
from attention_paths import make, prefix_kernel, workspace  # noqa: E402

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
# The power of two that the largest fp16 weight is at least: the smallest step of fp16, 2^-24, is that much less beside it.
LIFT_ROWS, LIFT_PREFIX = 15, 7


@pytest.fixture(scope="module")
def kvx():
    import kv_cache_attention_02_gb300 as k
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    k.lib()
    return k


def _tight(q, keys, values, lift):
    """The reference with its allowance for fp16 weights below the normal range (2^-25 of the largest weight for every
    row) cut down to 2^-25 of 2^-lift."""
    scale = q.shape[-1] ** -0.5
    out, lse, bound, lbound = ref.attend(q, keys, values, scale)
    if q.dtype is F16:
        top = (q.double() @ keys.double().T * scale).amax(-1)
        low = 2.0 ** -25 * torch.exp(top - lse)[:, None] * values.double().abs().sum(0)
        bound = bound - low * (1 - 2.0 ** -lift)
    return out, lse, bound, lbound


def _tailed(B, N, H, D, rows, names, sink, nats, dtype):
    """One key `nats` above all others, at row `sink`, whose value is 0; the others' values are about 1."""
    q, data = make(B, N, H, D, dtype=dtype, seed=7, **rows)
    q *= 0.2
    q[..., 0] = 8.0
    for k, v in names:
        data[k] *= 0.25
        data[k][..., 0] = 0.0
        data[k][..., sink, :] = 0.0
        data[k][..., sink, 0] = nats * math.sqrt(D) / 8.0
        data[v].mul_(0.1).add_(1.0)
        data[v][..., sink, :] = 0.0
    return q, data


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("nats", [12.0, 17.8, 20.5])
@pytest.mark.parametrize("B,N,H,D,n", [(1, 4, 2, 128, 2000), (1, 4, 1, 128, 65521), (2, 12, 1, 64, 40001),
                                       (40, 4, 8, 128, 1300)])
@pytest.mark.parametrize("sink", ["first", "last"])
def test_own_rows(kvx, B, N, H, D, n, nats, dtype, sink):
    q, rows = _tailed(B, N, H, D, dict(n=n), [("k", "v")], 0 if sink == "first" else n - 1, nats, dtype)
    out, lse = torch.empty_like(q), torch.empty(B, N * H, device="cuda")
    kvx.attend(q, out, lse=lse, **rows)
    torch.cuda.synchronize()
    for b in range(0, B, max(1, B // 3)):
        for h in range(H):
            some = slice(h * N, h * N + N)
            want = _tight(q[b, some], rows["k"][b, h], rows["v"][b, h], LIFT_ROWS)
            ref.check("out", out[b, some], want[0], want[2])
            ref.check("lse", lse[b, some], want[1], want[3])


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("nats", [12.0, 17.8, 20.5])
@pytest.mark.parametrize("B,N,H,D,P", [(32, 4, 1, 128, 65521), (32, 4, 64, 128, 1300), (1024, 4, 8, 128, 1300), (700, 5, 8, 64, 1100)])
@pytest.mark.parametrize("sink", ["first", "middle", "last"])
@pytest.mark.parametrize("new", [False, True])
def test_shared_rows(kvx, B, N, H, D, P, nats, dtype, sink, new):
    at = {"first": 0, "middle": P // 2, "last": P - 1}[sink]
    q, rows = _tailed(B, N, H, D, dict(P=P, new=new), [("prefix_k", "prefix_v")], at, nats, dtype)
    if new:
        rows["k_new"][..., 0] = -8.0
    assert prefix_kernel(kvx, q, **rows)
    out, lse = torch.empty_like(q), torch.empty(B, N * H, device="cuda")
    kvx.attend(q, out, lse=lse, **rows)
    torch.cuda.synchronize()
    for b in range(0, B, B // 3):
        for h in range(0, H, 3):
            keys, values, some = rows["prefix_k"][h], rows["prefix_v"][h], slice(h * N, h * N + N)
            if new:
                keys, values = torch.cat([keys, rows["k_new"][b, h, None]]), torch.cat([values, rows["v_new"][b, h, None]])
            want = _tight(q[b, some], keys, values, LIFT_PREFIX)
            ref.check("out", out[b, some], want[0], want[2])
            ref.check("lse", lse[b, some], want[1], want[3])


@pytest.mark.parametrize("path", ["clusters", "ranges", "pair", "tiles"])
@pytest.mark.parametrize("size,dtype", [(1e3, F16), (3e4, F16), (1e6, F16), (1e8, F16), (3e4, BF16), (1e8, BF16), (1e11, BF16),
                                        (1e30, BF16)])
def test_logits_of_any_size(kvx, path, size, dtype):
    """Logits of the given size, in steps that the largest one grows by again and again, and the largest twice: the output
    is the mean of those two rows' values."""
    D, n = 128, 1200
    shape = {"clusters": (2, 2, 2), "ranges": (40, 2, 8), "pair": (64, 2, 4), "tiles": (64, 5, 4)}[path]
    shared = path in ("pair", "tiles")
    q, rows = make(*shape, D, dtype=dtype, seed=8, **({"P": n} if shared else {"n": n if path == "ranges" else 300}))
    k, v = (rows["prefix_k"], rows["prefix_v"]) if shared else (rows["k"], rows["v"])
    count = k.shape[-2]
    assert prefix_kernel(kvx, q, **rows) == shared and (workspace(kvx, q, **rows) > 0) == (path != "clusters")
    q.zero_()
    k.zero_()
    # q . k * scale = size * (step of the row), steps 2^-3 apart in size: exact products, sums of one term
    root = 2.0 ** (math.ceil(math.log2(size) / 2) + 1)
    q[..., 0] = root
    steps = (torch.arange(count, device="cuda") // (count // 8)).clamp(max=8) / 8 - 0.5
    steps[steps == steps.max()] = -0.5
    a, b = count - 3, count // 2
    steps[a] = steps[b] = 1.0
    k[..., 0] = (steps * (size / root) * math.sqrt(D)).to(dtype)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    kvx.attend(q, out, lse=lse, **rows)
    torch.cuda.synchronize()
    B, H, N = shape[0], shape[2], shape[1]
    # Two equal logits, so two equal weights w', each w rounded once to 16 bits, over a sum of two unrounded w: w' / w is
    # within half a step of 1, and the output is rounded once. (A weight that is not exactly 1, as the logit and the
    # maximum may be rounded apart, cancels.) The rest of the weights are below 2^-700. fp32: four roundings and an exp2.
    va, vb = v[..., a, :].double(), v[..., b, :].double()
    mean, size = [(x / 2).expand(B, H, D).repeat_interleave(N, 1) for x in (va + vb, va.abs() + vb.abs())]
    half = ref.HALF_STEP[dtype]
    ref.check("out", out, mean, half * (mean.abs() + size) + 2.0 ** -20 * size + (2.0 ** -25 if dtype is F16 else 0.0))
    top = float(q[0, 0, 0].double()) * float(k.reshape(-1, count, D)[0, a, 0].double()) * D ** -0.5
    assert (lse - (top + math.log(2))).abs().max() <= 2.0 ** -21 * abs(top) + 2.0 ** -20
