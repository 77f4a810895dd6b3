"""Weights far below the largest one: a dominant key in front of a long tail."""
import math

import pytest

torch = pytest.importorskip("torch")
import attention_reference as ref  # noqa: E402
from attention_paths import make  # noqa: E402

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
# The power of two by which fp16 weights are multiplied: the smallest step of fp16, 2^-24, is that much less beside the
# largest weight.
LIFT_ROWS = 15


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
