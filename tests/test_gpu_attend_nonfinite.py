"""Attention where keys or values are not finite: what they reach, and what they must not."""
import pytest

torch = pytest.importorskip("torch")
import attention_reference as ref  # noqa: E402
from attention_paths import make, prefix_kernel  # noqa: E402

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def kvx():
    import kv_cache_attention_02_gb300 as k
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    k.lib()
    return k


# Shapes of the tensor-core kernel: up to 128 query rows a key head, and more.
@pytest.mark.parametrize("B,N,H,D,P", [(32, 4, 8, 128, 1100), (100, 1, 4, 64, 1300), (60, 5, 8, 64, 1200), (300, 2, 2, 128, 901)])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("new", [False, True])
def test_keys_of_rows_that_a_sequence_does_not_share(kvx, B, N, H, D, P, dtype, new):
    """Lengths that differ by whole tiles of 128 rows, neighbours by neighbours; the keys past the shorter ones are NaN,
    infinite, or finite with a product that is not. The sequences that share none of them are as if there were none."""
    q, rows = make(B, N, H, D, P=P, new=new, dtype=dtype, seed=P)
    lens = torch.tensor([0, 128, 256, 896, 1, 130], dtype=torch.int32, device="cuda").repeat(B // 6 + 1)[:B]
    k = rows["prefix_k"]
    k[:, 300] = float("nan")
    k[:, 400, 3] = float("inf")
    k[:, 500, 5] = -float("inf")
    if dtype is BF16:
        q[..., 7] = 1e20
        k[:, :300, 7] = 0
        if new:
            rows["k_new"][..., 7] = 0
        k[:, 600, 7] = 1e30
    assert prefix_kernel(kvx, q, prefix_lens=lens, **rows)
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    kvx.attend(q, out, lse=lse, prefix_lens=lens, **rows)
    torch.cuda.synchronize()
    short = lens <= 256
    some = {name: x[short] if name.endswith("new") else x for name, x in rows.items()}
    want = ref.attend_batch(q[short], prefix_lens=lens[short], **some)
    ref.check("out", out[short], want[0], want[2])
    ref.check("lse", lse[short], want[1], want[3])
    assert torch.isnan(out[~short]).all() and torch.isnan(lse[~short]).all()


@pytest.mark.parametrize("B,N,H,D,P", [(32, 4, 8, 128, 1100), (300, 2, 2, 128, 901), (4, 2, 2, 64, 100)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_a_logit_of_minus_infinity_takes_no_weight(kvx, B, N, H, D, P, dtype):
    """As if its row were not there, below a length and past it."""
    q, rows = make(B, N, H, D, P=P, n=20, dtype=dtype, seed=4)
    q[..., 0] = 1.0
    less = {name: torch.cat([x[..., :5, :], x[..., 15:, :]], -2) for name, x in rows.items()}
    for name in ("prefix_k", "k"):
        rows[name][..., 5:15, 0] = -float("inf")
    lens = torch.tensor([P, P - 300 if P > 300 else 9], dtype=torch.int32, device="cuda").repeat(B)[:B]
    out, lse = torch.empty_like(q), torch.empty(B, N * H, device="cuda")
    kvx.attend(q, out, lse=lse, prefix_lens=lens, **rows)
    torch.cuda.synchronize()
    want = ref.attend_batch(q, prefix_lens=torch.where(lens > 15, lens - 10, lens.clamp(max=5)), **less)
    ref.check("out", out, want[0], want[2])
    ref.check("lse", lse, want[1], want[3])
