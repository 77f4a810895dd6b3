"""The shared rows without the tensor-core kernel: the row kernel answers the same calls."""
import pytest

torch = pytest.importorskip("torch")
import attention_reference as ref  # noqa: E402
from attention_paths import make, prefix_kernel  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture
def kvx():
    import kv_cache_attention_02_gb300 as k
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield k
    k.lib().kvevict_test_without_prefix_kernel(0)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("B,N,H,D,P,n,new", [(32, 4, 8, 128, 1100, 0, False), (32, 4, 8, 128, 1100, 0, True),
                                            (33, 4, 4, 64, 4000, 90, True), (300, 5, 2, 64, 901, 0, False),
                                            (300, 2, 2, 128, 901, 200, False)])
def test_same_answers(kvx, B, N, H, D, P, n, new, dtype):
    q, rows = make(B, N, H, D, P=P, n=n, new=new, dtype=dtype, seed=P + n)
    lens = torch.arange(B, dtype=torch.int32, device="cuda") * P // B
    assert prefix_kernel(kvx, q, **rows)
    assert kvx.lib().kvevict_test_without_prefix_kernel(1) == kvx.OK
    assert not prefix_kernel(kvx, q, **rows)
    ref.check_attend(kvx, q, **rows)
    ref.check_attend(kvx, q, prefix_lens=lens, **rows)
    assert kvx.lib().kvevict_test_without_prefix_kernel(0) == kvx.OK
    assert prefix_kernel(kvx, q, **rows)
    ref.check_attend(kvx, q, prefix_lens=lens, **rows)


def test_a_handle(kvx):
    B, N, H, D, P = 32, 4, 8, 128, 1100
    q, rows = make(B, N, H, D, P=P, new=True, seed=1)
    h = kvx.KVEvict(batch=B, n_layers=1, n_kv_heads=H, head_dim=D, layer_budgets=[8], n_sink=1, max_prefill=4, with_values=True)
    want = ref.attend_batch(q, **rows)
    for without in (1, 0):
        assert kvx.lib().kvevict_test_without_prefix_kernel(without) == kvx.OK
        out, lse = torch.empty_like(q), torch.empty(B, N * H, device="cuda")
        h.attend(0, q, out, lse=lse, **rows)
        torch.cuda.synchronize()
        ref.check("out", out, want[0], want[2])
        ref.check("lse", lse, want[1], want[3])
