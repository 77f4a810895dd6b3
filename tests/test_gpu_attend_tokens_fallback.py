"""Prompts and drafted trees without the tensor-core kernel: the kernel for few query rows answers the same calls."""
import pytest

torch = pytest.importorskip("torch")
import tokens_reference as tref  # noqa: E402
from tokens_inputs import ints, make, normal, trees  # noqa: E402

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture
def kvx():
    import kv_cache_attention_02_gb300 as k
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    assert k.lib().kvevict_test_without_tokens_kernel(1) == k.OK
    yield k
    assert k.lib().kvevict_test_without_tokens_kernel(0) == k.OK


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("B,S,N,H,D,n", [(4, 256, 1, 8, 128, 0), (2, 1100, 4, 2, 64, 0), (3, 300, 3, 2, 128, 700),
                                         (1, 400, 4, 2, 64, 3000), (2, 60, 130, 2, 64, 33)])
def test_prompts(kvx, B, S, N, H, D, n, dtype):
    q, args = make(B, S, N, H, D, n=n, dtype=dtype, seed=S)
    tref.check("prompt", kvx.attend_prompt, q, **args)
    lens = ints(*[n * (b + 1) // (B + 1) for b in range(B)]) if n else None
    tref.check("ragged prompt", kvx.attend_prompt, q, new_lens=ints(*[S - 40 * b for b in range(B)]), lens=lens, **args)


@pytest.mark.parametrize("B", [1, 128, 129, 300])
@pytest.mark.parametrize("N,n", [(3, 0), (4, 50)])
def test_packed(kvx, B, N, n):
    gen = torch.Generator().manual_seed(B)
    count = torch.randint(0, 12, (B,), generator=gen)
    count[-1] = 400
    at = torch.cat([torch.zeros(1, dtype=torch.long), count.cumsum(0)]).int()
    q, args = make(B, int(at[-1]) + 5, N, 2, 64, n=n, dtype=BF16, packed=True, seed=B)
    lens = torch.randint(0, n + 1, (B,), generator=gen, dtype=torch.int32).cuda() if n else None
    tref.check("packed", kvx.attend_prompt, q, starts=at.cuda(), lens=lens, **args)


@pytest.mark.parametrize("B,T,N,H,D,n", [(9, 16, 4, 8, 128, 3000), (2, 64, 16, 1, 128, 5000), (40, 64, 5, 2, 64, 300)])
def test_trees(kvx, B, T, N, H, D, n):
    q, args = make(B, T, N, H, D, n=n, seed=n)
    tref.check("tree", kvx.attend_tree, q, parents=trees(B, T, n), new_lens=ints(*[max(1, T - b) for b in range(B)]), **args)


def test_a_handle(kvx):
    """With a compaction pending, by either kernel."""
    B, H, D, N, T, budget = 9, 8, 128, 4, 16, 600
    kw = dict(batch=B, n_layers=1, n_kv_heads=H, head_dim=D, layer_budgets=[budget], n_sink=1, max_prefill=budget, with_values=True)
    h, twin = kvx.KVEvict(**kw), kvx.KVEvict(**kw)
    gen = torch.Generator(device="cuda").manual_seed(1)
    keys, values, k_new, v_new = (normal(gen, B, 1, H, *s, D) for s in ((budget,), (budget,), (), ()))
    for x in (h, twin):
        x.prefill(keys, values=values)
        x.step(k_new, v_new=v_new)
    torch.cuda.synchronize()
    rows = [[[torch.from_numpy(r.view("float16").copy()).cuda() for r in (twin.read_state(b, 0, g)[0], twin.read_values(b, 0, g))]
             for g in range(H)] for b in range(B)]
    k, v = (torch.stack([torch.stack([r[i] for r in row]) for row in rows]) for i in (0, 1))
    q, args = make(B, T, N, H, D, seed=T)
    for without in (1, 0):
        assert kvx.lib().kvevict_test_without_tokens_kernel(without) == kvx.OK
        tref.check("tree", lambda *x, k, v, **y: h.attend_tree(0, *x, **y), q, k=k, v=v, parents=trees(B, T, 1), **args)
    h.check()


def test_starts_that_do_not_ascend(kvx):
    """Sequences that overlap are computed or left out, whichever; rows of no sequence stay, and the call ends."""
    q, args = make(200, 300, 2, 2, 64, packed=True, seed=5)
    starts = ints(*[(0, 290)[i & 1] for i in range(201)])
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:-1], 7.0, device="cuda")
    kvx.attend_prompt(q, out, lse=lse, starts=starts, **args)
    torch.cuda.synchronize()
    assert (out[290:] == 7.0).all() and (lse[290:] == 7.0).all()
