"""Attention of whole prompts and of trees of drafted tokens against their 64-bit forms."""
import pytest

torch = pytest.importorskip("torch")
import tokens_reference as tref  # noqa: E402
from tokens_inputs import ints, make, normal, trees  # noqa: E402

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", params=["chosen", "tensor"])
def kvx(request):
    """By the kernel that the library chooses (another one for few query rows), and all by the tensor cores'."""
    import kv_cache_attention_02_gb300 as k
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    k.lib().kvevict_test_without_few_kernel(request.param == "tensor")
    yield k
    k.lib().kvevict_test_without_few_kernel(0)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("S", [1, 2, 31, 42, 43, 127, 128, 129, 255, 257, 500, 1100])
def test_prompt_lengths(kvx, S, D, dtype):
    q, args = make(2, S, 3, 2, D, dtype=dtype, seed=S)
    tref.check("prompt", kvx.attend_prompt, q, **args)


@pytest.mark.parametrize("N", [1, 2, 3, 5, 7, 8, 12, 16, 40, 130])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [0, 75])
def test_prompt_head_groups(kvx, N, D, n):
    q, args = make(2, 190 if N < 100 else 30, N, 2, D, n=n, seed=N)
    tref.check("prompt", kvx.attend_prompt, q, **args)


@pytest.mark.parametrize("N", [64, 65, 100, 127, 128, 131, 256])
@pytest.mark.parametrize("D,n", [(64, 0), (128, 200)])
def test_many_query_heads_a_key_head(kvx, N, D, n):
    """One or two tokens a half block; more than 128 heads go in several groups (131, a prime: one each)."""
    q, args = make(2, 7, N, 2, D, n=n, dtype=BF16, seed=N)
    tref.check("prompt", kvx.attend_prompt, q, **args)
    tref.check("tree", kvx.attend_tree, q, parents=trees(2, 7, N), **args)


@pytest.mark.parametrize("B,S,N,H,D,n,dtype", [
    (1, 3000, 4, 1, 128, 0, F16), (1, 2500, 1, 3, 64, 0, BF16), (3, 2049, 5, 2, 128, 0, BF16), (1, 700, 3, 2, 128, 9000, F16),
    (2, 64, 8, 8, 128, 5000, BF16), (40, 300, 4, 8, 64, 0, F16), (5, 1, 4, 2, 128, 3001, F16), (1, 130, 16, 1, 64, 20000, BF16)])
def test_prompt_work_cut_over_the_gpu(kvx, B, S, N, H, D, n, dtype):
    """Blocks that end in another CTA than they began in, even lengths, then unequal ones."""
    q, args = make(B, S, N, H, D, n=n, dtype=dtype, seed=S)
    tref.check("prompt", kvx.attend_prompt, q, **args)
    gen = torch.Generator().manual_seed(S)
    new_lens = torch.randint(-2, S + 3, (B,), generator=gen, dtype=torch.int32)
    new_lens[0] = S
    lens = torch.randint(-2, n + 3, (B,), generator=gen, dtype=torch.int32).cuda() if n else None
    tref.check("ragged prompt", kvx.attend_prompt, q, new_lens=new_lens.cuda(), lens=lens, **args)


PACKED = [[0, 5], [0, 0, 1, 1, 130, 500], [3, 90, 90, 300, 301, 650, 650], [0, 1100, 1101], [0] * 30 + [40] * 40 + [200] + [201] * 33]


@pytest.mark.parametrize("at", PACKED)
@pytest.mark.parametrize("N,D,n,dtype", [(4, 128, 0, BF16), (3, 64, 0, F16), (1, 128, 140, F16), (6, 64, 33, BF16)])
def test_packed_sequences(kvx, at, N, D, n, dtype):
    """Sequences one behind another, empty ones among them, tokens before the first and behind the last."""
    q, args = make(len(at) - 1, at[-1] + 9, N, 2, D, n=n, dtype=dtype, packed=True, seed=at[-1])
    lens = torch.arange(len(at) - 1, dtype=torch.int32, device="cuda") * 37 % (n + 1) if n else None
    tref.check("packed", kvx.attend_prompt, q, starts=ints(*at), lens=lens, **args)


def test_packed_without_starts_is_one_sequence(kvx):
    q, args = make(1, 77, 2, 3, 64, packed=True)
    tref.check("packed", kvx.attend_prompt, q, **args)


def test_starts_out_of_range_are_clamped(kvx):
    q, args = make(3, 60, 2, 2, 64, packed=True)
    tref.check("packed", kvx.attend_prompt, q, starts=ints(-4, 20, 41, 1 << 30), **args)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [1, 2, 5, 16, 31, 33, 63, 64])
@pytest.mark.parametrize("n", [0, 1, 300])
def test_trees(kvx, T, n, D, dtype):
    q, args = make(3, T, 3, 2, D, n=n, dtype=dtype, seed=T)
    tref.check("tree", kvx.attend_tree, q, parents=trees(3, T, T), **args)


@pytest.mark.parametrize("N", [1, 2, 4, 7, 8, 16, 40])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [128, 901])
def test_tree_head_groups(kvx, N, D, n):
    q, args = make(2, 13, N, 2, D, n=n, seed=N)
    tref.check("tree", kvx.attend_tree, q, parents=trees(2, 13, N), new_lens=ints(13, 6), lens=ints(n - 1, 57), **args)


@pytest.mark.parametrize("B,T,N,H,D,n,dtype", [
    (1, 16, 4, 1, 128, 40000, F16), (33, 8, 4, 8, 128, 700, BF16), (4, 64, 8, 2, 64, 6001, F16), (300, 3, 2, 4, 64, 90, F16),
    (7, 20, 5, 8, 128, 3000, BF16), (2, 64, 16, 1, 128, 5000, F16)])
def test_trees_cut_over_the_gpu(kvx, B, T, N, H, D, n, dtype):
    q, args = make(B, T, N, H, D, n=n, dtype=dtype, seed=n)
    tref.check("tree", kvx.attend_tree, q, parents=trees(B, T, n), **args)
    gen = torch.Generator().manual_seed(n)
    new_lens, lens = (torch.randint(0, x + 1, (B,), generator=gen, dtype=torch.int32).cuda() for x in (T, n))
    tref.check("ragged tree", kvx.attend_tree, q, parents=trees(B, T, n), new_lens=new_lens, lens=lens, **args)


def test_chain_is_causal(kvx):
    q, args = make(2, 40, 3, 2, 128, n=200)
    a = tref.check("chain", kvx.attend_tree, q, **args)
    b = tref.check("chain", kvx.attend_tree, q, parents=torch.arange(-1, 39, dtype=torch.int32, device="cuda"), **args)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_parents_that_are_not_before_their_token(kvx):
    """count as -1; so does every negative one. One tree for the whole batch."""
    q, args = make(2, 9, 4, 2, 64, n=20)
    tref.check("tree", kvx.attend_tree, q, parents=ints(0, 1, -5, 2, 9, 1 << 30, 3, -(1 << 31), 6), **args)


@pytest.mark.parametrize("D", [64, 128])
def test_layouts(kvx, D):
    """Keys as the cache takes them, values inside a fused projection, padded rows, heads and sequences that share rows."""
    B, S, N, H, n = 2, 150, 3, 2, 260
    G = N * H
    gen = torch.Generator(device="cuda").manual_seed(4)
    keys = normal(gen, B, 3, H, S, D)
    fused = normal(gen, B, S, G + 2 * H, D + 8)[..., :D]
    q, k_new, v_new = fused[:, :, :G], keys[:, 1].transpose(1, 2), fused[:, :, G + H:]
    rows = normal(gen, n, B, H + 1, D + 16)[..., :D]
    k, v = rows[:, :, :H].permute(1, 2, 0, 3), normal(gen, B, H, n, D)
    out = torch.full((B, G, S, D), 7.0, dtype=F16, device="cuda").transpose(1, 2)
    new_lens = ints(S - 1, S // 2)
    tref.check("layouts", kvx.attend_prompt, q, out=out, k_new=k_new, v_new=v_new, k=k, v=v, new_lens=new_lens)
    shared = [x[:, :, :1].expand(-1, -1, H, -1) for x in (k_new, v_new)]
    tref.check("one key head's", kvx.attend_prompt, q, k_new=shared[0], v_new=shared[1], k=k, v=v)
    tref.check("one sequence's rows", kvx.attend_prompt, q, k_new=k_new, v_new=v_new, k=k[:1].expand(B, -1, -1, -1), v=v[:1].expand(B, -1, -1, -1))
    tref.check("layouts of a tree", kvx.attend_tree, q[:, :50], k_new=k_new[:, :50], v_new=v_new[:, :50], k=k, v=v,
               parents=trees(B, 50))
    qkv = normal(gen, S, G + 2 * H, D)
    tref.check("packed layouts", kvx.attend_prompt, qkv[:, :G], k_new=qkv[:, G:G + H], v_new=qkv[:, G + H:], starts=ints(0, 60, S))


@pytest.mark.parametrize("scale", [0.5, 0.003, 30.0])
@pytest.mark.parametrize("S", [20, 300])
def test_scales(kvx, scale, S):
    q, args = make(2, S, 4, 2, 128, n=100, seed=9)
    tref.check("scale", kvx.attend_prompt, q, scale=scale, **args)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("n", [0, 40])
def test_thousands_of_sequences(kvx, packed, n):
    """Most of them empty, several for each thread that adds up the work."""
    B, N, H, D = 2500, 2, 2, 64
    gen = torch.Generator().manual_seed(1)
    count = torch.randint(0, 4, (B,), generator=gen) * (torch.rand(B, generator=gen) < 0.1)
    count[100:900] = 0
    count[-3:] = torch.tensor([0, 90, 0])
    at = torch.cat([torch.zeros(1, dtype=torch.long), count.cumsum(0)]).int()
    lens = torch.randint(0, n + 1, (B,), generator=gen, dtype=torch.int32).cuda() if n else None
    if packed:
        q, args = make(B, int(at[-1]) + 2, N, H, D, n=n, packed=True, seed=6)
        tref.check("packed", kvx.attend_prompt, q, starts=at.cuda(), lens=lens, **args)
    else:
        q, args = make(B, 90, N, H, D, n=n, seed=6)
        tref.check("batch", kvx.attend_prompt, q, new_lens=count.int().cuda(), lens=lens, **args)


@pytest.mark.parametrize("S,n", [(20, 0), (20, 4000), (300, 60), (2500, 0)])
def test_without_log_sums(kvx, S, n):
    q, args = make(1, S, 3, 2, 128, n=n, seed=S)
    want, _ = tref.check("prompt", kvx.attend_prompt, q, **args)
    out = torch.empty_like(q)
    kvx.attend_prompt(q, out, **args)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
