"""Query/key norm with rotation against its 64-bit form."""
import pytest

torch = pytest.importorskip("torch")
import attention_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def kvx():
    import kv_cache_attention_02_gb300 as k
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    k.lib()
    return k


def _inputs(B, S, G, H, D, dtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    qkv = (torch.randn(B, S, G + 2 * H, D, generator=gen, device="cuda") * 3).to(dtype)
    w = [(1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(dtype) for _ in range(2)]
    return qkv[:, :, :G], qkv[:, :, G:G + H], w


def _check(kvx, q, k, qw, kw, q_out, k_out, theta=1e4, positions=None, pos0=0):
    keep_q, keep_k = q.clone(), k.clone()
    kvx.qk_norm_rope(q, k, q_out, k_out, rope_theta=theta, q_weight=qw, k_weight=kw, eps=EPS, positions=positions, pos0=pos0)
    torch.cuda.synchronize()
    B, S = q.shape[:2]
    p = positions if positions is not None else (torch.arange(S, device="cuda") + pos0).expand(B, S)
    for name, x, w, o in (("q", keep_q, qw, q_out), ("k", keep_k, kw, k_out)):
        y, size = ref.qk(x, w, p, theta, EPS)
        ref.check(name, o, y, ref.qk_bound(y, size, o.dtype))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("out", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,S,G,H", [(1, 1, 1, 1), (1, 1, 4, 4), (3, 1, 24, 8), (2, 37, 5, 1), (1, 300, 7, 3), (2, 5000, 3, 2)])
def test_against_64_bits(kvx, dtype, out, D, B, S, G, H):
    q, k, (qw, kw) = _inputs(B, S, G, H, D, dtype)
    q_out = torch.full((B, S, G, D), float("nan"), dtype=out, device="cuda")
    k_out = torch.full((B, H, S, D), float("nan"), dtype=out, device="cuda").transpose(1, 2)
    _check(kvx, q, k, qw, kw, q_out, k_out, theta=500000.0, pos0=17)


@pytest.mark.parametrize("pos0", [0, -1000, 131071, 10 ** 6, 2 ** 31 - 5])
def test_far_positions(kvx, pos0):
    q, k, (qw, kw) = _inputs(1, 4, 4, 2, 128, torch.float32, seed=2)
    outs = [torch.empty_like(x, dtype=torch.float16) for x in (q, k)]
    _check(kvx, q, k, qw, kw, *outs, pos0=pos0)


@pytest.mark.parametrize("S", [1, 700])
def test_positions_and_missing_weights(kvx, S):
    q, k, (qw, kw) = _inputs(2, S, 6, 2, 64, torch.bfloat16, seed=3)
    pos = torch.randint(-50, 200000, (2, S), device="cuda", dtype=torch.int32)
    for w in ((qw, kw), (None, kw), (qw, None), (None, None)):
        outs = [torch.empty(x.shape, dtype=torch.bfloat16, device="cuda") for x in (q, k)]
        _check(kvx, q / 4, k / 4, *w, *outs, positions=pos)


def test_zero_and_large_rows(kvx):
    """A row of zeros stays zero (eps); a row of the type's largest values keeps its norm in fp32's range."""
    q = torch.zeros(1, 3, 2, 64, dtype=torch.bfloat16, device="cuda")
    q[0, 1] = 1e18                         # squares to 1e36, 64 of them: under fp32's largest
    q[0, 2] = 1e-30
    outs = [torch.empty(q.shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    w = torch.ones(64, device="cuda")
    _check(kvx, q, q.clone(), w, w, *outs)
    assert torch.equal(outs[0][0, 0], torch.zeros_like(outs[0][0, 0]))


def test_one_side_alone_in_place_and_neighbours(kvx):
    q, k, (qw, kw) = _inputs(2, 9, 4, 2, 128, torch.float16, seed=4)
    both = [torch.empty(x.shape, dtype=torch.float16, device="cuda") for x in (q, k)]
    kvx.qk_norm_rope(q, k, *both, rope_theta=1e4, q_weight=qw, k_weight=kw)
    alone = [torch.empty_like(x) for x in both]
    kvx.qk_norm_rope(q, None, alone[0], None, rope_theta=1e4, q_weight=qw)
    kvx.qk_norm_rope(None, k, None, alone[1], rope_theta=1e4, k_weight=kw)
    # queries and keys inside the fused projection, its values left as they were
    qkv = torch.cat([q, k, torch.full_like(k, 5.0)], 2)
    kvx.qk_norm_rope(qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, :4], qkv[:, :, 4:6], rope_theta=1e4, q_weight=qw, k_weight=kw)
    for i, x in enumerate((qkv[:, :, :4], qkv[:, :, 4:6])):
        assert torch.equal(alone[i], both[i]) and torch.equal(x, both[i])
    assert (qkv[:, :, 6:] == 5).all()
    # one layer of a [B, L, H, D] batch of new keys; the others untouched
    k_new = torch.full((2, 3, 2, 128), 9.0, dtype=torch.float16, device="cuda")
    kvx.qk_norm_rope(None, k[:, 4:5], None, k_new[:, 1, None], rope_theta=1e4, k_weight=kw, pos0=4)
    assert torch.equal(k_new[:, 1], both[1][:, 4]) and (k_new[:, ::2] == 9).all()


def test_streams_and_graph(kvx):
    q, k, (qw, kw) = _inputs(2, 33, 4, 2, 128, torch.bfloat16, seed=5)
    want = [torch.empty(x.shape, dtype=torch.float16, device="cuda") for x in (q, k)]
    got = [torch.empty_like(x) for x in want]

    def call(outs, stream=None):
        kvx.qk_norm_rope(q, k, *outs, rope_theta=1e4, q_weight=qw, k_weight=kw, stream=stream)
    call(want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    call(got, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(got)
    q.mul_(-1)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], -want[0]) and torch.equal(got[1], want[1])
