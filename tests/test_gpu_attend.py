"""Attention over own rows, a shared prefix and the token's own key against its 64-bit form."""
import math

import pytest

torch = pytest.importorskip("torch")
import attention_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def kvx():
    import kv_cache_attention_02_gb300 as k
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    k.lib()
    return k


def _make(B, N, H, D, n=0, P=0, new=False, dtype=F16, seed=0, spread=1.5):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def r(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)
    rows = {}
    if n:
        rows.update(k=r(B, H, n, D), v=r(B, H, n, D))
    if new:
        rows.update(k_new=r(B, H, D), v_new=r(B, H, D))
    if P:
        rows.update(prefix_k=r(H, P, D), prefix_v=r(H, P, D))
    return r(B, N * H, D, scale=spread), rows


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 200, 1025])
def test_lengths(kvx, n, D, dtype):
    q, rows = _make(2, 3, 2, D, n=n, new=n % 2 == 0, dtype=dtype, seed=n)
    ref.check_attend(kvx, q, **rows)


@pytest.mark.parametrize("N", [1, 2, 7, 8, 9, 16, 17, 32, 40])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [0, 70])
def test_head_groups(kvx, N, D, P):
    q, rows = _make(2, N, 2, D, n=45, P=P, new=True, seed=N)
    ref.check_attend(kvx, q, **rows)


@pytest.mark.parametrize("B,H,n", [(1, 1, 5000), (1, 8, 3000), (40, 8, 130), (3, 1, 1), (300, 4, 33), (1, 1, 40000)])
def test_splits(kvx, B, H, n):
    q, rows = _make(B, 4, H, 128, n=n, seed=n)
    ref.check_attend(kvx, q, **rows)


@pytest.mark.parametrize("B,N,H,D,n,dtype", [(40, 4, 8, 128, 401, F16), (9, 3, 4, 128, 3001, BF16), (3, 12, 2, 128, 17000, F16),
                                            (1, 40, 1, 64, 60001, BF16), (600, 1, 4, 64, 90, F16), (1500, 2, 4, 128, 3, F16),
                                            (5, 16, 8, 64, 5000, F16)])
@pytest.mark.parametrize("new", [False, True])
def test_many_tiles(kvx, B, N, H, D, n, dtype, new):
    """Work cut into ranges that begin and end inside a unit; even lengths, then ragged ones with empty sequences."""
    q, rows = _make(B, N, H, D, n=n, new=new, dtype=dtype, seed=n)
    ref.check_attend(kvx, q, **rows)
    lens = torch.randint(0, n + 1, (B,), dtype=torch.int32, device="cuda")
    lens[B // 2:B // 2 + 40] = 0
    lens[0] = n
    ref.check_attend(kvx, q, lens=lens, **rows)


@pytest.mark.parametrize("B,N,H,D,n", [(40, 4, 8, 128, 401), (2, 40, 2, 128, 11000), (1500, 2, 4, 64, 90)])
@pytest.mark.parametrize("top", [0, 1, 40, 300])
def test_room_for_many_tiles_but_few_rows(kvx, B, N, H, D, n, top):
    """Room that would be cut into a range per CTA, lengths that make fewer tiles than there are CTAs."""
    q, rows = _make(B, N, H, D, n=n, new=top == 40, seed=n)
    lens = torch.randint(0, top + 1, (B,), dtype=torch.int32, device="cuda").clamp(max=n)
    lens[3:] = lens[3:] // 40
    ref.check_attend(kvx, q, lens=lens, **rows)


def test_many_short_sequences(kvx):
    """Thousands of sequences, most of them empty, over ranges that hold many each (checked where there are rows)."""
    B, H, n = 6000, 8, 40
    q, rows = _make(B, 2, H, 128, n=n, seed=16)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    some = torch.tensor([0, 1, 2, 700, 3001, 3002, 5998, 5999], device="cuda")
    lens[some] = torch.tensor([1, n, 0, 33, n, 17, 16, n], dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(q, float("nan")), torch.empty(B, 2 * H, device="cuda")
    kvx.attend(q, out, lens=lens, lse=lse, **rows)
    torch.cuda.synchronize()
    want = ref.attend_batch(q[some], k=rows["k"][some], v=rows["v"][some], lens=lens[some])
    ref.check("out", out[some], want[0], want[2])
    ref.check("lse", lse[some], want[1], want[3])
    rest = torch.ones(B, dtype=torch.bool, device="cuda")
    rest[some] = False
    assert (out[rest] == 0).all() and (lse[rest] == -math.inf).all()


@pytest.mark.parametrize("B,N,H,D,n,P", [(40, 4, 8, 128, 401, 700), (200, 3, 4, 64, 400, 300), (30, 20, 8, 128, 350, 1000),
                                        (1, 4, 2, 128, 30000, 20000)])
def test_many_tiles_with_prefix(kvx, B, N, H, D, n, P):
    q, rows = _make(B, N, H, D, n=n, P=P, new=True, seed=P)
    ref.check_attend(kvx, q, **rows)
    lens = torch.randint(0, n + 1, (B,), dtype=torch.int32, device="cuda")
    plens = torch.randint(0, P + 1, (B,), dtype=torch.int32, device="cuda")
    lens[B // 3:B // 2], plens[B // 4:B // 2] = 0, 0
    ref.check_attend(kvx, q, lens=lens, prefix_lens=plens, **rows)


def test_prefix_strides_of_all_kinds(kvx):
    """Padded rows, heads inside rows, and a prefix that is the same for all heads (which TMA cannot describe)."""
    q, rows = _make(60, 4, 3, 128, P=900, seed=14)
    k, v = rows["prefix_k"], rows["prefix_v"]
    padded = torch.zeros(3, 909, 136, dtype=F16, device="cuda")
    padded[:, :900, :128] = k
    inside = torch.zeros(900, 3, 136, dtype=F16, device="cuda")
    inside[:, :, :128] = v.transpose(0, 1)
    ref.check_attend(kvx, q, prefix_k=padded[:, :900, :128], prefix_v=inside[:, :, :128].transpose(0, 1))
    same = [x[:1].expand(3, -1, -1) for x in (k, v)]
    ref.check_attend(kvx, q, prefix_k=same[0], prefix_v=same[1])


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,N,P", [(1, 1, 1), (1, 4, 127), (5, 3, 128), (2, 4, 129), (32, 4, 1000), (40, 4, 257), (7, 40, 640),
                                   (130, 2, 384), (64, 5, 2100), (3, 2, 9000), (700, 4, 300)])
def test_prefix_alone(kvx, B, N, P, D, dtype):
    q, rows = _make(B, N, 2, D, P=P, dtype=dtype, seed=P)
    ref.check_attend(kvx, q, **rows)


# Enough rows for the tensor-core kernel, which reads them once: up to 128 query rows a key head (both of its streams on
# the same rows) and more (a row block each), blocks cut over CTAs and whole, tiles that end inside, odd head groups.
SHARED = [(128, 1, 8, 128, 130), (100, 1, 4, 64, 1300), (32, 4, 8, 128, 1100), (2, 40, 2, 128, 11000), (3, 12, 2, 64, 45000),
          (33, 4, 8, 128, 500), (70, 8, 2, 128, 1000), (130, 2, 4, 64, 1000), (300, 5, 2, 64, 901), (512, 4, 8, 128, 129),
          (700, 3, 2, 128, 257), (17, 40, 3, 64, 5000), (43, 3, 8, 128, 8191)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("B,N,H,D,P", SHARED)
def test_large_prefix(kvx, B, N, H, D, P, dtype):
    q, rows = _make(B, N, H, D, P=P, dtype=dtype, seed=P)
    ref.check_attend(kvx, q, **rows)


@pytest.mark.parametrize("B,N,H,D,P", SHARED)
@pytest.mark.parametrize("n", [0, 5, 90])
def test_large_prefix_with_own_rows(kvx, B, N, H, D, P, n):
    """Beside few own rows (or the token's own alone) and beside more; then unequal lengths of both, none among them, and
    shared rows that no sequence has left as NaN."""
    dtype = BF16 if P % 2 else F16
    q, rows = _make(B, N, H, D, n=n, P=P, new=n != 5, dtype=dtype, seed=P + n)
    ref.check_attend(kvx, q, **rows)
    gen = torch.Generator().manual_seed(P)
    plens = torch.randint(0, P - 60, (B,), dtype=torch.int32, generator=gen).cuda()
    plens[B // 3:B // 2] = 0
    extra = {"prefix_lens": plens}
    top = int(plens.max())
    rows["prefix_k"][:, top:], rows["prefix_v"][:, top:] = float("nan"), float("nan")
    if n:
        extra["lens"] = torch.randint(0, n + 1, (B,), dtype=torch.int32, generator=gen).cuda()
        extra["lens"][B // 4:B // 2 + 1] = 0
    ref.check_attend(kvx, q, **extra, **rows)


@pytest.mark.parametrize("B,N,H,D,P", SHARED[::3])
def test_large_prefix_alone_with_unequal_lengths(kvx, B, N, H, D, P):
    q, rows = _make(B, N, H, D, P=P, seed=P + 1)
    plens = torch.randint(0, P + 1, (B,), dtype=torch.int32, device="cuda")
    plens[0], plens[B // 2:] = P, 0
    out, lse = ref.check_attend(kvx, q, prefix_lens=plens, **rows)
    assert (out[B // 2:] == 0).all() and (lse[B // 2:] == -math.inf).all()
    out, lse = ref.check_attend(kvx, q, prefix_lens=torch.zeros_like(plens), **rows)
    assert (out == 0).all()


@pytest.mark.parametrize("scale", [1e-3, 0.5, 3.0])
@pytest.mark.parametrize("B,N,H,D,P", [(32, 4, 8, 128, 1100), (300, 5, 2, 64, 901)])
def test_large_prefix_and_large_logits(kvx, B, N, H, D, P, scale):
    q, rows = _make(B, N, H, D, P=P, seed=5)
    rows["prefix_k"] *= torch.linspace(0.1, 4, P, device="cuda").to(F16)[:, None]
    ref.check_attend(kvx, q, scale=scale, **rows)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("B,N,H,D,n,P,new", [(4, 3, 8, 128, 64, 333, True), (33, 4, 2, 128, 100, 2000, True),
                                            (33, 4, 2, 64, 100, 2000, False), (70, 8, 1, 128, 17, 1500, True),
                                            (16, 12, 2, 64, 0, 900, True), (300, 2, 1, 128, 9, 700, True)])
def test_prefix_with_own_rows(kvx, B, N, H, D, n, P, new, dtype):
    q, rows = _make(B, N, H, D, n=n, P=P, new=new, dtype=dtype, seed=P + n)
    ref.check_attend(kvx, q, **rows)
    lens = torch.randint(0, n + 1, (B,), dtype=torch.int32, device="cuda") if n else None
    plens = torch.randint(0, P + 1, (B,), dtype=torch.int32, device="cuda")
    plens[0], plens[-1] = 0, P
    ref.check_attend(kvx, q, prefix_lens=plens, **({"lens": lens} if n else {}), **rows)


@pytest.mark.parametrize("B,P", [(6, 0), (6, 90), (48, 700), (200, 513)])
@pytest.mark.parametrize("new", [False, True])
def test_empty_ragged_and_poisoned_rows(kvx, B, P, new):
    """Lengths of zero, one and out of range; rows past a length hold NaN and infinities."""
    n = 50
    q, rows = _make(B, 4, 2, 128, n=n, P=P, new=new, seed=P)
    lens = torch.tensor([0, 1, n, n + 9, -3, 17] * (B // 6 + 1), dtype=torch.int32, device="cuda")[:B]
    extra = {}
    if P:
        extra["prefix_lens"] = torch.tensor([0, P, 1, -1, 0, P // 2] * (B // 6 + 1), dtype=torch.int32, device="cuda")[:B]
    for b in range(B):
        at = min(max(int(lens[b]), 0), n)
        rows["k"][b, :, at:], rows["v"][b, :, at:] = float("nan"), float("inf")
    out, lse = ref.check_attend(kvx, q, lens=lens, **extra, **rows)
    if not new:
        assert (out[0] == 0).all() and (lse[0] == -math.inf).all()


def test_prefix_rows_past_every_length_are_not_used(kvx):
    q, rows = _make(140, 4, 2, 128, P=600, seed=8)
    plens = torch.full((140,), 301, dtype=torch.int32, device="cuda")
    plens[3] = 0
    rows["prefix_k"][:, 301:], rows["prefix_v"][:, 301:] = float("nan"), float("nan")
    ref.check_attend(kvx, q, prefix_lens=plens, **rows)


@pytest.mark.parametrize("B,N,H", [(130, 4, 2), (30, 4, 8), (300, 3, 2)])
def test_strides_of_a_large_prefix(kvx, B, N, H):
    """Queries inside a fused projection, outputs inside a larger buffer whose other rows stay; lengths out of range."""
    D, P = 128, 1300
    q, rows = _make(B, N, H, D, P=P, seed=21)
    qkv = torch.cat([q, q * 3, q], 1)
    big = torch.full((B + 1, 2 * N * H, D), 3.0, dtype=F16, device="cuda")
    ref.check_attend(kvx, qkv[:, N * H:2 * N * H], out=big[:B, N * H:], **rows)
    assert (big[:, :N * H] == 3).all() and (big[B] == 3).all()
    plens = torch.full((B,), P + 7, dtype=torch.int32, device="cuda")
    plens[::3] = -5
    ref.check_attend(kvx, qkv[:, N * H:2 * N * H], out=big[:B, N * H:], prefix_lens=plens, **rows)
    assert (big[:, :N * H] == 3).all() and (big[B] == 3).all()


@pytest.mark.parametrize("P", [0, 300, 2500])
@pytest.mark.parametrize("B", [3, 50])
def test_strides(kvx, B, P):
    """Rows between sequences ([B, n, H, D]), queries inside a fused projection, outputs inside a larger buffer."""
    H, N, D, n = 2, 4, 128, 70
    q, rows = _make(B, N, H, D, n=n, P=P, new=True, seed=11)
    qkv = torch.cat([q, q, q], 1)
    for name in ("k", "v"):
        rows[name] = rows[name].transpose(1, 2).contiguous().transpose(1, 2)
    if P:
        for name in ("prefix_k", "prefix_v"):
            rows[name] = torch.stack([rows[name].transpose(0, 1)] * 2, 1)[:, 1].transpose(0, 1)
    big = torch.full((B + 1, 2 * N * H, D), 3.0, dtype=F16, device="cuda")
    ref.check_attend(kvx, qkv[:, N * H:2 * N * H], out=big[:B, N * H:], **rows)
    assert (big[:, :N * H] == 3).all() and (big[B] == 3).all()


@pytest.mark.parametrize("which", ["k", "v", "k_new", "v_new", "prefix_k", "prefix_v", "row"])
@pytest.mark.parametrize("B,n", [(3, 70), (60, 400)])
def test_buffers_at_16_bytes(kvx, B, n, which):
    """Buffers and strides that are multiples of 16 bytes but not of 32."""
    q, rows = _make(B, 4, 2, 128, n=n, P=100, new=True, seed=3)
    for name in ([which] if which != "row" else ["k", "v"]):
        x = rows[name]
        pad = torch.zeros(*x.shape[:-1], 136, dtype=F16, device="cuda")
        if which == "row":
            pad[..., :128] = x
            rows[name] = pad[..., :128]
        else:
            flat = torch.zeros(x.numel() + 8, dtype=F16, device="cuda")
            flat[8:] = x.reshape(-1)
            rows[name] = flat[8:].view(x.shape)
            assert rows[name].data_ptr() % 32 == 16
    ref.check_attend(kvx, q, **rows)


@pytest.mark.parametrize("scale", [1e-3, 0.5, 3.0])
@pytest.mark.parametrize("P", [0, 260])
@pytest.mark.parametrize("B", [2, 40])
def test_scales_and_large_logits(kvx, B, P, scale):
    """From flat weights to one key that takes everything, the running maximum moving often and far."""
    q, rows = _make(B, 4, 2, 64, n=150, P=P, seed=5)
    rows["k"] *= torch.linspace(0.1, 4, 150, device="cuda").to(F16)[:, None]
    if P:
        rows["prefix_k"] *= torch.linspace(0.1, 4, P, device="cuda").to(F16)[:, None]
    ref.check_attend(kvx, q, scale=scale, **rows)


@pytest.mark.parametrize("B", [2, 40])
def test_infinite_and_nan_rows_that_count(kvx, B):
    """A NaN in a row that counts shows in its sequence alone; a key of -inf logits takes no weight."""
    q, rows = _make(B, 2, 2, 64, n=40, P=200, seed=6)
    want, wlse = ref.check_attend(kvx, q, **rows)
    rows["v"][1, 0, 7] = float("nan")
    out, lse = torch.empty_like(q), torch.empty_like(wlse)
    kvx.attend(q, out, lse=lse, **rows)
    torch.cuda.synchronize()
    assert torch.isnan(out[1, :2]).all() and torch.equal(out[1, 2:], want[1, 2:]) and torch.equal(lse, wlse)
    assert torch.equal(out[0], want[0]) and torch.equal(out[2:], want[2:])
    rows["k"][1, 0, 7] = float("nan")
    kvx.attend(q, out, lse=lse, **rows)
    torch.cuda.synchronize()
    assert torch.isnan(out[1, :2]).all() and torch.isnan(lse[1, :2]).all() and torch.equal(lse[0], wlse[0])


def test_offsets_past_32_bits(kvx):
    """Strides whose products pass 2^31 elements: the second sequence and the last rows of a long buffer."""
    H, N, D, n = 2, 4, 128, 40
    far = 2 ** 31 + 1024                       # elements between sequences
    if torch.cuda.mem_get_info()[0] < 24 * 2 ** 30:
        pytest.skip("needs 24 GB")
    base = [torch.zeros(far + 2 ** 20, dtype=F16, device="cuda") for _ in range(2)]
    q, rows = _make(2, N, H, D, n=n, seed=9)
    for name, x in zip(("k", "v"), base):
        view = x.as_strided((2, H, n, D), (far, n * D, D, 1))
        view.copy_(rows[name])
        rows[name] = view
    ref.check_attend(kvx, q, **rows)
    step = 2 ** 25 + 128                       # elements between rows: row 63 is past 2^31
    q, rows = _make(2500, N, 1, D, P=64, seed=10)
    for name, x in zip(("prefix_k", "prefix_v"), base):
        view = x.as_strided((1, 64, D), (0, step, 1))
        view.copy_(rows[name])
        rows[name] = view
    ref.check_attend(kvx, q, **rows)


@pytest.mark.parametrize("B,n,P", [(2, 300, 0), (2, 30, 100), (40, 30, 3000), (150, 0, 1000), (40, 2100, 0), (150, 900, 900)])
def test_repeat_streams_and_graphs(kvx, B, n, P):
    """The same bits call after call, on another stream, and from two captured graphs that replay together."""
    q, rows = _make(B, 4, 2, 128, n=n, P=P, seed=12)
    want, wlse = ref.check_attend(kvx, q, **rows)
    side = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(q) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, o in zip(side, outs):
            o.zero_()
        torch.cuda.synchronize()
        for s, o in zip(side, outs):
            kvx.attend(q, o, stream=s, **rows)
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, o in zip(graphs, outs):
        with torch.cuda.graph(g):
            kvx.attend(q, o, **rows)
    torch.cuda.synchronize()
    for _ in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for s, g in zip(side, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
    q.neg_()
    other = torch.empty_like(q)
    kvx.attend(q, other, **rows)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], other) and not torch.equal(other, want)


@pytest.mark.parametrize("B,P", [(3, 500), (120, 900)])
def test_parts_join_by_lse(kvx, B, P):
    """Prefix and own rows in two calls, joined by their log sums, are the one call."""
    q, rows = _make(B, 4, 2, 128, n=80, P=P, seed=13)
    out, lse = ref.check_attend(kvx, q, **rows)
    a, la = ref.check_attend(kvx, q, k=rows["k"], v=rows["v"])
    b, lb = ref.check_attend(kvx, q, prefix_k=rows["prefix_k"], prefix_v=rows["prefix_v"])
    total = torch.logaddexp(la, lb)
    joined = a * (la - total).exp()[..., None] + b * (lb - total).exp()[..., None]
    # three roundings to fp16 (both parts and the whole) and the weights' half steps in the prefix part
    assert (joined - out).abs().max() <= 4 * 2.0 ** -11 * max(a.abs().max(), b.abs().max(), 1.0)
    torch.testing.assert_close(total, lse, rtol=1e-6, atol=1e-5)


@pytest.mark.parametrize("n,P", [(2100, 0), (10, 3000)])
def test_workspace_of_the_c_call(kvx, n, P):
    """Too little workspace launches nothing; the size asked for is enough, and nothing past it is written."""
    import ctypes
    B, G, H, D = 40, 8, 2, 128
    q, rows = _make(B, G // H, H, D, n=n, P=P, seed=17)
    want, wlse = ref.check_attend(kvx, q, **rows)
    out, lse = torch.full_like(q, 5.0), torch.empty_like(wlse)
    args, stream = kvx._attention(q, out, rows["k"], rows["v"], None, None, None, rows.get("prefix_k"), rows.get("prefix_v"),
                                  None, lse, None, None, None)
    need = ctypes.c_size_t(0)
    assert kvx.lib().kvevict_attend_workspace(args, 0, ctypes.addressof(need)) == kvx.OK and need.value > 0
    space = torch.full((need.value + 4096,), 7, dtype=torch.uint8, device="cuda")

    def call(at, size):
        filled = bytearray(args)
        kvx.struct.pack_into("=Q", filled, kvx._WORKSPACE_AT, at)
        kvx.struct.pack_into("=Q", filled, kvx._WORKSPACE_BYTES_AT, size)
        rc = kvx.lib().kvevict_attend(bytes(filled), stream)
        torch.cuda.synchronize()
        return rc
    for at, size in ((0, 0), (0, need.value), (space.data_ptr(), need.value - 1), (space.data_ptr() + 8, need.value)):
        assert call(at, size) == kvx.ERR_WORKSPACE and "workspace" in kvx.last_error()
    assert (out == 5).all()
    assert call(space.data_ptr(), need.value) == kvx.OK
    assert torch.equal(out, want) and torch.equal(lse, wlse) and (space[need.value:] == 7).all()


@pytest.mark.parametrize("n,P", [(300, 0), (2100, 0), (10, 3000)])
def test_other_stream_than_the_current_one(kvx, n, P):
    """The workspace belongs to the call's stream: by handle, by object, and the default stream from a side stream."""
    q, rows = _make(40, 4, 2, 128, n=n, P=P, seed=18)
    want, _ = ref.check_attend(kvx, q, **rows)
    side = torch.cuda.Stream()
    for given, current in ((side, None), (side.cuda_stream, None), (0, side), (torch.cuda.default_stream(), side)):
        out = torch.zeros_like(q)
        torch.cuda.synchronize()
        with torch.cuda.stream(current):
            for _ in range(3):
                kvx.attend(q, out, stream=given, **rows)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_bounded_wait_leaves_nan(kvx):
    """A wait that runs out cannot reach the return code: NaN in every output instead, and the next call is unaffected.
    The library's test hook leaves one copy unissued; nothing faults or hangs."""
    import time
    q, rows = _make(250, 1, 1, 128, P=600, seed=15)     # one block of rows: all of it depends on the first tile
    want, wlse = ref.check_attend(kvx, q, **rows)
    out, lse = torch.zeros_like(q), torch.zeros_like(wlse)
    assert kvx.lib().kvevict_test_stall_next_step(None) == kvx.OK
    t0 = time.time()
    kvx.attend(q, out, lse=lse, **rows)
    torch.cuda.synchronize()
    assert 0.5 < time.time() - t0 < 10.0
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    kvx.attend(q, out, lse=lse, **rows)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wlse)
