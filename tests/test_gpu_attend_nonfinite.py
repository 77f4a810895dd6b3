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


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("path", ["clusters", "ranges", "pair", "tiles"])
def test_a_value_that_counts_and_is_not_finite(kvx, path, value, D):
    """It shows: its column is not finite in the sequences that have the row, whichever kernel runs. Everything else,
    the log sums among it, is as it was."""
    if path in ("pair", "tiles"):
        B, N, H = 64, 2 if path == "pair" else 5, 4
        q, rows = make(B, N, H, D, P=2000 * 128 // D, seed=3)
    else:
        B, N, H = (3, 2, 2) if path == "clusters" else (60, 2, 8)
        q, rows = make(B, N, H, D, n=50 if path == "clusters" else 600, seed=3)
    assert prefix_kernel(kvx, q, **rows) == (path in ("pair", "tiles"))
    want, lse = ref.check_attend(kvx, q, **rows)
    rows["v" if "v" in rows else "prefix_v"][..., 0, 17, 9] = float(value)      # of the first key head
    if "v" in rows:
        rows["v"][1:, 0, 17, 9] = 1.0                                           # of the first sequence
    out, again = torch.empty_like(q), torch.empty_like(lse)
    kvx.attend(q, out, lse=again, **rows)
    torch.cuda.synchronize()
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[:1 if "v" in rows else B, :N, 9] = True
    assert not torch.isfinite(out[hit]).any()
    if "v" in rows:
        hit[:, :N, 9] = True
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(again, lse)


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


@pytest.mark.parametrize("B,N,H,D,P", [(64, 2, 4, 128, 2000), (64, 5, 4, 64, 2000), (3, 2, 2, 64, 100)])
def test_a_logit_of_infinity(kvx, B, N, H, D, P):
    """+inf: NaN in the sequences that have the row. Nothing but -inf: as if there were no rows."""
    q, rows = make(B, N, H, D, P=P, seed=6)
    lens = torch.tensor([P, 17], dtype=torch.int32, device="cuda").repeat(B)[:B]
    want, wlse = ref.check_attend(kvx, q, prefix_lens=lens, **rows)
    q[:, :N, 0] = 1.0                                                  # the first key head's queries
    want[:, :N], wlse[:, :N] = [x[:, :N] for x in ref.check_attend(kvx, q, prefix_lens=lens, **rows)]
    rows["prefix_k"][0, 40, 0] = float("inf")
    out, lse = torch.empty_like(q), torch.empty_like(wlse)
    kvx.attend(q, out, lse=lse, prefix_lens=lens, **rows)
    torch.cuda.synchronize()
    hit = torch.zeros(B, N * H, dtype=torch.bool, device="cuda")
    hit[::2, :N] = True
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], wlse[~hit])
    rows["prefix_k"][0, :, 0] = -float("inf")
    kvx.attend(q, out, lse=lse, prefix_lens=lens, **rows)
    torch.cuda.synchronize()
    assert (out[:, :N] == 0).all() and (lse[:, :N] == -float("inf")).all()
    assert torch.equal(out[:, N:], want[:, N:]) and torch.equal(lse[:, N:], wlse[:, N:])


# Few own rows beside a large prefix (joined in the clusters' kernel), and many (in the ranges' join).
BESIDE = [(32, 4, 8, 128, 1100, 0), (40, 3, 8, 128, 900, 5), (300, 2, 2, 128, 901, 0), (32, 4, 8, 128, 1100, 400),
          (300, 2, 2, 128, 901, 200)]


@pytest.mark.parametrize("B,N,H,D,P,n", BESIDE)
def test_shared_keys_of_nan_beside_finite_own_rows(kvx, B, N, H, D, P, n):
    """A head whose shared keys are all NaN answers with NaN in every sequence that shares some; the others are untouched."""
    q, rows = make(B, N, H, D, P=P, n=n, new=True, seed=P + n)
    lens = torch.full((B,), P, dtype=torch.int32, device="cuda")
    lens[5:9] = 0
    assert prefix_kernel(kvx, q, prefix_lens=lens, **rows)
    want, wlse = ref.check_attend(kvx, q, prefix_lens=lens, **rows)
    rows["prefix_k"][1] = float("nan")
    out, lse = torch.empty_like(q), torch.empty_like(wlse)
    kvx.attend(q, out, lse=lse, prefix_lens=lens, **rows)
    torch.cuda.synchronize()
    hit = torch.zeros(B, N * H, dtype=torch.bool, device="cuda")
    hit[lens > 0, N:2 * N] = True
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], wlse[~hit])


@pytest.mark.parametrize("B,N,H,D,P,n", BESIDE + [(4000, 4, 8, 64, 130, 0)])
def test_a_wait_that_runs_out_beside_own_rows(kvx, B, N, H, D, P, n):
    """NaN wherever the lost part belongs, however far the own rows' logits are above it; right results next time. (The
    library's test hook leaves one copy unissued: the bounded wait runs out, nothing hangs.)"""
    q, rows = make(B, N, H, D, P=P, n=n, new=True, seed=P + n)
    rows["k_new"] = (q[:, ::N] * 40).contiguous()            # own logits far above the shared rows'
    assert prefix_kernel(kvx, q, **rows)
    want, wlse = torch.empty_like(q), torch.empty(B, N * H, device="cuda")
    kvx.attend(q, want, lse=wlse, **rows)
    torch.cuda.synchronize()
    assert torch.isfinite(want).all() and torch.isfinite(wlse).all()
    out, lse = torch.zeros_like(q), torch.zeros_like(wlse)
    assert kvx.lib().kvevict_test_stall_next_step(None) == kvx.OK
    kvx.attend(q, out, lse=lse, **rows)
    torch.cuda.synchronize()
    # the first CTA's first block of query rows: the first key head's, 128 of them, or 256 where there are more
    first = min(B, 128 // N if B * N <= 128 else 256 // N)
    assert torch.isnan(out[:first, :N]).all() and torch.isnan(lse[:first, :N]).all()
    # lost or right, nothing in between
    lost = torch.isnan(lse)
    assert torch.equal(torch.isnan(out), lost[..., None].expand_as(out))
    assert torch.equal(out[~lost], want[~lost]) and torch.equal(lse[~lost], wlse[~lost])
    kvx.attend(q, out, lse=lse, **rows)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wlse)


def test_a_wait_that_runs_out_on_a_handle(kvx):
    """The handle reports it, too, and attention that waits for nothing goes on."""
    B, N, H, D, P = 32, 4, 8, 128, 1100
    q, rows = make(B, N, H, D, P=P, new=True, seed=1)
    h = kvx.KVEvict(batch=B, n_layers=1, n_kv_heads=H, head_dim=D, layer_budgets=[8], n_sink=1, max_prefill=4, with_values=True)
    want, out = torch.empty_like(q), torch.zeros_like(q)
    h.attend(0, q, want, **rows)
    torch.cuda.synchronize()
    h.check()
    assert kvx.lib().kvevict_test_stall_next_step(None) == kvx.OK
    h.attend(0, q, out, **rows)
    torch.cuda.synchronize()
    assert torch.isnan(out[:, :N]).all()
    with pytest.raises(kvx.KVEvictError) as e:
        h.check()
    assert e.value.code == kvx.ERR_DEVICE_CHECK
    h.attend(0, q, out, **rows)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
