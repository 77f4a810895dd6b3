"""The operators together, as a decoding model uses them: norm and rotation, attention over the cache and a shared
prefix, insertion with eviction."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import attention_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu
THETA, EPS = 500000.0, 1e-6


@pytest.fixture(scope="module")
def kvx():
    import kv_cache_attention_02_gb300 as k
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    k.lib()
    return k


def _rows(h, b, l, hh):
    """One row's keys and values as the cache holds them, as fp16 tensors."""
    keys = h.read_state(b, l, hh)[0].view(np.float16)
    return [torch.from_numpy(x.copy()).cuda() for x in (keys, h.read_values(b, l, hh).view(np.float16))]


@pytest.mark.parametrize("D,N,prefix", [(128, 3, 0), (64, 4, 37), (128, 9, 300)])
def test_decode_loop(kvx, D, N, prefix):
    B, L, H, S, T, budget = 2, 3, 2, 30, 40, 33
    G = N * H
    kw = dict(batch=B, n_layers=L, n_kv_heads=H, head_dim=D, layer_budgets=[budget, 24, 16], n_sink=2, tau_init=1.0,
              tau_end=2.0, anneal_steps=50, rope_theta=THETA, seed=5, max_prefill=S, with_values=True)
    h, twin, plain = kvx.KVEvict(**kw), kvx.KVEvict(**kw), kvx.KVEvict(**kw)
    gen = torch.Generator(device="cuda").manual_seed(1)

    def r(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)
    qw, kw_ = 1 + 0.1 * r(D), 1 + 0.1 * r(D)
    shared = {}
    if prefix:
        shared = {"prefix_k": r(H, prefix, D).half(), "prefix_v": r(H, prefix, D).half()}
    # the prompt: keys straight into the layout the cache takes
    pre_k = torch.empty(B, L, H, S, D, dtype=torch.float16, device="cuda")
    pre_v = r(B, L, H, S, D).half()
    for l in range(L):
        kvx.qk_norm_rope(None, r(B, S, H, D), None, pre_k[:, l].transpose(1, 2), rope_theta=THETA, k_weight=kw_, eps=EPS,
                         pos0=prefix)
    for x in (h, twin, plain):
        x.prefill(pre_k, values=pre_v)
    ev = [torch.empty(B, L, H, dtype=torch.int32, device="cuda") for _ in range(3)]
    pending = 0
    for t in range(T):
        k_new = torch.empty(B, L, H, D, dtype=torch.float16, device="cuda")
        v_new = r(B, L, H, D).half()
        for l in range(L):
            q, k = r(B, 1, G, D), r(B, 1, H, D)
            q_out = torch.empty(B, 1, G, D, dtype=torch.float16, device="cuda")
            kvx.qk_norm_rope(q, k, q_out, k_new[:, l, None], rope_theta=THETA, q_weight=qw, k_weight=kw_, eps=EPS,
                             pos0=prefix + h.next_pos)
            out = torch.empty(B, G, D, dtype=torch.float16, device="cuda")
            lse = torch.empty(B, G, device="cuda")
            h.attend(l, q_out[:, 0], out, k_new=k_new[:, l], v_new=v_new[:, l], lse=lse, **shared)
            if t % 5 != 4:
                continue
            # the rows through a twin: reading them applies the pending compaction, which h keeps
            torch.cuda.synchronize()
            kv = [[_rows(twin, b, l, hh) for hh in range(H)] for b in range(B)]
            keys = torch.stack([torch.stack([x[0] for x in row]) for row in kv])
            values = torch.stack([torch.stack([x[1] for x in row]) for row in kv])
            assert keys.shape[2] == min(S + t, [budget, 24, 16][l])
            want = ref.attend_batch(q_out[:, 0], k=keys, v=values, k_new=k_new[:, l], v_new=v_new[:, l], **shared)
            ref.check("out", out, want[0], want[2])
            ref.check("lse", lse, want[1], want[3])
        h.step(k_new, ev[0], v_new=v_new)
        twin.step(k_new, ev[1], v_new=v_new)
        plain.step(k_new, ev[2], v_new=v_new)
        assert torch.equal(ev[0], ev[1]) and torch.equal(ev[0], ev[2])
        pending += int((ev[0] >= 0).sum())
    assert pending > 0
    # attention changed nothing in the handle: the bits of a handle that never had any
    for a, b in zip(h.read_state(1, 1, 1), plain.read_state(1, 1, 1)):
        assert np.array_equal(a, b)
    h.check()


@pytest.mark.parametrize("B,budget,prefix", [(40, 20, 2500), (3, 20, 0), (60, 700, 0), (60, 300, 1700)])
def test_cache_rows_beside_a_large_prefix(kvx, B, budget, prefix):
    """Every way the rows are read (clusters, ranges, beside the tensor-core kernel) with a compaction pending; then after it."""
    H, N, D, T = 2, 4, 128, 9
    kw = dict(batch=B, n_layers=2, n_kv_heads=H, head_dim=D, layer_budgets=[budget, 12], n_sink=1, rope_theta=THETA,
              max_prefill=budget, with_values=True)
    h, twin = kvx.KVEvict(**kw), kvx.KVEvict(**kw)
    gen = torch.Generator(device="cuda").manual_seed(2)

    def r(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").half()
    keys, values = r(B, 2, H, budget, D), r(B, 2, H, budget, D)
    steps_k, steps_v = r(T, B, 2, H, D), r(T, B, 2, H, D)
    for x in (h, twin):
        x.prefill(keys, values=values)
        x.decode(steps_k, values=steps_v)
    q, k_new, v_new = r(B, N * H, D), r(B, H, D), r(B, H, D)
    shared = {"prefix_k": r(H, prefix, D), "prefix_v": r(H, prefix, D)} if prefix else {}
    for l, rows in ((0, budget), (1, 12)):
        kv = [[_rows(twin, b, l, hh) for hh in range(H)] for b in range(B)]
        k, v = (torch.stack([torch.stack([x[i] for x in row]) for row in kv]) for i in (0, 1))
        assert k.shape == (B, H, rows, D)
        want = ref.attend_batch(q, k=k, v=v, k_new=k_new, v_new=v_new, **shared)
        for again in range(2):
            out, lse = torch.full_like(q, float("nan")), torch.empty(B, N * H, device="cuda")
            h.attend(l, q, out, k_new=k_new, v_new=v_new, lse=lse, **shared)
            torch.cuda.synchronize()
            ref.check("out", out, want[0], want[2])
            ref.check("lse", lse, want[1], want[3])
            if l == 1:
                h.flush()                  # the second time with the compaction applied
    h.check()


def test_attend_refuses(kvx):
    q = torch.zeros(2, 4, 64, dtype=torch.float16, device="cuda")
    kw = dict(batch=2, n_layers=2, n_kv_heads=2, head_dim=64, avg_budget=16)
    keys_only, h = kvx.KVEvict(**kw), kvx.KVEvict(with_values=True, **kw)
    for handle, l, query in ((keys_only, 0, q), (h, 2, q), (h, -1, q), (h, 0, q[:1]), (h, 0, q.bfloat16())):
        with pytest.raises(kvx.KVEvictError) as e:
            handle.attend(l, query, torch.empty_like(query))
        assert e.value.code == kvx.ERR_INVALID_ARG
    out, lse = torch.ones_like(q), torch.zeros(2, 4, device="cuda")
    h.attend(0, q, out, lse=lse)           # an empty cache: nothing to attend to
    torch.cuda.synchronize()
    assert (out == 0).all() and (lse == float("-inf")).all()
