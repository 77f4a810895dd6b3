"""Attention of prompts and drafted trees in use: values that are not finite, streams, graphs, threads, workspaces, far
offsets, waits that run out, and the operators together around a cache."""
import ctypes
import math
import threading
import time

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import attention_reference as ref  # noqa: E402
import tokens_reference as tref  # noqa: E402
from tokens_inputs import ints, make, normal, trees  # noqa: E402

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
NAN, INF = float("nan"), math.inf


@pytest.fixture(scope="module", params=["chosen", "tensor"])
def kvx(request):
    """By the kernel that the library chooses (another one for few query rows), and all by the tensor cores'."""
    import kv_cache_attention_02_gb300 as k
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    k.lib().kvevict_test_without_few_kernel(request.param == "tensor")
    k.all_tensor = request.param == "tensor"
    yield k
    k.lib().kvevict_test_without_few_kernel(0)


# (blocks of 128 query rows, of 256, cut ones)
SHAPES = [(2, 30, 3, 2, 64, 0), (2, 300, 3, 2, 128, 70), (1, 2100, 4, 1, 128, 0), (3, 40, 2, 2, 128, 5000)]


@pytest.mark.parametrize("B,S,N,H,D,n", SHAPES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_later_tokens_do_not_show(kvx, B, S, N, H, D, n, dtype):
    """Keys and values of NaN and infinity from one token on: all tokens before it have the bits that they had."""
    q, args = make(B, S, N, H, D, n=n, dtype=dtype, seed=S)
    want, wlse = tref.check("prompt", kvx.attend_prompt, q, **args)
    for at in (S - 1, S // 2, S // 3):
        for name, bad in (("v_new", NAN), ("v_new", INF), ("k_new", NAN), ("k_new", -INF)):
            changed = dict(args, **{name: args[name].clone()})
            changed[name][:, at:, :, 5] = bad
            out, lse = torch.empty_like(want), torch.empty_like(wlse)
            kvx.attend_prompt(q, out, lse=lse, **changed)
            torch.cuda.synchronize()
            assert torch.equal(out[:, :at], want[:, :at]) and torch.equal(lse[:, :at], wlse[:, :at])
            if name == "v_new":
                assert not torch.isfinite(out[:, at:, :, 5]).any() and torch.equal(lse, wlse)
                assert torch.equal(out[..., :5], want[..., :5]) and torch.equal(out[..., 6:], want[..., 6:])
            elif bad != bad:
                assert out[:, at:].isnan().all() and lse[:, at:].isnan().all()


@pytest.mark.parametrize("N,D,n", [(3, 64, 0), (4, 128, 300), (9, 128, 140)])
def test_other_branches_do_not_show(kvx, N, D, n):
    B, T, H = 2, 40, 2
    q, args = make(B, T, N, H, D, n=n, seed=T)
    parents = trees(B, T, 1)
    want, wlse = tref.check("tree", kvx.attend_tree, q, parents=parents, **args)
    seen = torch.stack([tref.ancestors(p.tolist(), T) for p in parents]).cuda()
    for at in (0, 7, 39):
        sees = seen[:, :, at]
        for name in ("v_new", "k_new"):
            changed = dict(args, **{name: args[name].clone()})
            changed[name][:, at, :, 9] = NAN
            out, lse = torch.empty_like(want), torch.empty_like(wlse)
            kvx.attend_tree(q, out, lse=lse, parents=parents, **changed)
            torch.cuda.synchronize()
            assert torch.equal(out[~sees], want[~sees]) and torch.equal(lse[~sees], wlse[~sees])
            assert out[sees][..., 9].isnan().all()
            assert (torch.equal(lse, wlse) if name == "v_new" else lse[sees].isnan().all())


@pytest.mark.parametrize("S,n", [(100, 200), (300, 1000), (40, 5000)])
def test_rows_and_tokens_past_a_length_may_hold_anything(kvx, S, n):
    B, N, H, D = 3, 4, 2, 128
    q, args = make(B, S, N, H, D, n=n, seed=S)
    lens, new_lens = ints(n, n // 3, 0), ints(S // 2, S - 1, 1)
    want, wlse = tref.check("prompt", kvx.attend_prompt, q, lens=lens, new_lens=new_lens, **args)
    for b in range(B):
        for name in ("k", "v"):
            args[name][b, :, int(lens[b]):] = NAN
            args[name + "_new"][b, int(new_lens[b]):] = NAN
        q[b, int(new_lens[b]):] = NAN
    out, lse = torch.full_like(want, 7.0), torch.full_like(wlse, 7.0)
    kvx.attend_prompt(q, out, lse=lse, lens=lens, new_lens=new_lens, **args)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wlse)


def test_neighbours_in_a_packed_batch_do_not_show(kvx):
    q, args = make(3, 330, 2, 2, 64, packed=True)
    at = ints(0, 100, 230, 330)
    want, wlse = tref.check("packed", kvx.attend_prompt, q, starts=at, **args)
    for x in (q, args["k_new"], args["v_new"]):
        x[100:230] = NAN
    out, lse = torch.empty_like(want), torch.empty_like(wlse)
    kvx.attend_prompt(q, out, lse=lse, starts=at, **args)
    torch.cuda.synchronize()
    rest = torch.ones(330, dtype=torch.bool, device="cuda")
    rest[100:230] = False
    assert torch.equal(out[rest], want[rest]) and torch.equal(lse[rest], wlse[rest])
    assert out[~rest].isnan().all() and lse[~rest].isnan().all()


@pytest.mark.parametrize("S,n", [(60, 200), (300, 500)])
def test_keys_that_take_no_weight_and_all_of_it(kvx, S, n):
    """Logits of -inf only: out 0 and lse -inf. Logits of any size, the largest far from the others."""
    q, args = make(1, S, 2, 2, 128, n=n, dtype=BF16, seed=1)
    q[..., 0] = 1.0
    none = dict(args, k=args["k"].clone(), k_new=args["k_new"].clone())
    none["k"][..., 0], none["k_new"][..., 0] = -INF, -INF
    out, lse = torch.empty_like(q), torch.empty(1, S, 4, device="cuda")
    kvx.attend_prompt(q, out, lse=lse, **none)
    torch.cuda.synchronize()
    assert (out == 0).all() and (lse == -INF).all()
    for size in (1e3, 1e9, 1e30):
        big = dict(args, k=args["k"] * size)
        tref.check("large logits", kvx.attend_prompt, q, **big)
        tref.check("large logits", kvx.attend_tree, q[:, :50], k=big["k"], v=args["v"], k_new=args["k_new"][:, :50] * size,
                   v_new=args["v_new"][:, :50], parents=trees(1, 50))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("nats", [12.0, 17.8])
@pytest.mark.parametrize("S,N", [(30, 4), (70, 4)])
def test_a_long_tail_behind_a_dominant_key(kvx, S, N, nats, dtype):
    """fp16 weights keep 2^-7 of the largest one's smallest step: 2^-25 of 2^-7 for each row of the tail."""
    H, D, n = 1, 128, 20000
    q, args = make(1, S, N, H, D, n=n, dtype=dtype, seed=2)
    q *= 0.2
    q[..., 0] = 8.0
    for x in ("k", "k_new"):
        args[x].mul_(0.25)[..., 0] = 0.0
    args["v"].mul_(0.1).add_(1.0)
    args["k"][..., 5, :], args["v"][..., 5, :] = 0.0, 0.0
    args["k"][..., 5, 0] = nats * math.sqrt(D) / 8.0
    out, lse = torch.empty_like(q), torch.empty(1, S, N, device="cuda")
    kvx.attend_prompt(q, out, lse=lse, **args)
    torch.cuda.synchronize()
    want, wlse, bound, lbound, _ = tref.attend_batch(q, **args)
    if dtype is F16:
        keys = torch.cat([args["k"][0, 0], args["k_new"][0, :1, 0]]).double()
        top = (q[0].double() @ keys.T * D ** -0.5).amax(-1)
        low = 2.0 ** -25 * torch.exp(top - wlse[0])[..., None] * (args["v"][0, 0].double().abs().sum(0))
        bound = bound - (low * (1 - 2.0 ** -7))[None]
    ref.check("out", out, want, bound)
    ref.check("lse", lse, wlse, lbound)


def test_offsets_past_32_bits(kvx):
    """Strides whose products pass 2^31 elements: sequences of rows, tokens of a prompt, heads of its output."""
    far = 2 ** 31 + 1024
    if torch.cuda.mem_get_info()[0] < 40 * 2 ** 30:
        pytest.skip("needs 40 GB")
    base = [torch.zeros(far + 2 ** 28, dtype=F16, device="cuda") for _ in range(4)]
    B, S, N, H, D, n = 2, 140, 2, 2, 128, 300
    q, args = make(B, S, N, H, D, n=n, seed=9)
    for name, x in zip(("k", "v", "k_new"), base):
        view = x.as_strided((B, *args[name].shape[1:]), (far, *args[name].stride()[1:]))
        view.copy_(args[name])
        args[name] = view
    out = base[3].as_strided(q.shape, (far, *q.stride()[1:]))
    out.fill_(7.0)
    tref.check("far sequences", kvx.attend_prompt, q, out=out, **args)
    step = 2 ** 24 + 128                       # elements between tokens: token 139 is past 2^31
    q, args = make(1, S, N, H, D, seed=10)
    for name, x in zip(("k_new", "v_new"), base):
        view = x.as_strided(args[name].shape, (0, step, D, 1))
        view.copy_(args[name])
        args[name] = view
    qf = base[2].as_strided(q.shape, (0, step, D, 1))
    qf.copy_(q)
    out = base[3].as_strided(q.shape, (0, step, D, 1))
    out.fill_(7.0)
    tref.check("far tokens", kvx.attend_prompt, qf, out=out, **args)


def _calls(kvx, seed=0):
    """One block a CTA, ranges of whole blocks, cut blocks, and a tree over ranges."""
    found = []
    for B, S, N, H, D, n in ((1, 60, 3, 2, 128, 0), (3, 900, 4, 2, 128, 100), (1, 400, 4, 2, 64, 3000)):
        q, args = make(B, S, N, H, D, n=n, seed=seed)
        found.append((kvx.attend_prompt, q, args))
    q, args = make(9, 16, 4, 8, 128, n=3000, seed=seed)
    found.append((kvx.attend_tree, q, dict(args, parents=trees(9, 16, seed))))
    return found


@pytest.mark.parametrize("which", range(4))
def test_repeat_streams_and_graphs(kvx, which):
    """The same bits call after call, on other streams at once, and from two captured graphs that replay together."""
    call, q, args = _calls(kvx)[which]
    want, wlse = tref.check("call", call, q, **args)
    side = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(q) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for s, o in zip(side, outs):
            call(q, o, stream=s, **args)
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, o in zip(graphs, outs):
        with torch.cuda.graph(g):
            call(q, o, **args)
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
    call(q, other, **args)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], other) and not torch.equal(other, want)


def test_two_threads_at_once(kvx):
    jobs = [_calls(kvx, seed) for seed in (1, 2)]
    streams = [torch.cuda.Stream() for _ in jobs]

    def once(job, stream):
        outs = [torch.zeros_like(q) for _, q, _ in job]
        stream.wait_stream(torch.cuda.current_stream())          # the zeros are there
        for (call, q, args), out in zip(job, outs):
            call(q, out, stream=stream, **args)
        return outs
    torch.cuda.synchronize()
    want = [once(job, s) for job, s in zip(jobs, streams)]
    torch.cuda.synchronize()
    found, errors = [[] for _ in jobs], []

    def work(i):
        try:
            with torch.cuda.stream(streams[i]):
                for _ in range(20):
                    found[i].append(once(jobs[i], streams[i]))
        except Exception as e:      # noqa: BLE001 -- shown by the test's own thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for w, runs in zip(want, found):
        assert len(runs) == 20 and all(torch.equal(a, b) for run in runs for a, b in zip(w, run))


@pytest.mark.parametrize("which", range(4))
def test_other_stream_than_the_current_one(kvx, which):
    call, q, args = _calls(kvx)[which]
    want, _ = tref.check("call", call, q, **args)
    side = torch.cuda.Stream()
    for given, current in ((side, None), (side.cuda_stream, None), (0, side), (torch.cuda.default_stream(), side)):
        out = torch.zeros_like(q)
        torch.cuda.synchronize()
        with torch.cuda.stream(current):
            for _ in range(3):
                call(q, out, stream=given, **args)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_workspace_of_the_c_call(kvx):
    """Too little workspace launches nothing; the size asked for is enough, and nothing past it is written."""
    _, q, args = _calls(kvx)[2]
    want, wlse = tref.check("call", kvx.attend_prompt, q, **args)
    out, lse = torch.full_like(q, 5.0), torch.empty_like(wlse)
    packed, stream = kvx._tokens(q, out, args["k_new"], args["v_new"], None, None, None, args["k"], args["v"], None, lse, None, None,
                                 False)
    need = ctypes.c_size_t(0)
    assert kvx.lib().kvevict_attend_tokens_workspace(packed, 0, ctypes.addressof(need)) == kvx.OK and need.value > 0
    space = torch.full((need.value + 4096,), 7, dtype=torch.uint8, device="cuda")

    def call(at, size):
        filled = bytearray(packed)
        kvx.struct.pack_into("=Q", filled, kvx._WORKSPACE_AT, at)
        kvx.struct.pack_into("=Q", filled, kvx._TOKENS_BYTES_AT, size)
        rc = kvx.lib().kvevict_attend_prompt(bytes(filled), stream)
        torch.cuda.synchronize()
        return rc
    for at, size in ((0, 0), (0, need.value), (space.data_ptr(), need.value - 1), (space.data_ptr() + 8, need.value)):
        assert call(at, size) == kvx.ERR_WORKSPACE and "workspace" in kvx.last_error()
    assert (out == 5).all()
    assert call(space.data_ptr(), need.value) == kvx.OK
    assert torch.equal(out, want) and torch.equal(lse, wlse) and (space[need.value:] == 7).all()


def test_empty_calls_and_sequences(kvx):
    q, args = make(2, 5, 2, 2, 64)
    none = ints(0, -3)
    for call in (kvx.attend_prompt, kvx.attend_tree):
        tref.check("empty", call, q, new_lens=none, **args)
        call(q[:0], torch.empty_like(q[:0]), **{x: y[:0] for x, y in args.items()})
        call(q[:, :0], torch.empty_like(q[:, :0]), **{x: y[:, :0] for x, y in args.items()})
    q, args = make(2, 5, 2, 2, 64, packed=True)
    tref.check("empty", kvx.attend_prompt, q, starts=ints(*[3] * 200), **args)
    kvx.attend_prompt(q, q, starts=ints(0), **args)             # no sequence


@pytest.mark.parametrize("B,S,N,H,D,n", [(1, 30, 4, 1, 128, 0), (1, 300, 4, 1, 64, 100), (1, 2000, 4, 2, 128, 0), (4, 16, 4, 8, 128, 900)])
def test_a_wait_that_runs_out(kvx, B, S, N, H, D, n):
    """NaN where the lost tile belongs, what is elsewhere right, and the next call as ever. (The library's test hook leaves one
    copy unissued: the bounded wait runs out, nothing hangs.)"""
    if not kvx.all_tensor:
        pytest.skip("the kernel for few query rows waits for nothing")
    q, args = make(B, S, N, H, D, n=n, seed=3)
    want, wlse = tref.check("call", kvx.attend_prompt, q, **args)
    out, lse = torch.zeros_like(q), torch.zeros_like(wlse)
    assert kvx.lib().kvevict_test_stall_next_step(None) == kvx.OK
    t0 = time.time()
    kvx.attend_prompt(q, out, lse=lse, **args)
    torch.cuda.synchronize()
    assert 0.5 < time.time() - t0 < 10.0
    assert out[0, 0, 0].isnan().all() and lse[0, 0, 0].isnan()
    lost = lse.isnan()
    assert torch.equal(out.isnan(), lost[..., None].expand_as(out))
    assert torch.equal(out[~lost], want[~lost]) and torch.equal(lse[~lost], wlse[~lost])
    kvx.attend_prompt(q, out, lse=lse, **args)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wlse)


# ---------------------------------------------------------------- around a cache
def _rows(h, b, l, hh):
    keys = h.read_state(b, l, hh)[0].view(np.float16)
    return [torch.from_numpy(x.copy()).cuda() for x in (keys, h.read_values(b, l, hh).view(np.float16))]


def _layer(h, l):
    kv = [[_rows(h, b, l, hh) for hh in range(h.H)] for b in range(h.B)]
    return [torch.stack([torch.stack([x[i] for x in row]) for row in kv]) for i in (0, 1)]


@pytest.mark.parametrize("B,H,D,N,T,budget", [(2, 2, 64, 3, 7, 20), (1, 8, 128, 3, 16, 512), (3, 2, 128, 4, 33, 127), (9, 8, 128, 4, 8, 600),
                                              (2, 2, 64, 5, 64, 128), (2, 1, 128, 1, 5, 383)])
def test_trees_over_a_handle(kvx, B, H, D, N, T, budget):
    """Rows as the cache holds them, with a compaction pending (a twin's, as reading applies it) and without; before any
    eviction, too. The handle keeps its bits."""
    kw = dict(batch=B, n_layers=2, n_kv_heads=H, head_dim=D, layer_budgets=[budget, 9], n_sink=1, rope_theta=5e5, max_prefill=budget,
              with_values=True)
    h, twin, plain = (kvx.KVEvict(**kw) for _ in range(3))
    gen = torch.Generator(device="cuda").manual_seed(budget)
    keys, values = (normal(gen, B, 2, H, budget - 3, D) for _ in range(2))
    for x in (h, twin, plain):
        x.prefill(keys, values=values)
    q, args = make(B, T, N, H, D, seed=T)
    args["parents"] = trees(B, T, T)
    args["new_lens"] = ints(*[max(1, T - b) for b in range(B)])
    for t in range(8):
        if t in (0, 3, 6, 7):
            torch.cuda.synchronize()
            for l in range(2):
                k, v = _layer(twin, l)
                assert k.shape[2] == min(budget - 3 + t, [budget, 9][l])
                tref.check(f"layer {l} after {t}", lambda *x, k, v, **y: h.attend_tree(l, *x, **y), q, k=k, v=v, **args)
        step = [normal(gen, B, 2, H, D) for _ in range(2)]
        for x in (h, twin, plain):
            x.step(step[0], v_new=step[1])
    for a, b in zip(h.read_state(B - 1, 0, H - 1), plain.read_state(B - 1, 0, H - 1)):
        assert np.array_equal(a, b)
    h.check()


def test_an_evicted_row_that_is_not_finite(kvx):
    """The row that a step evicted is still in place, its compaction pending: it is not looked at."""
    B, H, D, budget = 1, 1, 128, 40
    h = kvx.KVEvict(batch=B, n_layers=1, n_kv_heads=H, head_dim=D, layer_budgets=[budget], n_sink=1, max_prefill=budget, with_values=True)
    gen = torch.Generator(device="cuda").manual_seed(1)
    keys, values = (normal(gen, B, 1, H, budget, D) for _ in range(2))
    values[:, :, :, 1:] = INF                     # (row 0 is a sink)
    h.prefill(keys, values=values)
    h.step(normal(gen, B, 1, H, D), v_new=normal(gen, B, 1, H, D))
    q, args = make(B, 4, 2, H, D, seed=2)
    out = torch.empty_like(q)
    h.attend_tree(0, q, out, **args)
    torch.cuda.synchronize()
    assert not torch.isfinite(out).any()          # the others count
    ev = torch.empty(B, 1, H, dtype=torch.int32, device="cuda")
    h.reset()
    values[:] = 1.0
    h.prefill(keys, values=values)
    probe = [normal(gen, B, 1, H, D) for _ in range(2)]
    h.step(probe[0], ev, v_new=probe[1])
    gone = int(ev[0, 0, 0])
    values[0, 0, 0, gone] = NAN
    h.reset()
    h.prefill(keys, values=values)
    h.step(probe[0], ev, v_new=probe[1])
    assert int(ev[0, 0, 0]) == gone < budget
    h.attend_tree(0, q, out, **args)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all()


def test_handle_refusals(kvx):
    q, args = make(2, 5, 2, 2, 64)
    kw = dict(batch=2, n_layers=2, n_kv_heads=2, head_dim=64, avg_budget=16)
    keys_only, h = kvx.KVEvict(**kw), kvx.KVEvict(with_values=True, **kw)
    half = {x: y[:1] for x, y in args.items()}
    wide = {x: y.bfloat16() for x, y in args.items()}
    for handle, l, query, a in ((keys_only, 0, q, args), (h, 2, q, args), (h, -1, q, args), (h, 0, q[:1], half),
                                (h, 0, q.bfloat16(), wide)):
        with pytest.raises(kvx.KVEvictError) as e:
            handle.attend_tree(l, query, torch.empty_like(query), **a)
        assert e.value.code == kvx.ERR_INVALID_ARG
    tref.check("empty cache", lambda *x, **y: h.attend_tree(0, *x, **y), q, **args)


def test_a_wait_that_runs_out_on_a_handle(kvx):
    if not kvx.all_tensor:
        pytest.skip("the kernel for few query rows waits for nothing")
    h = kvx.KVEvict(batch=1, n_layers=1, n_kv_heads=2, head_dim=64, avg_budget=16, max_prefill=8, with_values=True)
    q, args = make(1, 5, 2, 2, 64)
    want, out = torch.empty_like(q), torch.zeros_like(q)
    h.attend_tree(0, q, want, **args)
    torch.cuda.synchronize()
    h.check()
    assert kvx.lib().kvevict_test_stall_next_step(None) == kvx.OK
    h.attend_tree(0, q, out, **args)
    torch.cuda.synchronize()
    assert out[0, :, :2].isnan().all()
    with pytest.raises(kvx.KVEvictError) as e:
        h.check()
    assert e.value.code == kvx.ERR_DEVICE_CHECK
    h.attend_tree(0, q, out, **args)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_speculative_serving(kvx):
    """As a serving loop has them together, behind a shared prefix: norm and rotation, the prompt's attention joined with
    the prefix's, prefill, a drafted tree, the accepted path as steps, and the next token's attention."""
    B, L, H, N, D, S, P, T, budget, theta = 2, 2, 2, 3, 128, 50, 333, 9, 80, 5e5
    G = N * H
    gen = torch.Generator(device="cuda").manual_seed(6)

    def r(*shape):
        return normal(gen, *shape)
    h = kvx.KVEvict(batch=B, n_layers=L, n_kv_heads=H, head_dim=D, layer_budgets=[budget] * L, n_sink=2, rope_theta=theta, max_prefill=S,
                    with_values=True)
    pk, pv = r(L, H, P, D), r(L, H, P, D)
    pre_k, pre_v = torch.empty(B, L, H, S, D, dtype=F16, device="cuda"), r(B, L, H, S, D)
    part = [(torch.empty(B, S, G, D, dtype=F16, device="cuda"), torch.empty(B, S, G, device="cuda")) for _ in range(2)]
    for l in range(L):
        q, k = r(B, S, G, D), r(B, S, H, D)
        q_rot = torch.empty_like(q)
        kvx.qk_norm_rope(q, k, q_rot, pre_k[:, l].transpose(1, 2), rope_theta=theta, pos0=P)
        keys, values = pre_k[:, l].transpose(1, 2), pre_v[:, l].transpose(1, 2)
        flat = (B * S, G)
        kvx.attend(q_rot.view(*flat, D), part[0][0].view(*flat, D), prefix_k=pk[l], prefix_v=pv[l], lse=part[0][1].view(flat))
        kvx.attend_prompt(q_rot, part[1][0], k_new=keys, v_new=values, lse=part[1][1])
        out = torch.empty_like(q)
        kvx.attend_join(out, part)
        torch.cuda.synchronize()
        shared = [x[l][None].expand(B, -1, -1, -1) for x in (pk, pv)]
        want, _, bound, _, _ = tref.attend_batch(q_rot, k_new=keys, v_new=values, k=shared[0], v=shared[1])
        ref.check("prompt", out, want, 2 * bound)
    h.prefill(pre_k, values=pre_v)
    parents = ints(-1, 0, 0, 1, 1, 2, 3, 6, 6)
    depth = ints(0, 1, 1, 2, 2, 2, 3, 4, 4)
    path = [0, 1, 3, 6, 8]                               # accepted, say
    tree_k, tree_v = torch.empty(B, L, T, H, D, dtype=F16, device="cuda"), r(B, L, T, H, D)
    queries, answers = [], []
    for l in range(L):
        q, k = r(B, T, G, D), r(B, T, H, D)
        q_rot = torch.empty_like(q)
        kvx.qk_norm_rope(q, k, q_rot, tree_k[:, l], rope_theta=theta, positions=(depth + P + h.next_pos).expand(B, -1).contiguous())
        own = [(torch.empty_like(q), torch.empty(B, T, G, device="cuda")) for _ in range(2)]
        h.attend_tree(l, q_rot, own[0][0], k_new=tree_k[:, l], v_new=tree_v[:, l], parents=parents, lse=own[0][1])
        kvx.attend(q_rot.view(B * T, G, D), own[1][0].view(B * T, G, D), prefix_k=pk[l], prefix_v=pv[l], lse=own[1][1].view(B * T, G))
        out = torch.empty_like(q)
        kvx.attend_join(out, own)
        torch.cuda.synchronize()
        queries.append(q_rot), answers.append(out)
    # the accepted tokens one by one, as a loop without drafting has them: the same answers, within the calls' roundings
    for t in path:
        for l in range(L):
            one = torch.empty(B, G, D, dtype=F16, device="cuda")
            h.attend(l, queries[l][:, t], one, k_new=tree_k[:, l, t], v_new=tree_v[:, l, t], prefix_k=pk[l], prefix_v=pv[l])
            torch.cuda.synchronize()
            # both are within their bounds of the same sum: values are below 6 in size, three roundings to fp16 each
            assert (one.float() - answers[l][:, t].float()).abs().max() <= 6 * 2.0 ** -11 * 6
        h.step(tree_k[:, :, t].contiguous(), v_new=tree_v[:, :, t].contiguous())
    assert h.next_pos == S + len(path)
    h.check()
