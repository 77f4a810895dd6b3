"""Attention of prompts and drafted trees at the edges of its kernels' work: which kernel and cut a call takes, values and
logits that are not finite between them, far offsets."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")
import tokens_reference as tref  # noqa: E402
from tokens_inputs import ints, make, trees  # noqa: E402

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
NAN, INF = float("nan"), math.inf


@pytest.fixture(scope="module")
def kvx():
    import kv_cache_attention_02_gb300 as k
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    k.lib()
    return k


def _by(kvx, kernel, call, *x, **y):
    """The call by one of the two kernels: "few" (query rows) or "tensor"; "chosen": by whichever the library takes."""
    lib = kvx.lib()
    try:
        lib.kvevict_test_without_few_kernel(kernel == "tensor")
        lib.kvevict_test_without_tokens_kernel(kernel == "few")
        call(*x, **y)
    finally:
        lib.kvevict_test_without_few_kernel(0)
        lib.kvevict_test_without_tokens_kernel(0)
    torch.cuda.synchronize()


def _needs_152_sms():
    if torch.cuda.get_device_properties(0).multi_processor_count != 152:
        pytest.skip("the rules are for 152 SMs")


@pytest.mark.parametrize("tree,B,S,N,H,D,n,kernel", [
    (False, 1, 37, 1, 4, 64, 0, "few"), (False, 2, 30, 3, 2, 64, 0, "few"), (True, 1, 8, 1, 4, 64, 32, "few"),
    (True, 1, 16, 3, 8, 128, 512, "few"), (True, 1, 16, 4, 8, 128, 2048, "few"),
    (False, 1, 300, 4, 8, 128, 0, "tensor"), (False, 4, 256, 1, 8, 128, 0, "tensor"), (True, 8, 8, 4, 8, 128, 2048, "tensor"),
    (True, 9, 16, 4, 8, 128, 3000, "tensor")])
def test_which_kernel_answers(kvx, tree, B, S, N, H, D, n, kernel):
    """The kernels sum in different orders: a call's bits tell which one took it."""
    _needs_152_sms()
    call = kvx.attend_tree if tree else kvx.attend_prompt
    q, args = make(B, S, N, H, D, n=n, seed=S)
    if tree:
        args["parents"] = trees(B, S, S)
    found = {}
    for by in ("few", "tensor", "chosen"):
        found[by] = torch.empty(q.shape[:-1], device="cuda")
        _by(kvx, by, call, q, torch.empty_like(q), lse=found[by], **args)
    assert not torch.equal(found["few"], found["tensor"])
    assert torch.equal(found["chosen"], found[kernel])


@pytest.mark.parametrize("B,S,N,H,D,n,cut", [
    (1, 400, 4, 2, 64, 3000, True), (3, 40, 2, 2, 128, 5000, True), (1, 2100, 4, 1, 128, 0, True), (9, 16, 4, 8, 128, 3000, True),
    (4, 256, 1, 8, 128, 0, False), (3, 900, 4, 2, 128, 100, False), (2, 300, 3, 2, 128, 70, False)])
def test_which_calls_are_cut(kvx, B, S, N, H, D, n, cut):
    """Blocks are cut over CTAs where a workspace is asked for."""
    _needs_152_sms()
    q, args = make(B, S, N, H, D, n=n, seed=1)
    packed, _ = kvx._tokens(q, q, args["k_new"], args["v_new"], None, None, None, args.get("k"), args.get("v"), None, None, None, None,
                            False)
    need = ctypes.c_size_t(0)
    assert kvx.lib().kvevict_attend_tokens_workspace(packed, 0, ctypes.addressof(need)) == kvx.OK
    assert (need.value > 0) == cut


@pytest.mark.parametrize("B", [127, 128, 129])
def test_packed_sequences_at_the_few_kernels_limit(kvx, B):
    """It is taken for at most 128, a sequence a thread."""
    _needs_152_sms()
    starts = ints(*[0] * (B - 3), 4, 8, 12, 16)
    q, args = make(B, 16, 3, 2, 64, packed=True, seed=B)
    found = {}

    def checked(by):
        _, found[by] = tref.check("packed", kvx.attend_prompt, q, starts=starts, **args)
    for by in ("few", "tensor", "chosen"):
        _by(kvx, by, checked, by)
    assert not torch.equal(found["few"], found["tensor"])
    assert torch.equal(found["chosen"], found["few" if B <= 128 else "tensor"])


# (prompts of either kernel; blocks of 128 and 256 query rows, whole and cut)
SHAPES = [(2, 30, 3, 2, 64, 40), (2, 300, 3, 2, 128, 70), (1, 400, 4, 2, 64, 3000), (3, 40, 2, 2, 128, 5000)]


@pytest.mark.parametrize("kernel", ["few", "tensor"])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("B,S,N,H,D,n", SHAPES)
def test_logits_of_infinity(kvx, B, S, N, H, D, n, dtype, kernel):
    """NaN in out and lse of the heads that see the key, the same bits everywhere else."""
    q, args = make(B, S, N, H, D, n=n, dtype=dtype, seed=S)
    q[..., 0] = 1.0
    calls = [("k", S, kvx.attend_prompt, {}), ("k_new", S, kvx.attend_prompt, {})]
    if S <= 64:
        calls.append(("k_new", S, kvx.attend_tree, dict(parents=trees(B, S, 1))))
    for name, _, call, more in calls:
        want, wlse = torch.empty_like(q), torch.empty(q.shape[:-1], device="cuda")
        _by(kvx, kernel, call, q, want, lse=wlse, **args, **more)
        for at in (0, args[name].shape[2 if name == "k" else 1] - 1, 17):
            bad = dict(args, **{name: args[name].clone()})
            sees = torch.zeros(B, S, H, dtype=torch.bool)
            if name == "k":
                bad["k"][0, 1, at, 0] = INF
                sees[0, :, 1] = True
            else:
                bad["k_new"][0, at, 1, 0] = INF
                sees[0, :, 1] = tref.ancestors(more["parents"][0].tolist(), S)[:, at] if more else torch.arange(S) >= at
            sees = sees.repeat_interleave(N, 2).cuda()
            out, lse = torch.empty_like(want), torch.empty_like(wlse)
            _by(kvx, kernel, call, q, out, lse=lse, **bad, **more)
            assert out[sees].isnan().all() and lse[sees].isnan().all()
            assert torch.equal(out[~sees], want[~sees]) and torch.equal(lse[~sees], wlse[~sees])


@pytest.fixture(scope="module")
def far_space():
    """Six buffers of two rows' room, 2^31 elements and more apart."""
    if torch.cuda.mem_get_info()[0] < 50 * 2 ** 30:
        pytest.skip("needs 50 GB")
    yield [torch.empty(FAR + 2 ** 28, dtype=F16, device="cuda") for _ in range(6)]


FAR = 2 ** 31 + 1024


def _far(space, x, heads, between=FAR):
    """x in one of the buffers, with its dimension of two heads (or its tokens) so far apart."""
    strides = list(x.stride())
    strides[heads] = between
    view = space.as_strided(x.shape, strides)
    view.copy_(x)
    return view


@pytest.mark.parametrize("kernel", ["few", "tensor"])
@pytest.mark.parametrize("S,n", [(20, 0), (150, 0), (150, 3000), (40, 5000)])
def test_heads_far_apart(kvx, far_space, S, n, kernel):
    """More than 2^31 elements between the heads of queries, outputs, keys and values; whole blocks and cut ones."""
    q, args = make(1, S, 1, 2, 128, n=n, seed=S)
    call = kvx.attend_tree if S == 40 else kvx.attend_prompt
    args.update(dict(parents=trees(1, S, 2)) if S == 40 else {})
    q = _far(far_space[0], q, 2)
    out = _far(far_space[1], torch.full_like(q, 7.0), 2)
    for i, (name, heads) in enumerate((("k_new", 2), ("v_new", 2), ("k", 1), ("v", 1))):
        if name in args:
            args[name] = _far(far_space[2 + i], args[name], heads)
    _by(kvx, kernel, lambda: tref.check("far heads", call, q, out=out, **args))


@pytest.mark.parametrize("kernel", ["few", "tensor"])
def test_packed_tokens_far_apart(kvx, far_space, kernel):
    """A sequence whose first token is past 2^31 elements."""
    q, args = make(4, 140, 1, 2, 128, packed=True, seed=3)
    step = 2 ** 24 + 128
    q = _far(far_space[0], q, 0, step)
    out = _far(far_space[1], torch.full_like(q, 7.0), 0, step)
    args = {name: _far(far_space[2 + i], x, 0, step) for i, (name, x) in enumerate(args.items())}
    _by(kvx, kernel, lambda: tref.check("far tokens", kvx.attend_prompt, q, out=out, starts=ints(0, 60, 129, 131, 140), **args))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128])
def test_values_that_only_a_blocks_second_half_visits(kvx, D, dtype):
    """A block's first 128 tokens do not look at its second tile of keys, where a value is NaN: the same bits, call after call."""
    q, args = make(4, 256, 1, 8, D, dtype=dtype, seed=D)
    want, wlse = tref.check("prompt", kvx.attend_prompt, q, **args)
    for at in (129, 200, 255):
        changed = dict(args, v_new=args["v_new"].clone())
        changed["v_new"][:, at, :, 3] = NAN
        for _ in range(10):
            out, lse = torch.empty_like(want), torch.empty_like(wlse)
            kvx.attend_prompt(q, out, lse=lse, **changed)
            torch.cuda.synchronize()
            assert torch.equal(out[:, :at], want[:, :at]) and torch.equal(lse, wlse)
            assert out[:, at:, :, 3].isnan().all()
            assert torch.equal(out[..., :3], want[..., :3]) and torch.equal(out[..., 4:], want[..., 4:])


def test_workspace_of_the_largest_descriptions(kvx):
    """As much work as the arguments allow, far more than any memory: the size that every cut call asks for."""
    def need(B, S, G, H, n):
        packed = kvx._TOKENS.pack(0, B, S, G, H, 128, n, 0, 0.0, 0, *(0,) * 12, *(0,) * 19, 0)
        size = ctypes.c_size_t(0)
        assert kvx.lib().kvevict_attend_tokens_workspace(packed, 0, ctypes.addressof(size)) == kvx.OK
        return size.value
    cut = need(1, 400, 4, 2, 3000)
    assert cut > 0
    assert need(1, 1 << 29, 1 << 26, 1 << 26, (1 << 29) - 1) == need(1 << 10, 1 << 29, 1 << 16, 1 << 16, (1 << 29) - 1) == \
        need(64, 4096, 32, 8, 1 << 20)
