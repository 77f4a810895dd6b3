"""Joins of attention parts against their 64-bit form."""
import math

import pytest

torch = pytest.importorskip("torch")
import attention_reference as ref  # noqa: E402
import tokens_reference as tref  # noqa: E402

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def kvx():
    import kv_cache_attention_02_gb300 as k
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    k.lib()
    return k


def _parts(shape, count, dtype, seed=0, spread=3.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s):
        return torch.randn(*s, generator=gen, device="cuda")
    return [(r(*shape).to(dtype), r(*shape[:-1]) * spread + 5) for _ in range(count)]


def _check(kvx, parts, out=None, lse=None):
    want, wlse, bound, lbound = tref.join(parts)
    out = torch.full_like(parts[0][0], 7.0) if out is None else out
    lse = torch.full(out.shape[:-1], 7.0, device="cuda") if lse is None else lse
    kvx.attend_join(out, parts, lse=lse)
    torch.cuda.synchronize()
    ref.check("out", out, want, bound)
    ref.check("lse", lse, wlse, lbound)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("count", [1, 2, 3, 4, 5, 8])
@pytest.mark.parametrize("room", [(1,), (37,), (3, 50)])
def test_parts(kvx, room, count, D, dtype):
    _check(kvx, _parts((*room, 5, D), count, dtype, seed=count))


@pytest.mark.parametrize("spread", [0.0, 60.0, 1e4, 1e30])
def test_log_sums_of_any_size(kvx, spread):
    _check(kvx, _parts((40, 4, 128), 3, F16, spread=spread))


def test_parts_without_rows(kvx):
    parts = _parts((30, 4, 64), 3, BF16)
    for i, (part, lse) in enumerate(parts):
        gone = (torch.arange(30, device="cuda") >> i & 1) == 1
        lse[gone] = -math.inf
        part[gone] = float("nan")                    # whatever it holds
    _check(kvx, parts)
    out, lse = torch.empty_like(parts[0][0]), torch.empty(30, 4, device="cuda")
    kvx.attend_join(out, parts, lse=lse)
    assert (out[7] == 0).all() and (lse[7] == -math.inf).all()


@pytest.mark.parametrize("bad", [float("nan"), math.inf])
def test_lost_parts_show(kvx, bad):
    parts = _parts((6, 4, 128), 2, F16)
    parts[1][1][3, 2] = bad
    out, lse = torch.empty_like(parts[0][0]), torch.empty(6, 4, device="cuda")
    kvx.attend_join(out, parts, lse=lse)
    assert out[3, 2].isnan().all() and lse[3, 2].isnan()
    assert out.isnan().sum() == 128 and lse.isnan().sum() == 1


def test_in_place_and_strides(kvx):
    parts = _parts((2, 33, 8, 128), 3, F16)
    wide = torch.zeros(2, 8, 33, 136, dtype=F16, device="cuda")
    view = wide[..., :128].transpose(1, 2)
    view.copy_(parts[1][0])
    parts[1] = (view, parts[1][1])
    same = parts[2][0][:, :1].expand(-1, 33, -1, -1)          # one token's part for all
    parts[2] = (same, parts[2][1])
    want, wlse, bound, lbound = tref.join(parts)
    kvx.attend_join(view, parts, lse=parts[1][1])
    torch.cuda.synchronize()
    ref.check("out", view, want, bound)
    ref.check("lse", parts[1][1], wlse, lbound)
    assert (wide[..., 128:] == 0).all()


def test_prompt_behind_a_shared_prefix(kvx):
    """As they are used together: the prefix's part for all prompts at once, the prompts' own, and their join."""
    import tokens_inputs as inputs
    B, S, N, H, D, P = 3, 170, 4, 2, 128, 700
    q, args = inputs.make(B, S, N, H, D, dtype=BF16, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(8)
    pk, pv = (inputs.normal(gen, H, P, D, dtype=BF16) for _ in range(2))
    parts = [(torch.empty_like(q), torch.empty(B, S, N * H, device="cuda")) for _ in range(2)]
    flat = (B * S, N * H)
    kvx.attend(q.view(*flat, D), parts[0][0].view(*flat, D), prefix_k=pk, prefix_v=pv, lse=parts[0][1].view(flat))
    kvx.attend_prompt(q, parts[1][0], lse=parts[1][1], **args)
    out, lse = torch.empty_like(q), torch.empty(B, S, N * H, device="cuda")
    kvx.attend_join(out, parts, lse=lse)
    torch.cuda.synchronize()
    rows = [x[None].expand(B, -1, -1, -1) for x in (pk, pv)]
    want, wlse, bound, lbound, _ = tref.attend_batch(q, k=rows[0], v=rows[1], **args)
    # the parts carry a rounding of their own: half a step of each, by its weight
    ref.check("out", out, want, 2 * bound)
    ref.check("lse", lse, wlse, 2 * lbound)
