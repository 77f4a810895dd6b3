"""Attention of prompts and drafted trees at the edges of its kernels' work: which kernel and cut a call takes, values and
logits that are not finite between them, far offsets."""
import math

import pytest

torch = pytest.importorskip("torch")
import tokens_reference as tref  # noqa: E402
from tokens_inputs import make  # noqa: E402

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
