"""Numbers that the calls around the step cannot compute with, and outputs that overlap: refused before anything runs."""
import pytest

torch = pytest.importorskip("torch")
from test_attention_refusals import _attention, _qk, kvx  # noqa: E402,F401


@pytest.mark.parametrize("pos0,seq", [(1 << 31, 1), ((1 << 31) - 1, 2), (-(1 << 31) - 1, 1), (1 << 40, 1), ((1 << 63) - 1, 3),
                                      (-(1 << 63), 1)])
def test_positions_past_32_bits(kvx, pos0, seq):  # noqa: F811
    """A frequency of 53 bits leaves a position of 2^33 an angle's error of 2^-20, one of 2^50 no angle at all."""
    assert kvx.lib().kvevict_qk_norm_rope(_qk(kvx, pos0=pos0, seq=seq), None) == kvx.ERR_INVALID_ARG
    assert "pos0" in kvx.last_error()
    x = torch.zeros(2, seq, 4, 64)
    with pytest.raises((ValueError, kvx.KVEvictError), match="pos0"):
        kvx.qk_norm_rope(x, None, x.half(), None, rope_theta=1e4, pos0=pos0)


@pytest.mark.parametrize("eps", [1e-46, 1e-60, 5e-324])
def test_eps_that_is_zero_in_32_bits(kvx, eps):  # noqa: F811
    """It would make a row of zeros NaN where the formula has 0."""
    x = torch.zeros(2, 3, 4, 64)
    with pytest.raises(ValueError, match="eps"):
        kvx.qk_norm_rope(x, None, x.half(), None, rope_theta=1e4, eps=eps)


@pytest.mark.parametrize("kw", [dict(q_out_stride=(0, 64, 64)), dict(k_out_stride=(64, 0, 64)), dict(q_out_stride=(128, 64, 8)),
                                dict(q_out_stride=(128, -8, 64))])
def test_rotated_rows_that_overlap(kvx, kw):  # noqa: F811
    """Outputs that broadcast (strides of 0), or whose rows begin inside one another."""
    args = _qk(kvx, batch=2, seq=2, n_kv_heads=2, **kw)
    assert kvx.lib().kvevict_qk_norm_rope(args, None) == kvx.ERR_INVALID_ARG
    assert "overlap" in kvx.last_error()


@pytest.mark.parametrize("stride", [(0, 64), (256, 0), (256, 32), (-16, 64)])
def test_outputs_that_overlap(kvx, stride):  # noqa: F811
    assert kvx.lib().kvevict_attend(_attention(kvx, batch=2, q_stride=(256, 64), out_stride=stride), None) == kvx.ERR_INVALID_ARG
    assert "overlap" in kvx.last_error()
