"""What kvevict_qk_norm_rope, kvevict_attend and kvevict_attend_cache refuse, before anything runs on a GPU."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

A = 1 << 20   # an aligned address that no call here gets to use


@pytest.fixture(scope="module")
def kvx():
    import kv_cache_attention_02_gb300 as k
    k.lib()
    return k


def _qk(kvx, **kw):
    f = dict(in_dtype=0, out_dtype=0, weight_dtype=0, batch=1, seq=1, n_heads=2, n_kv_heads=1, head_dim=64, eps=1e-6,
             reserved=0, rope_theta=1e4, pos0=0, q=A, k=A, q_out=A, k_out=A, q_weight=0, k_weight=0, positions=0)
    st = {s: (64, 64, 64) for s in ("q_stride", "k_stride", "q_out_stride", "k_out_stride")}
    for key, value in kw.items():
        (st if key in st else f)[key] = value
    return kvx._QK.pack(*f.values(), *(x for s in st.values() for x in s))


@pytest.mark.parametrize("kw,frag", [
    (dict(in_dtype=3), "in_dtype"), (dict(out_dtype=2), "out_dtype"), (dict(weight_dtype=-1), "weight_dtype"),
    (dict(batch=-1), "batch"), (dict(seq=-1), "seq"), (dict(n_heads=-1), "n_heads"), (dict(n_heads=65536), "65536"),
    (dict(head_dim=96), "head_dim"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"),
    (dict(rope_theta=0.0), "rope_theta"), (dict(rope_theta=float("inf")), "rope_theta"), (dict(reserved=1), "reserved"),
    (dict(q=0), "null"), (dict(k_out=0), "null"), (dict(q=A + 8), "aligned"), (dict(k_out=A + 2), "aligned"),
    (dict(q_stride=(64, 64, 60)), "16 bytes"), (dict(batch=2, k_out_stride=(4, 64, 64)), "16 bytes"),
    (dict(q_weight=A + 1), "aligned"), (dict(positions=A + 2), "aligned"),
])
def test_qk_refusals(kvx, kw, frag):
    assert kvx.lib().kvevict_qk_norm_rope(_qk(kvx, **kw), None) == kvx.ERR_INVALID_ARG
    assert frag in kvx.last_error()


def test_qk_nothing_to_do(kvx):
    assert kvx.lib().kvevict_qk_norm_rope(None, None) == kvx.ERR_INVALID_ARG
    for kw in (dict(batch=0), dict(seq=0), dict(n_heads=0, n_kv_heads=0)):
        assert kvx.lib().kvevict_qk_norm_rope(_qk(kvx, q=0, k=0, q_out=0, k_out=0, **kw), None) == kvx.OK


def _attention(kvx, **kw):
    f = dict(dtype=0, batch=1, n_heads=4, n_kv_heads=2, head_dim=64, n=8, prefix=8, reserved=0, scale=0.0, reserved2=0,
             q=A, out=A, lse=A, k=A, v=A, lens=0, k_new=A, v_new=A, prefix_k=A, prefix_v=A, prefix_lens=0, workspace=0)
    st = dict(q_stride=(64, 64), out_stride=(64, 64), k_stride=(64, 64, 64), v_stride=(64, 64, 64), k_new_stride=(64, 64),
              v_new_stride=(64, 64), prefix_k_stride=(64, 64), prefix_v_stride=(64, 64))
    last = kw.pop("workspace_bytes", 0)
    for key, value in kw.items():
        (st if key in st else f)[key] = value
    return kvx._ATTENTION.pack(*f.values(), *(x for s in st.values() for x in s), last)


@pytest.mark.parametrize("kw,frag", [
    (dict(dtype=2), "dtype"), (dict(batch=-1), "batch"), (dict(n_heads=3), "multiple"), (dict(n_heads=0), "multiple"),
    (dict(n_kv_heads=0), "multiple"), (dict(head_dim=80), "head_dim"), (dict(n=-1), "2^30"),
    (dict(n=1 << 29, prefix=1 << 29), "2^30"), (dict(prefix=-4), "2^30"), (dict(batch=1 << 26), "2^26"),
    (dict(scale=-1.0), "scale"), (dict(scale=float("inf")), "scale"), (dict(scale=float("nan")), "scale"),
    (dict(reserved=2), "reserved"), (dict(reserved2=2), "reserved"), (dict(q=0), "null"), (dict(out=0), "null"),
    (dict(k=0), "null"), (dict(v=0), "null"), (dict(prefix_v=0), "null"), (dict(k_new=0), "together"),
    (dict(v_new=0), "together"), (dict(q=A + 2), "aligned"), (dict(v=A + 8), "aligned"), (dict(k_new=A + 4), "aligned"),
    (dict(prefix_k=A + 2), "aligned"), (dict(out_stride=(64, 4)), "16 bytes"), (dict(k_stride=(64, 64, 68)), "16 bytes"),
    (dict(batch=2, v_new_stride=(4, 64)), "16 bytes"), (dict(prefix_v_stride=(64, 1)), "16 bytes"), (dict(lens=A + 1), "4-byte"),
    (dict(lse=A + 2), "4-byte"),
])
def test_attend_refusals(kvx, kw, frag):
    assert kvx.lib().kvevict_attend(_attention(kvx, **kw), None) == kvx.ERR_INVALID_ARG
    assert frag in kvx.last_error()


def test_attend_null_and_empty(kvx):
    lib = kvx.lib()
    assert lib.kvevict_attend(None, None) == kvx.ERR_INVALID_ARG
    assert lib.kvevict_attend(_attention(kvx, batch=0, q=0, out=0, k=0, v=0), None) == kvx.OK
    assert lib.kvevict_attend_cache(None, 0, _attention(kvx), None) == kvx.ERR_INVALID_ARG
    assert lib.kvevict_attend_workspace(_attention(kvx), 0, None) == kvx.ERR_INVALID_ARG
    n = ctypes.c_size_t(1)
    assert lib.kvevict_attend_workspace(None, 0, ctypes.addressof(n)) == kvx.ERR_INVALID_ARG
    assert lib.kvevict_attend_workspace(_attention(kvx, head_dim=32), 0, ctypes.addressof(n)) == kvx.ERR_INVALID_ARG


def test_tensors_are_checked(kvx):
    q, k = torch.zeros(2, 4, 64, dtype=torch.float16), torch.zeros(2, 2, 5, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA device"):
        kvx.attend(q, q, k=k, v=k)
    with pytest.raises(ValueError, match="together"):
        kvx.attend(q, q, k=k)
    with pytest.raises(ValueError, match="nothing to attend"):
        kvx.attend(q, q)
    with pytest.raises(ValueError, match="lens goes with"):
        kvx.attend(q, q, k_new=k[:, :, 0], v_new=k[:, :, 0], lens=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="fp16 or bf16"):
        kvx.attend(q.float(), q, k=k, v=k)
    with pytest.raises(ValueError, match="shape"):
        kvx.attend(q[0], q, k=k, v=k)
    with pytest.raises(ValueError, match="scale"):
        kvx.attend(q, q, k=k, v=k, scale=0.0)
    x = torch.zeros(2, 3, 4, 64)
    with pytest.raises(ValueError, match="CUDA device"):
        kvx.qk_norm_rope(x, None, x.half(), None, rope_theta=1e4)
    with pytest.raises(ValueError, match="must be given"):
        kvx.qk_norm_rope(None, None, None, None, rope_theta=1e4)
    with pytest.raises(ValueError, match="goes with"):
        kvx.qk_norm_rope(x, None, None, None, rope_theta=1e4)
    with pytest.raises(ValueError, match="fp16 or bf16"):
        kvx.qk_norm_rope(x, None, x, None, rope_theta=1e4)


@pytest.mark.parametrize("scale", [1e-39, 3e38])
def test_scales_outside_the_normal_floats_are_refused(kvx, scale):
    """Below them a scale would round towards 0, the default's mark; above 2^127 its base-2 form overflows."""
    assert kvx.lib().kvevict_attend(_attention(kvx, scale=scale), None) == kvx.ERR_INVALID_ARG
    assert "scale" in kvx.last_error()


@pytest.mark.parametrize("scale", [1e-60, 1e-39, 3e38, 1e60, 10**400, float("inf"), float("nan")])
def test_python_scales_outside_the_normal_floats_are_refused(kvx, scale):
    q, k = torch.zeros(2, 4, 64, dtype=torch.float16), torch.zeros(2, 2, 5, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="scale"):
        kvx.attend(q, q, k=k, v=k, scale=scale)


def test_subnormal_rope_theta_is_refused(kvx):
    """Its highest power overflows a double."""
    assert kvx.lib().kvevict_qk_norm_rope(_qk(kvx, rope_theta=1e-320), None) == kvx.ERR_INVALID_ARG
    assert "rope_theta" in kvx.last_error()


@pytest.mark.parametrize("kw,frag", [
    (dict(eps=1e39), "eps"), (dict(eps=-1e-6), "eps"), (dict(eps=float("nan")), "eps"), (dict(pos0=1 << 63), "pos0"),
    (dict(pos0=-(1 << 63) - 1), "pos0"), (dict(rope_theta=10**400), "rope_theta"), (dict(rope_theta=0.0), "rope_theta"),
    (dict(rope_theta=float("nan")), "rope_theta"), (dict(rope_theta=1e-320), "rope_theta"),
])
def test_python_numbers_out_of_range_are_refused(kvx, kw, frag):
    x = torch.zeros(2, 3, 4, 64)
    with pytest.raises(ValueError, match=frag):
        kvx.qk_norm_rope(x, None, x.half(), None, **{"rope_theta": 1e4, **kw})
