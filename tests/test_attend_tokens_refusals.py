"""What kvevict_attend_prompt, kvevict_attend_tree and kvevict_attend_join refuse, before anything runs on a GPU."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

A = 1 << 20   # an aligned address that no call here gets to use


@pytest.fixture(scope="module")
def kvx():
    import kv_cache_attention_02_gb300 as k
    k.lib()
    return k


def _tokens(kvx, **kw):
    f = dict(dtype=0, batch=2, seq=8, n_heads=4, n_kv_heads=2, head_dim=64, n=8, reserved=0, scale=0.0, reserved2=0, q=A, out=A,
             lse=A, k_new=A, v_new=A, starts=0, new_lens=0, parents=0, k=A, v=A, lens=0, workspace=0)
    st = dict(q_stride=(2048, 256, 64), out_stride=(2048, 256, 64), k_new_stride=(1024, 128, 64), v_new_stride=(1024, 128, 64),
              k_stride=(1024, 512, 64), v_stride=(1024, 512, 64))
    last = kw.pop("parents_stride", 8), kw.pop("workspace_bytes", 0)
    for key, value in kw.items():
        (st if key in st else f)[key] = value
    return kvx._TOKENS.pack(*f.values(), *(x for s in st.values() for x in s), *last)


BOTH = [
    (dict(dtype=2), "dtype"), (dict(batch=-1), "batch"), (dict(seq=-1), "seq"), (dict(n_heads=3), "multiple"),
    (dict(n_heads=0), "multiple"), (dict(n_kv_heads=0), "multiple"), (dict(head_dim=80), "head_dim"), (dict(n=-1), "n must"),
    (dict(n=(1 << 30) - 8), "2^30"), (dict(batch=1 << 26), "2^26"), (dict(scale=-1.0), "scale"), (dict(scale=1e-39), "scale"),
    (dict(scale=float("nan")), "scale"), (dict(scale=3e38), "scale"), (dict(reserved=2), "reserved"),
    (dict(reserved2=2), "reserved"), (dict(starts=A, new_lens=A), "together"), (dict(q=0), "null"), (dict(out=0), "null"),
    (dict(k_new=0), "null"), (dict(v_new=0), "null"), (dict(k=0), "null"), (dict(v=0), "null"), (dict(q=A + 2), "aligned"),
    (dict(out=A + 8), "aligned"), (dict(k_new=A + 4), "aligned"), (dict(v=A + 8), "aligned"),
    (dict(q_stride=(2048, 252, 64)), "16 bytes"), (dict(v_new_stride=(1024, 128, 68)), "16 bytes"),
    (dict(k_stride=(1024, 512, 60)), "16 bytes"), (dict(out_stride=(2048, 256, 0)), "overlap"),
    (dict(out_stride=(0, 256, 64)), "overlap"), (dict(k_new_stride=(1024, 0, 64)), "strides of keys"),
    (dict(k_new_stride=(-1024, 128, 64)), "strides of keys"), (dict(v_new_stride=(1024, 32, 64)), "strides of keys"),
    (dict(k_stride=(1 << 39, 512, 64)), "strides of keys"), (dict(v_stride=(1024, -512, 64)), "strides of keys"),
    (dict(v_stride=(1024, 512, 0)), "strides of keys"), (dict(q_stride=(2048, 256, 0)), "strides of q"),
    (dict(q_stride=(2048, 0, 64)), "strides of q"), (dict(q_stride=(-2048, 256, 64)), "strides of q"),
    (dict(q_stride=(2048, 256, 32)), "strides of q"), (dict(lse=A + 2), "4-byte"), (dict(lens=A + 1), "4-byte"),
    (dict(new_lens=A + 2), "4-byte"),
]


@pytest.mark.parametrize("kw,frag", BOTH + [(dict(parents=A), "parents"), (dict(starts=A + 2), "4-byte"),
                                            (dict(seq=1 << 29, n_heads=8), "2^30")])
def test_prompt_refusals(kvx, kw, frag):
    assert kvx.lib().kvevict_attend_prompt(_tokens(kvx, **kw), None) == kvx.ERR_INVALID_ARG
    assert frag in kvx.last_error()


@pytest.mark.parametrize("kw,frag", BOTH + [(dict(seq=65), "64 tokens"), (dict(starts=A), "starts"), (dict(parents=A + 1), "4-byte")])
def test_tree_refusals(kvx, kw, frag):
    assert kvx.lib().kvevict_attend_tree(_tokens(kvx, **kw), None) == kvx.ERR_INVALID_ARG
    assert frag in kvx.last_error()


def test_nothing_to_do(kvx):
    lib = kvx.lib()
    for call in (lib.kvevict_attend_prompt, lib.kvevict_attend_tree):
        assert call(None, None) == kvx.ERR_INVALID_ARG
        for kw in (dict(batch=0), dict(seq=0)):
            assert call(_tokens(kvx, q=0, out=0, k_new=0, v_new=0, k=0, v=0, **kw), None) == kvx.OK
    assert lib.kvevict_attend_tree_cache(None, 0, _tokens(kvx), None) == kvx.ERR_INVALID_ARG
    n = ctypes.c_size_t(1)
    assert lib.kvevict_attend_tokens_workspace(_tokens(kvx), 0, None) == kvx.ERR_INVALID_ARG
    assert lib.kvevict_attend_tokens_workspace(None, 0, ctypes.addressof(n)) == kvx.ERR_INVALID_ARG
    assert lib.kvevict_attend_tokens_workspace(_tokens(kvx, head_dim=32), 0, ctypes.addressof(n)) == kvx.ERR_INVALID_ARG
    assert lib.kvevict_attend_tokens_workspace(_tokens(kvx, seq=0), 0, ctypes.addressof(n)) == kvx.OK and n.value == 0


def _join(kvx, **kw):
    f = dict(dtype=0, batch=2, seq=3, n_heads=4, head_dim=64, parts=2, reserved=(0, 0), part=(A, A), part_lse=(A, A), out=A, lse=A,
             part_stride=((768, 256, 64),) * 2, out_stride=(768, 256, 64))
    f.update(kw)
    eight = [(tuple(f[x]) + (0,) * 8)[:8] for x in ("part", "part_lse")]
    strides = (tuple(x for s in f["part_stride"] for x in s) + (0,) * 24)[:24]
    return kvx._JOIN.pack(*(f[x] for x in ("dtype", "batch", "seq", "n_heads", "head_dim", "parts")), *f["reserved"], *eight[0], *eight[1],
                          f["out"], f["lse"], *strides, *f["out_stride"])


@pytest.mark.parametrize("kw,frag", [
    (dict(dtype=2), "dtype"), (dict(batch=-1), "batch"), (dict(seq=-1), "seq"), (dict(n_heads=-1), "n_heads"),
    (dict(head_dim=96), "head_dim"), (dict(parts=0), "parts"), (dict(parts=9), "parts"), (dict(reserved=(0, 1)), "reserved"),
    (dict(batch=1 << 20, seq=1 << 20), "2^34"), (dict(out=0), "null"), (dict(part=(A, 0)), "null"), (dict(part_lse=(0, A)), "null"),
    (dict(out=A + 8), "aligned"), (dict(part=(A + 2, A)), "aligned"), (dict(part_lse=(A, A + 2)), "4-byte"), (dict(lse=A + 1), "4-byte"),
    (dict(out_stride=(768, 252, 64)), "16 bytes"), (dict(out_stride=(768, 256, 32)), "overlap"),
    (dict(part_stride=((768, 256, 64), (768, 256, 60))), "16 bytes"),
])
def test_join_refusals(kvx, kw, frag):
    assert kvx.lib().kvevict_attend_join(_join(kvx, **kw), None) == kvx.ERR_INVALID_ARG
    assert frag in kvx.last_error()


def test_join_nothing_to_do(kvx):
    assert kvx.lib().kvevict_attend_join(None, None) == kvx.ERR_INVALID_ARG
    for kw in (dict(batch=0), dict(seq=0), dict(n_heads=0)):
        assert kvx.lib().kvevict_attend_join(_join(kvx, out=0, **kw), None) == kvx.OK


def test_tensors_are_checked(kvx):
    f16 = torch.float16
    q, x = torch.zeros(2, 5, 4, 64, dtype=f16), torch.zeros(2, 5, 2, 64, dtype=f16)
    k = torch.zeros(2, 2, 9, 64, dtype=f16)
    ints = torch.zeros(2, dtype=torch.int32)
    for call in (kvx.attend_prompt, kvx.attend_tree):
        with pytest.raises(ValueError, match="CUDA device"):
            call(q, q, k_new=x, v_new=x)
        with pytest.raises(ValueError, match="together"):
            call(q, q, k_new=x, v_new=x, k=k)
        with pytest.raises(ValueError, match="lens goes with"):
            call(q, q, k_new=x, v_new=x, lens=ints)
        with pytest.raises(ValueError, match="fp16 or bf16"):
            call(q.float(), q, k_new=x, v_new=x)
        with pytest.raises(ValueError, match="scale"):
            call(q, q, k_new=x, v_new=x, scale=0.0)
        with pytest.raises(ValueError, match="scale"):
            call(q, q, k_new=x, v_new=x, scale=10**400)
        with pytest.raises(ValueError, match="dimensions"):
            call(q, q, k_new=x[0], v_new=x)
        with pytest.raises(ValueError, match="shape"):
            call(q[0, 0], q, k_new=x, v_new=x)
    with pytest.raises(ValueError, match="shape"):
        kvx.attend_tree(q[0], q[0], k_new=x[0], v_new=x[0])
    with pytest.raises(ValueError, match="starts goes with"):
        kvx.attend_prompt(q, q, k_new=x, v_new=x, starts=ints)
    with pytest.raises(ValueError, match="new_lens goes with"):
        kvx.attend_prompt(q[0], q[0], k_new=x[0], v_new=x[0], new_lens=ints)
    with pytest.raises(ValueError, match="batch \\+ 1"):
        kvx.attend_prompt(q[0], q[0], k_new=x[0], v_new=x[0], starts=ints[:0])
    with pytest.raises(ValueError, match="1 to 8"):
        kvx.attend_join(q, [])
    with pytest.raises(ValueError, match="CUDA device"):
        kvx.attend_join(q, [(q, q[..., 0].float())])
    with pytest.raises(ValueError, match="shape"):
        kvx.attend_join(q[0, 0], [])
    with pytest.raises(ValueError, match="fp16 or bf16"):
        kvx.attend_join(q.float(), [(q, q)])
