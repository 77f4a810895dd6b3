"""GB300-native cumulative proxy-attention KV-cache eviction.

H2O-adapted, Keyformer-adapted (frozen Gumbel regulariser, annealed
temperature) and PyramidKV-adapted (per-layer budget taper) eviction as one
fused sm_103a decode step, plus tensor-core prompt scoring. This module is the
thin Python face of the C ABI in ``include/kvevict.h``: it only marshals
arguments (tensor pointers, sizes, the current CUDA stream) into
``libkvevict.so``. Every step of the method runs in the library's kernels;
there is no CPU or PyTorch fallback, and importing fails loudly when the
library has not been built.
"""
from __future__ import annotations

import ctypes
import os
import struct

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvevict.so")

OK, ERR_INVALID_ARG, ERR_BAD_STATE, ERR_CUDA, ERR_OOM, ERR_DEVICE_CHECK, ERR_WORKSPACE = 0, -1, -2, -3, -4, -5, -6
SCORE_CUMULATIVE, SCORE_CURRENT = 0, 1
PREFILL_BULK, PREFILL_SEQUENTIAL = 0, 1
DTYPE_FP16, DTYPE_BF16, DTYPE_FP32 = 0, 1, 2
DECODE_AUTO, DECODE_STREAM, DECODE_RESIDENT = 0, 1, 2
MAX_LAYERS = 256
MAX_PREFILL = 16384
MAX_TREE, MAX_JOIN = 64, 8

i32, i64, u64, f32, f64, P = (ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_float,
                              ctypes.c_double, ctypes.c_void_p)


class Config(ctypes.Structure):
    """Mirror of ``kvevict_config``."""
    _fields_ = [("batch", i32), ("n_layers", i32), ("n_kv_heads", i32), ("head_dim", i32),
                ("avg_budget", i32), ("pyramid_beta", f64), ("layer_budgets", P), ("n_sink", i32),
                ("tau_init", f32), ("tau_end", f32), ("anneal_steps", i32), ("rope_theta", f64),
                ("seed", u64), ("max_prefill", i32), ("recent", i32), ("score_mode", i32),
                ("prefill_mode", i32), ("with_values", i32), ("decode_kernel", i32)]


class KVEvictError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"kvevict error {code}: {msg}")
        self.code = code


_lib = None

# every symbol the header declares, with its ctypes signature
SIGNATURES = {
    "kvevict_budgets": (ctypes.c_int, [i32, i32, i32, f64, P]),
    "kvevict_create": (ctypes.c_int, [P, P, P]),
    "kvevict_destroy": (ctypes.c_int, [P]),
    "kvevict_reset": (ctypes.c_int, [P, P]),
    "kvevict_test_stall_next_step": (ctypes.c_int, [P]),
    "kvevict_prefill": (ctypes.c_int, [P, P, i32, P]),
    "kvevict_prefill_ex": (ctypes.c_int, [P, P, i32, P, P]),
    "kvevict_prefill_kv": (ctypes.c_int, [P, P, P, i32, P, P]),
    "kvevict_step_kv": (ctypes.c_int, [P, P, P, P, P]),
    "kvevict_decode_kv": (ctypes.c_int, [P, P, P, i32, P, P]),
    "kvevict_read_values": (ctypes.c_int, [P, i32, i32, i32, P, P, P]),
    "kvevict_step": (ctypes.c_int, [P, P, P, P]),
    "kvevict_decode": (ctypes.c_int, [P, P, i32, P, P]),
    "kvevict_run_host": (ctypes.c_int, [P, P, i32, P, i32, P, P]),
    "kvevict_read_state": (ctypes.c_int, [P, i32, i32, i32, P, P, P, P, P, P]),
    "kvevict_check": (ctypes.c_int, [P, P]),
    "kvevict_flush": (ctypes.c_int, [P, P]),
    "kvevict_next_pos": (ctypes.c_int, [P, P]),
    "kvevict_layer_budget": (ctypes.c_int, [P, i32, P]),
    "kvevict_decode_kernel_for": (ctypes.c_int, [P, i32, P]),
    "kvevict_layer_stats": (ctypes.c_int, [P, i32, P, P, P, P]),
    "kvevict_device_bytes": (ctypes.c_int, [P, P]),
    "kvevict_state_bytes": (ctypes.c_int, [P, P]),
    "kvevict_save_state": (ctypes.c_int, [P, P, ctypes.c_size_t, P]),
    "kvevict_load_state": (ctypes.c_int, [P, P, ctypes.c_size_t, P]),
    "kvevict_last_error": (ctypes.c_char_p, []),
    "kvevict_prefill_scores_noalloc": (ctypes.c_int, [P, i32, i32, i32, P, P]),
    "kvevict_qk_norm_rope": (ctypes.c_int, [P, P]),
    "kvevict_attend": (ctypes.c_int, [P, P]),
    "kvevict_attend_workspace": (ctypes.c_int, [P, i32, P]),
    "kvevict_test_without_prefix_kernel": (ctypes.c_int, [i32]),
    "kvevict_attend_cache": (ctypes.c_int, [P, i32, P, P]),
    "kvevict_attend_prompt": (ctypes.c_int, [P, P]),
    "kvevict_attend_tree": (ctypes.c_int, [P, P]),
    "kvevict_attend_tree_cache": (ctypes.c_int, [P, i32, P, P]),
    "kvevict_attend_tokens_workspace": (ctypes.c_int, [P, i32, P]),
    "kvevict_attend_join": (ctypes.c_int, [P, P]),
    "kvevict_test_without_few_kernel": (ctypes.c_int, [i32]),
    "kvevict_test_without_tokens_kernel": (ctypes.c_int, [i32]),
}


def lib() -> ctypes.CDLL:
    """Load ``libkvevict.so`` (built in-tree by ``__graft_entry__.build()``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build the CUDA library first "
                              "(python -c 'import __graft_entry__ as g; g.build()')")
        found = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(found, name)
            fn.restype = res
            fn.argtypes = args
        _lib = found                  # whole: other threads may be here, too
    return _lib


def _check(rc: int):
    if rc != OK:
        raise KVEvictError(rc, lib().kvevict_last_error().decode())


def last_error() -> str:
    return lib().kvevict_last_error().decode()


def budgets(n_layers: int, avg_budget: int, n_sink: int, beta: float) -> list[int]:
    """Per-layer budget taper computed by the library (host only)."""
    out = (i32 * max(1, n_layers))()
    _check(lib().kvevict_budgets(n_layers, avg_budget, n_sink, beta, ctypes.addressof(out)))
    return list(out)[:n_layers]


def prefill_scores_noalloc(keys, colsum, stream=None):
    """Causal column sums of prompts with no device allocation.

    keys: device fp16 [heads, S, D]; colsum: device float32 [heads, S] (output).
    For callers that cannot allocate device memory; see the C declaration of
    kvevict_prefill_scores_noalloc for the size limit and sharing rules.
    """
    heads, S, D = (int(x) for x in keys.shape)
    assert tuple(colsum.shape) == (heads, S)
    _check(lib().kvevict_prefill_scores_noalloc(_ptr(keys), heads, S, D, _ptr(colsum),
                                                _stream(stream)))


# ``kvevict_qk``, ``kvevict_attention``, ``kvevict_tokens`` and ``kvevict_join`` of include/kvevict.h, field by field.
_QK = struct.Struct("=8i f i d q 7Q 12q")
_ATTENTION = struct.Struct("=8i f i 12Q 18q Q")
_TOKENS = struct.Struct("=8i f i 12Q 19q Q")
_JOIN = struct.Struct("=8i 18Q 27q")
_U64 = struct.Struct("=Q")
_WORKSPACE_AT, _WORKSPACE_BYTES_AT = 40 + 11 * 8, _ATTENTION.size - 8    # offsets in kvevict_attention
_TOKENS_BYTES_AT = _TOKENS.size - 8      # in kvevict_tokens, whose workspace is at the same offset
_NO3, _NO4 = (0, 0, 0), (0, 0, 0, 0)     # strides of tensors that are not there
_NO_PARTS = [(0,) * (MAX_JOIN - i) for i in range(MAX_JOIN + 1)]   # of a join's parts behind the last of i


def _torch():
    """torch, with its types' codes (imported on first use: the library itself does not need it)."""
    global _IN, _OUT, _loaded
    if _loaded is not None:
        return _loaded
    import torch
    _IN = {torch.float16: DTYPE_FP16, torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_FP32}
    _OUT = {torch.float16: DTYPE_FP16, torch.bfloat16: DTYPE_BF16}
    _loaded = torch                   # last: other threads may be here, too
    return torch


_IN, _OUT, _loaded = {}, {}, None


def _wrong(name, t, shape, dtype, device):
    if t.shape != shape:
        return ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    if t.dtype is not dtype:
        return ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return ValueError(f"{name} must be on the current CUDA device, got {t.device}" if not t.is_cuda or t.get_device() != device
                      else f"{name} must be contiguous" if t.stride()[-1] == 1
                      else f"the last dimension of {name} must be contiguous")


def _strided(name, t, shape, dtype, device):
    """Pointer and strides of one call's tensor, after the checks."""
    if t is None:
        raise ValueError(f"{name} must be given")
    stride = t.stride()
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device or stride[-1] != 1:
        raise _wrong(name, t, shape, dtype, device)
    return t.data_ptr(), stride


def _dense(name, t, shape, dtype, device):
    """Pointer of a contiguous tensor, after the checks; null for None."""
    if t is None:
        return 0
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        raise _wrong(name, t, shape, dtype, device)
    return t.data_ptr()


def _place(torch, t, stream):
    """The current device and the stream of a call whose first tensor is t."""
    if not t.is_cuda:
        raise ValueError(f"tensors must be on the current CUDA device, got {t.device}")
    device = torch.cuda.current_device()
    if stream is None:
        return device, torch._C._cuda_getCurrentRawStream(device)
    return device, _stream(stream)


def qk_norm_rope(q, k, q_out, k_out, *, rope_theta, q_weight=None, k_weight=None, eps=1e-6, positions=None, pos0=0,
                 stream=None):
    """RMS norm of every query and key head and the rotation to the token's position, in one pass.

    q [B, S, G, D], k [B, S, H, D]: fp16, bf16 or fp32 (views of a fused projection are fine). q_out, k_out: their
    shapes in fp16 or bf16, in any layout with a contiguous last dimension; ``prompt_keys[:, l].transpose(1, 2)``
    writes layer l of what ``KVEvict.prefill`` takes, ``k_new[:, l, None]`` of what ``KVEvict.step`` takes. q_weight,
    k_weight [D] or None (no norm). positions: int32 [B, S], else token s is at pos0 + s, in 32 bits too. Either of q and k may be
    None with its output. Errors: ValueError, KVEvictError.
    """
    torch = _torch()
    if q is None and k is None:
        raise ValueError("q or k must be given")
    if (q is None) != (q_out is None) or (k is None) != (k_out is None):
        raise ValueError("q goes with q_out and k with k_out")
    some, some_out = (q, q_out) if q is not None else (k, k_out)
    if some.dim() != 4 or (k is not None and k.dim() != 4):
        raise ValueError("q and k must have shape [batch, seq, heads, head_dim]")
    if not 2.0**-1022 <= rope_theta <= 1.7e308:
        raise ValueError("rope_theta must be > 0, normal and finite")
    if not (eps == 0 or 2.0**-149 <= eps <= 3.4e38):         # (below, it would round to 0)
        raise ValueError("eps must be 0, or from 2^-149 and finite")
    if not -1 << 63 <= pos0 < 1 << 63:
        raise ValueError("pos0 must fit 64 bits")
    B, S, _, D = some.shape
    if positions is None and not -1 << 31 <= pos0 <= (1 << 31) - max(S, 1):
        raise ValueError("pos0 and the positions after it must fit 32 bits")
    kind, kind_out = some.dtype, some_out.dtype
    if kind not in _IN or kind_out not in _OUT:
        raise ValueError("q and k must be fp16, bf16 or fp32, q_out and k_out fp16 or bf16")
    device, s = _place(torch, some, stream)
    G = H = pq = pqo = pk = pko = 0
    sq = sqo = sk = sko = _NO4
    if q is not None:
        G = q.shape[2]
        pq, sq = _strided("q", q, (B, S, G, D), kind, device)
        pqo, sqo = _strided("q_out", q_out, (B, S, G, D), kind_out, device)
    if k is not None:
        H = k.shape[2]
        pk, sk = _strided("k", k, (B, S, H, D), kind, device)
        pko, sko = _strided("k_out", k_out, (B, S, H, D), kind_out, device)
    wt = None if q_weight is None and k_weight is None else (q_weight if q_weight is not None else k_weight).dtype
    if wt is not None and wt not in _IN:
        raise ValueError("q_weight and k_weight must be fp16, bf16 or fp32")
    args = _QK.pack(_IN[kind], _OUT[kind_out], _IN[wt] if wt is not None else DTYPE_FP32, B, S, G, H, D, eps, 0, rope_theta,
                    pos0, pq, pk, pqo, pko, _dense("q_weight", q_weight, (D,), wt, device),
                    _dense("k_weight", k_weight, (D,), wt, device),
                    _dense("positions", positions, (B, S), torch.int32, device), *sq[:3], *sk[:3], *sqo[:3], *sko[:3])
    rc = lib().kvevict_qk_norm_rope(args, s)
    if rc:
        _check(rc)


def _attention(q, out, k, v, lens, k_new, v_new, prefix_k, prefix_v, prefix_lens, lse, scale, stream, kv_heads):
    """The ``kvevict_attention`` of a call and its stream."""
    torch = _torch()
    if q.dim() != 3:
        raise ValueError("q must have shape [batch, heads, head_dim]")
    B, G, D = q.shape
    kind = q.dtype
    if kind not in _OUT:
        raise ValueError("q must be fp16 or bf16")
    if (k is None) != (v is None) or (k_new is None) != (v_new is None) or (prefix_k is None) != (prefix_v is None):
        raise ValueError("k and v, k_new and v_new, prefix_k and prefix_v go together")
    if lens is not None and k is None or prefix_lens is not None and prefix_k is None:
        raise ValueError("lens goes with k and prefix_lens with prefix_k")
    if scale is not None and not 2.0**-126 <= scale <= 2.0**127:
        raise ValueError("scale must be from 2^-126 to 2^127")
    H, n, prefix = kv_heads, 0, 0
    if k is not None:
        if k.dim() != 4:
            raise ValueError("k must have shape [batch, kv_heads, rows, head_dim]")
        _, H, n, _ = k.shape
    if prefix_k is not None:
        if prefix_k.dim() != 3:
            raise ValueError("prefix_k must have shape [kv_heads, rows, head_dim]")
        prefix = prefix_k.shape[1]
        if H is None:
            H = prefix_k.shape[0]
    if H is None:
        if k_new is None:
            raise ValueError("nothing to attend to: k, k_new or prefix_k must be given")
        if k_new.dim() != 3:
            raise ValueError("k_new must have shape [batch, kv_heads, head_dim]")
        H = k_new.shape[1]
    device, s = _place(torch, q, stream)
    pk = pv = pkn = pvn = ppk = ppv = 0
    sk = sv = _NO4
    skn = svn = spk = spv = _NO3
    pq, sq = _strided("q", q, (B, G, D), kind, device)
    po, so = _strided("out", out, (B, G, D), kind, device)
    if n:
        pk, sk = _strided("k", k, (B, H, n, D), kind, device)
        pv, sv = _strided("v", v, (B, H, n, D), kind, device)
    if k_new is not None:
        pkn, skn = _strided("k_new", k_new, (B, H, D), kind, device)
        pvn, svn = _strided("v_new", v_new, (B, H, D), kind, device)
    if prefix:
        ppk, spk = _strided("prefix_k", prefix_k, (H, prefix, D), kind, device)
        ppv, spv = _strided("prefix_v", prefix_v, (H, prefix, D), kind, device)
    return _ATTENTION.pack(
        _OUT[kind], B, G, H, D, n, prefix, 0, scale or 0.0, 0, pq, po, _dense("lse", lse, (B, G), torch.float32, device), pk, pv,
        _dense("lens", lens, (B,), torch.int32, device), pkn, pvn, ppk, ppv,
        _dense("prefix_lens", prefix_lens, (B,), torch.int32, device), 0,
        sq[0], sq[1], so[0], so[1], sk[0], sk[1], sk[2], sv[0], sv[1], sv[2], skn[0], skn[1], svn[0], svn[1], spk[0], spk[1],
        spv[0], spv[1], 0), s


def _with_workspace(args, cache, q, stream, tokens=False):
    """The same call with the workspace it needs, taken from torch's allocator for its stream, and that tensor."""
    torch, need = _torch(), ctypes.c_size_t(0)
    size, end = (lib().kvevict_attend_tokens_workspace, _TOKENS_BYTES_AT) if tokens else \
        (lib().kvevict_attend_workspace, _WORKSPACE_BYTES_AT)
    _check(size(args, cache, ctypes.addressof(need)))
    if stream == torch._C._cuda_getCurrentRawStream(q.get_device()):
        space = torch.empty(need.value, dtype=torch.uint8, device=q.device)
    else:
        with torch.cuda.stream(torch.cuda.ExternalStream(stream or 0)):
            space = torch.empty(need.value, dtype=torch.uint8, device=q.device)
    return b"".join((args[:_WORKSPACE_AT], _U64.pack(space.data_ptr()), args[_WORKSPACE_AT + 8:end],
                     _U64.pack(need.value))), space


def attend(q, out, *, k=None, v=None, lens=None, k_new=None, v_new=None, prefix_k=None, prefix_v=None,
           prefix_lens=None, lse=None, scale=None, stream=None):
    """Attention of one query token a sequence over its own rows, the token's own key and shared rows.

    q, out [B, G, D] fp16 or bf16, everything else of q's type; k, v [B, H, n, D] with lens int32 [B] or None (n);
    k_new, v_new [B, H, D]; prefix_k, prefix_v [H, P, D], read once for the whole batch, with prefix_lens int32 [B] or
    None (P). Query head i reads key head i // (G // H). lse: float32 [B, G] output or None. scale: 2^-126 to 2^127,
    1/sqrt(D) unless given. A sequence with no rows gets out 0 and lse -inf. Any layout with a contiguous last
    dimension and strides of whole 16-byte pieces. Errors: ValueError, KVEvictError.
    """
    args, s = _attention(q, out, k, v, lens, k_new, v_new, prefix_k, prefix_v, prefix_lens, lse, scale, stream, None)
    rc = lib().kvevict_attend(args, s)
    if rc == ERR_WORKSPACE:                 # most calls need none
        args, space = _with_workspace(args, 0, q, s)
        rc = lib().kvevict_attend(args, s)
    if rc:
        _check(rc)


def _tokens(q, out, k_new, v_new, starts, new_lens, parents, k, v, lens, lse, scale, stream, tree):
    """The ``kvevict_tokens`` of a call and its stream."""
    torch = _torch()
    if q is None or out is None or k_new is None or v_new is None:
        raise ValueError("q, out, k_new and v_new must be given")
    shape, own = q.shape, k_new.shape
    packed = len(shape) == 3 and not tree
    if len(shape) != 4 and not packed:
        raise ValueError("q must have shape [batch, tokens, heads, head_dim]" + ("" if tree else " or [tokens, heads, head_dim]"))
    kind = q.dtype
    if kind not in _OUT:
        raise ValueError("q must be fp16 or bf16")
    if (k is None) != (v is None):
        raise ValueError("k and v go together")
    if lens is not None and k is None:
        raise ValueError("lens goes with k")
    if scale is not None and not 2.0**-126 <= scale <= 2.0**127:
        raise ValueError("scale must be from 2^-126 to 2^127")
    if len(own) != len(shape):
        raise ValueError("k_new must have as many dimensions as q")
    H, D, B = own[-2], shape[-1], 1
    if packed:
        if new_lens is not None:
            raise ValueError("new_lens goes with a batch [batch, tokens, heads, head_dim], starts with packed tokens")
        if starts is not None:
            if starts.dim() != 1 or starts.shape[0] < 1:
                raise ValueError("starts must have shape [batch + 1]")
            B = starts.shape[0] - 1
        S, heads, _ = shape
        own = (S, H, D)
    else:
        if starts is not None:
            raise ValueError("starts goes with packed tokens [tokens, heads, head_dim]")
        B, S, heads, _ = shape
        own = (B, S, H, D)
    n = 0
    if k is not None:
        if k.dim() != 4:
            raise ValueError("k must have shape [batch, kv_heads, rows, head_dim]")
        n = k.shape[2]
    device, s = _place(torch, q, stream)
    pq, sq = _strided("q", q, shape, kind, device)
    po, so = _strided("out", out, shape, kind, device)
    pkn, skn = _strided("k_new", k_new, own, kind, device)
    pvn, svn = _strided("v_new", v_new, own, kind, device)
    if packed:
        sq, so, skn, svn = (0, *sq), (0, *so), (0, *skn), (0, *svn)
    pk = pv = pp = tree_stride = pl = pst = pnl = plens = 0
    sk = sv = _NO4
    if n:
        pk, sk = _strided("k", k, (B, H, n, D), kind, device)
        pv, sv = _strided("v", v, (B, H, n, D), kind, device)
    ints = torch.int32
    if parents is not None:
        if parents.dim() == 1:
            parents = parents.expand(B, -1)
        if parents.shape[-1:] == (1,):                          # (a single token's stride may be anything)
            parents = parents.as_strided((parents.shape[0], 1), (parents.stride(0), 1))
        pp, st = _strided("parents", parents, (B, S), ints, device)
        tree_stride = st[0]
    if lse is not None:
        pl = _dense("lse", lse, shape[:-1], torch.float32, device)
    if starts is not None:
        pst = _dense("starts", starts, (B + 1,), ints, device)
    if new_lens is not None:
        pnl = _dense("new_lens", new_lens, (B,), ints, device)
    if lens is not None:
        plens = _dense("lens", lens, (B,), ints, device)
    return _TOKENS.pack(
        _OUT[kind], B, S, heads, H, D, n, 0, scale or 0.0, 0, pq, po, pl, pkn, pvn, pst, pnl, pp, pk, pv, plens, 0,
        sq[0], sq[1], sq[2], so[0], so[1], so[2], skn[0], skn[1], skn[2], svn[0], svn[1], svn[2], sk[0], sk[1], sk[2],
        sv[0], sv[1], sv[2], tree_stride, 0), s


def _call_tokens(call, cache, q, args, stream):
    """Makes a call that takes a ``kvevict_tokens``, with a workspace where it needs one."""
    rc = call(args, stream)
    if rc == ERR_WORKSPACE:
        args, space = _with_workspace(args, cache, q, stream, True)
        rc = call(args, stream)
    if rc:
        _check(rc)


def attend_prompt(q, out, *, k_new, v_new, starts=None, new_lens=None, k=None, v=None, lens=None, lse=None, scale=None,
                  stream=None):
    """Causal attention of whole prompts: every token over its sequence's own rows and its tokens up to itself.

    A batch: q, out [B, S, G, D], k_new, v_new [B, S, H, D] with new_lens int32 [B] or None (S). Packed: q, out [T, G, D],
    k_new, v_new [T, H, D] with starts int32 [B + 1] (sequence b: starts[b] .. starts[b + 1] - 1; None: one sequence). fp16 or
    bf16. k, v [B, H, n, D] with lens int32 [B] or None (n): rows before the tokens, an earlier chunk's. Query head i
    reads key head i // (G // H). lse: float32, q's shape without D, or None. Tokens behind a sequence's last are not
    written. ``prompt_keys[:, l].transpose(1, 2)`` reads layer l of what ``KVEvict.prefill`` takes. Layouts and
    scale as in ``attend``. Errors: ValueError, KVEvictError.
    """
    args, s = _tokens(q, out, k_new, v_new, starts, new_lens, None, k, v, lens, lse, scale, stream, False)
    _call_tokens(lib().kvevict_attend_prompt, 0, q, args, s)


def attend_tree(q, out, *, k_new, v_new, parents=None, new_lens=None, k=None, v=None, lens=None, lse=None, scale=None,
                stream=None):
    """Attention of a tree of drafted tokens per sequence: each over the sequence's own rows, itself and its ancestors.

    q, out [B, T, G, D], k_new, v_new [B, T, H, D], T at most MAX_TREE, with new_lens int32 [B] or None (T). parents:
    int32 [B, T] or [T] (the same tree for all), the token that each one continues, always one before it, or -1
    where it continues the sequence itself; None: a chain. Everything else as in ``attend_prompt``.
    """
    args, s = _tokens(q, out, k_new, v_new, None, new_lens, parents, k, v, lens, lse, scale, stream, True)
    _call_tokens(lib().kvevict_attend_tree, 0, q, args, s)


def attend_join(out, parts, *, lse=None, stream=None):
    """Joins parts of an attention over disjoint rows (a shared prefix's and the rest) by their log sums.

    parts: 1 to MAX_JOIN pairs (part, its lse); out and every part [B, S, G, D] or [T, G, D], fp16 or bf16; lse, theirs and
    the output: float32, that shape without D. out may be one of the parts, and lse its lse. A part whose lse is -inf
    takes no weight. Layouts as in ``attend``. Errors: ValueError, KVEvictError.
    """
    torch = _torch()
    if out is None or parts is None:
        raise ValueError("out and parts must be given")
    if out.dim() not in (3, 4):
        raise ValueError("out must have shape [batch, tokens, heads, head_dim] or [tokens, heads, head_dim]")
    kind, shape = out.dtype, out.shape
    if kind not in _OUT:
        raise ValueError("out must be fp16 or bf16")
    parts = list(parts)
    if not 1 <= len(parts) <= MAX_JOIN:
        raise ValueError(f"1 to {MAX_JOIN} parts can be joined, got {len(parts)}")
    device, s = _place(torch, out, stream)
    flat = len(shape) == 3
    rows, count = shape[:-1], len(parts)
    pointers, lses, strides = (), (), ()
    for i, (part, part_lse) in enumerate(parts):
        if part is None or part_lse is None:
            raise ValueError(f"part {i} must be given, with its lse")
        at, st = _strided(f"part {i}", part, shape, kind, device)
        pointers += at,
        lses += _dense(f"lse of part {i}", part_lse, rows, torch.float32, device),
        strides += (0, st[0], st[1]) if flat else st[:3]
    none = _NO_PARTS[count]
    to, st = _strided("out", out, shape, kind, device)
    B, S, G, D = (1, *shape) if flat else shape
    args = _JOIN.pack(_OUT[kind], B, S, G, D, count, 0, 0, *pointers, *none, *lses, *none, to,
                      _dense("lse", lse, rows, torch.float32, device), *strides, *none, *none, *none,
                      *((0, st[0], st[1]) if flat else st[:3]))
    rc = lib().kvevict_attend_join(args, s)
    if rc:
        _check(rc)


def _ptr(t) -> int:
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        assert t.flags["C_CONTIGUOUS"]
        return t.ctypes.data
    assert t.is_contiguous(), "tensor must be contiguous"
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    import torch
    return torch.cuda.current_stream().cuda_stream


class KVEvict:
    """One handle: a device-resident eviction state for B x L x H cache rows."""

    def __init__(self, *, batch: int, n_layers: int, n_kv_heads: int, head_dim: int,
                 avg_budget: int = 512, pyramid_beta: float = 1.0, layer_budgets=None,
                 n_sink: int = 4, tau_init: float = 0.0, tau_end: float = 0.0,
                 anneal_steps: int = 0, rope_theta: float = 10000.0, seed: int = 0,
                 max_prefill: int = 0, recent: int = 0, score_mode: int = SCORE_CUMULATIVE,
                 prefill_mode: int = PREFILL_BULK, with_values: bool = False,
                 decode_kernel: int = DECODE_AUTO, stream=None):
        self._lb = None
        if layer_budgets is not None:
            self._lb = (i32 * n_layers)(*layer_budgets)
        self.cfg = Config(batch, n_layers, n_kv_heads, head_dim, avg_budget, pyramid_beta,
                          ctypes.addressof(self._lb) if self._lb is not None else None, n_sink,
                          tau_init, tau_end, anneal_steps, rope_theta, seed & (2 ** 64 - 1),
                          max_prefill, recent, score_mode, prefill_mode, int(bool(with_values)),
                          decode_kernel)
        self._h = P()
        _check(lib().kvevict_create(ctypes.addressof(self.cfg), _stream(stream),
                                    ctypes.addressof(self._h)))
        self.B, self.L, self.H, self.D = batch, n_layers, n_kv_heads, head_dim
        self.with_values = bool(with_values)
        self.budgets = [self.layer_budget(l) for l in range(n_layers)]

    # ------------------------------------------------------------------ lifecycle
    def close(self):
        if self._h:
            lib().kvevict_destroy(self._h)
            self._h = P()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def reset(self, stream=None):
        _check(lib().kvevict_reset(self._h, _stream(stream)))

    # ------------------------------------------------------------------ the path
    def prefill(self, keys, evicted=None, stream=None, values=None):
        """keys (values): device fp16 [B, L, H, S, D]; evicted: device int32 [S, B, L, H] or None."""
        S = int(keys.shape[3]) if keys is not None else 0
        if self.with_values:
            _check(lib().kvevict_prefill_kv(self._h, _ptr(keys), _ptr(values), S, _ptr(evicted),
                                            _stream(stream)))
        else:
            _check(lib().kvevict_prefill_ex(self._h, _ptr(keys), S, _ptr(evicted), _stream(stream)))

    def step(self, k_new, evicted=None, stream=None, v_new=None):
        """k_new (v_new): device fp16 [B, L, H, D]; evicted: device int32 [B, L, H] or None."""
        if self.with_values:
            _check(lib().kvevict_step_kv(self._h, _ptr(k_new), _ptr(v_new), _ptr(evicted),
                                         _stream(stream)))
        else:
            _check(lib().kvevict_step(self._h, _ptr(k_new), _ptr(evicted), _stream(stream)))

    def decode(self, keys, evicted=None, stream=None, values=None):
        """keys (values): device fp16 [T, B, L, H, D]; evicted: device int32 [T, B, L, H] or None."""
        if self.with_values:
            _check(lib().kvevict_decode_kv(self._h, _ptr(keys), _ptr(values), int(keys.shape[0]),
                                           _ptr(evicted), _stream(stream)))
        else:
            _check(lib().kvevict_decode(self._h, _ptr(keys), int(keys.shape[0]), _ptr(evicted),
                                        _stream(stream)))

    def attend(self, l: int, q, out, *, k_new=None, v_new=None, prefix_k=None, prefix_v=None, prefix_lens=None, lse=None,
               scale=None, stream=None):
        """``attend`` with layer l's kept keys and values as the own rows (a value-carrying handle; fp16).

        q, out [B, G, D]; k_new, v_new [B, H, D]: the token's own, before the step that inserts them, rotated at
        position next_pos, behind P shared rows at P + next_pos (and the prompt's keys from P on). Rows are as
        ``read_state`` and ``read_values`` give them; the handle is not changed. A captured call keeps the row count
        of its capture.
        """
        args, s = _attention(q, out, None, None, None, k_new, v_new, prefix_k, prefix_v, prefix_lens, lse, scale, stream,
                             self.H)
        rc = lib().kvevict_attend_cache(self._h, l, args, s)
        if rc == ERR_WORKSPACE:
            args, space = _with_workspace(args, 1, q, s)
            rc = lib().kvevict_attend_cache(self._h, l, args, s)
        _check(rc)

    def attend_tree(self, l: int, q, out, *, k_new, v_new, parents=None, new_lens=None, lse=None, scale=None, stream=None):
        """``attend_tree`` with layer l's kept keys and values as the own rows (a value-carrying handle; fp16).

        A token at depth d of its tree (0: it continues the sequence) is rotated at position next_pos + d. Rows are as
        ``read_state`` and ``read_values`` give them; the handle is not changed: the tokens that are accepted go in by
        ``step`` or ``decode``. A captured call keeps the row count of its capture.
        """
        args, s = _tokens(q, out, k_new, v_new, None, new_lens, parents, None, None, None, lse, scale, stream, True)
        _call_tokens(lambda d, at: lib().kvevict_attend_tree_cache(self._h, l, d, at), 1, q, args, s)

    def run_host(self, prefill_keys, decode_keys, evicted=None, stream=None):
        """End to end from host memory (pinned tensors or numpy uint16 arrays)."""
        S = int(prefill_keys.shape[3]) if prefill_keys is not None else 0
        T = int(decode_keys.shape[0]) if decode_keys is not None else 0
        _check(lib().kvevict_run_host(self._h, _ptr(prefill_keys), S, _ptr(decode_keys), T,
                                      _ptr(evicted), _stream(stream)))

    # ------------------------------------------------------------------ queries
    def read_state(self, b: int, l: int, h: int, stream=None):
        """(keys fp16-bits [n, D], scores f32 [n], gumbel f32 [n], positions i32 [n])."""
        cap = self.budgets[l] + 1 if 0 <= l < self.L else 1  # the library validates indices
        keys = np.zeros((cap, self.D), np.uint16)
        sc = np.zeros(cap, np.float32)
        g = np.zeros(cap, np.float32)
        pos = np.zeros(cap, np.int32)
        n = i32(0)
        _check(lib().kvevict_read_state(self._h, b, l, h, keys.ctypes.data, sc.ctypes.data,
                                        g.ctypes.data, pos.ctypes.data, ctypes.addressof(n),
                                        _stream(stream)))
        k = n.value
        return keys[:k], sc[:k], g[:k], pos[:k]

    def read_values(self, b: int, l: int, h: int, stream=None):
        """Value rows of one cache row, fp16 bits [n, D], in slot order."""
        cap = self.budgets[l] + 1 if 0 <= l < self.L else 1
        vals = np.zeros((cap, self.D), np.uint16)
        n = i32(0)
        _check(lib().kvevict_read_values(self._h, b, l, h, vals.ctypes.data, ctypes.addressof(n),
                                         _stream(stream)))
        return vals[: n.value]

    def flush(self, stream=None):
        """Apply the last step's pending compaction (one kernel launch)."""
        _check(lib().kvevict_flush(self._h, _stream(stream)))

    def test_stall_next_step(self):
        """Test hook: the next decode launch makes one bounded wait run out."""
        _check(lib().kvevict_test_stall_next_step(self._h))

    def check(self, stream=None):
        _check(lib().kvevict_check(self._h, _stream(stream)))

    @property
    def next_pos(self) -> int:
        p = i64(0)
        _check(lib().kvevict_next_pos(self._h, ctypes.addressof(p)))
        return p.value

    def decode_kernel_for(self, T: int) -> int:
        """DECODE_STREAM or DECODE_RESIDENT: the kernel a call of T steps runs."""
        k = i32(0)
        _check(lib().kvevict_decode_kernel_for(self._h, T, ctypes.addressof(k)))
        return k.value

    def layer_budget(self, l: int) -> int:
        b = i32(0)
        _check(lib().kvevict_layer_budget(self._h, l, ctypes.addressof(b)))
        return b.value

    def layer_stats(self, l: int) -> dict:
        """tokens_kept, stored_bytes, full_bytes and compression_ratio of layer l."""
        kept, stored, full, ratio = i32(0), ctypes.c_uint64(0), ctypes.c_uint64(0), ctypes.c_double(0)
        _check(lib().kvevict_layer_stats(self._h, l, ctypes.addressof(kept), ctypes.addressof(stored),
                                         ctypes.addressof(full), ctypes.addressof(ratio)))
        return {"tokens_kept": kept.value, "stored_bytes": stored.value, "full_bytes": full.value,
                "compression_ratio": ratio.value}

    def device_bytes(self) -> int:
        v = ctypes.c_size_t(0)
        _check(lib().kvevict_device_bytes(self._h, ctypes.addressof(v)))
        return v.value

    # ------------------------------------------------------- checkpoint / resume
    def state_bytes(self) -> int:
        v = ctypes.c_size_t(0)
        _check(lib().kvevict_state_bytes(self._h, ctypes.addressof(v)))
        return v.value

    def save_state(self, out=None, stream=None) -> np.ndarray:
        """Snapshot of the cache state as a uint8 host array (or into `out`)."""
        n = self.state_bytes()
        buf = np.empty(n, np.uint8) if out is None else out
        assert buf.dtype == np.uint8 and buf.flags["C_CONTIGUOUS"] and buf.size >= n
        _check(lib().kvevict_save_state(self._h, buf.ctypes.data, buf.size, _stream(stream)))
        return buf

    def load_state(self, snapshot, stream=None):
        """Replace the cache state with a snapshot from save_state."""
        buf = np.ascontiguousarray(snapshot, dtype=np.uint8)
        _check(lib().kvevict_load_state(self._h, buf.ctypes.data, buf.size, _stream(stream)))


def from_workload(wl, stream=None, with_values=False, decode_kernel=DECODE_AUTO) -> KVEvict:
    """Handle for a ``workloads.Workload`` configuration."""
    return KVEvict(batch=wl.batch, n_layers=wl.n_layers, n_kv_heads=wl.n_kv_heads,
                   head_dim=wl.head_dim, avg_budget=wl.avg_budget, pyramid_beta=wl.beta,
                   n_sink=wl.n_sink, tau_init=wl.tau_init, tau_end=wl.tau_end,
                   anneal_steps=wl.anneal_steps, rope_theta=wl.rope_theta, seed=wl.gumbel_seed,
                   max_prefill=wl.prefill, recent=getattr(wl, "recent", 0),
                   score_mode=getattr(wl, "score_mode", SCORE_CUMULATIVE),
                   prefill_mode=getattr(wl, "prefill_mode", PREFILL_BULK),
                   with_values=with_values, decode_kernel=decode_kernel, stream=stream)
