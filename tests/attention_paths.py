"""Inputs for attention tests, and which kernel takes a call's shared rows. Test infrastructure."""
import ctypes

import torch


def make(B, N, H, D, n=0, P=0, new=False, dtype=torch.float16, seed=0, spread=1.5):
    """Queries [B, N * H, D] and the rows of a call, normal with the seed."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def r(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)
    rows = {}
    if n:
        rows.update(k=r(B, H, n, D), v=r(B, H, n, D))
    if new:
        rows.update(k_new=r(B, H, D), v_new=r(B, H, D))
    if P:
        rows.update(prefix_k=r(H, P, D), prefix_v=r(H, P, D))
    return r(B, N * H, D, scale=spread), rows


def _need(kvx, args):
    need = ctypes.c_size_t(0)
    assert kvx.lib().kvevict_attend_workspace(args, 0, ctypes.addressof(need)) == kvx.OK
    return need.value


def _description(kvx, q, k=None, v=None, lens=None, k_new=None, v_new=None, prefix_k=None, prefix_v=None, prefix_lens=None):
    return kvx._attention(q, torch.empty_like(q), k, v, lens, k_new, v_new, prefix_k, prefix_v, prefix_lens, None, None, None,
                          None)[0]


def workspace(kvx, q, **rows):
    """Bytes of workspace that the call needs."""
    return _need(kvx, _description(kvx, q, **rows))


def prefix_kernel(kvx, q, **rows):
    """Whether the tensor-core kernel takes the shared rows: its parts need another workspace than the row kernel alone,
    which takes the same call where the shared rows have strides of 0, as TMA cannot describe them."""
    args = _description(kvx, q, **rows)
    fields = list(kvx._ATTENTION.unpack(args))
    fields[-5:-1] = [0] * 4                      # the strides of prefix_k and prefix_v
    return _need(kvx, args) != _need(kvx, kvx._ATTENTION.pack(*fields))
