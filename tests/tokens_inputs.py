"""Inputs for tests of attention with several query tokens a sequence. Test infrastructure."""
import torch


def normal(gen, *shape, dtype=torch.float16, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def make(B, S, N, H, D, n=0, dtype=torch.float16, seed=0, packed=False, spread=1.5):
    """Queries and the call's keys and values: a batch [B, S, ..] or S tokens in all, packed."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    room = (S,) if packed else (B, S)
    args = dict(k_new=normal(gen, *room, H, D, dtype=dtype), v_new=normal(gen, *room, H, D, dtype=dtype))
    if n:
        args.update(k=normal(gen, B, H, n, D, dtype=dtype), v=normal(gen, B, H, n, D, dtype=dtype))
    return normal(gen, *room, N * H, D, dtype=dtype, scale=spread), args


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def trees(B, T, seed=0):
    """Parents [B, T]: each token continues one of those before it, or the sequence."""
    gen = torch.Generator().manual_seed(seed)
    rows = [[int(torch.randint(-1, i, (1,), generator=gen)) if i else -1 for i in range(T)] for _ in range(B)]
    return torch.tensor(rows, dtype=torch.int32, device="cuda")
