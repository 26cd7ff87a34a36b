"""How near the balance loss's gradient has to come to fp64, also where its type holds it as a subnormal (test
infrastructure; tests/test_gpu_balance.py has the reference and where 2^-17 of `size` comes from)."""
import torch

P = 2.0 ** -18


def tolerance(grad, size, dtype):
    """Before its rounding the gradient is off by 2 P of size (p (|c - mean| + sum |c - mean| p), scaled); the
    rounding takes half a step: eps / 2 of the value, or below the least normal number of the type half of
    the step that all its subnormals have, tiny eps / 2. 1.01: the roundings' own products."""
    info = torch.finfo(dtype)
    near = 2 * P * size
    return near + 1.01 * torch.maximum(info.eps / 2 * (grad.abs() + near), torch.full_like(grad, info.tiny * info.eps / 2))


def problem(T, S, k, seed, dtype, device):
    g = torch.Generator(device).manual_seed(seed)
    like = dict(generator=g, device=device)
    scores = (torch.randn((T, S), **like) * 2 + torch.randn((1, S), **like)).to(dtype)
    ids = torch.topk(scores.float(), k, dim=1).indices.int()
    return scores, ids, torch.rand(T, **like) > 0.3


# Batches whose gradient lies in fp16's subnormals for a dloss of 1.7 (6e-8 to 6.1e-5), wholly or in part
LARGE = [(4097, 384, 8), (5000, 130, 16), (70000, 9, 2)]
