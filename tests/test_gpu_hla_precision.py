"""How exactly the head-decay attention weighs its tokens, on inputs whose sums cancel.

Documented: 16-bit products carry at least 16 significant bits of every inexact operand.  q and k are
positive, so no score cancels; v alternates in sign from token to token, so that an output is a small
rest of large terms and its own rounding does not hide theirs.  With A the sum of the terms'
magnitudes, an output is off by at most

    tokens of its block: 2^-17 A (two terms of P) + 2^-18 A (64 products added in fp32: 64 2^-24)
                         + 2^-20 A (the weights: some ten roundings and exponentials)   < 2^-16 A
    the state before:    the same, with a second 2^-17 for the terms of the decayed values  < 2^-15 A

and half a step of its type (of its smallest normal number for smaller ones).  fp32 (CUDA cores): the same bounds hold with room.
"""
import math

import pytest
import torch

from linear_vision_backbone_b200 import binding, build

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    build.build()
    binding.load()


def decays(pattern, T, H):
    """Log-decays: slow ones, and strong ones in between."""
    gen = torch.Generator().manual_seed(5)
    g = -0.03 * torch.rand(T, H, generator=gen)
    t = torch.arange(T)
    if pattern.startswith("every "):
        g[t % int(pattern[6:]) == 0] = -float("inf")
    elif pattern == "a quarter":
        g[torch.rand(T, H, generator=gen) < 0.25] = -20.0
    elif pattern == "half":
        g[t % 128 < 64] = -110.0
    elif pattern == "one in 32":
        g[t % 32 == 1] = -110.0
    elif pattern == "strong and slow heads":
        g[:, ::2] *= 300.0
    return g


@pytest.mark.parametrize("pattern", ["every 3", "every 4", "every 8", "every 37", "a quarter", "half", "one in 32",
                                     "strong and slow heads", "slow"])
@pytest.mark.parametrize("dtype,dk,dv", [("f16", 64, 64), ("bf16", 64, 64), ("f16", 128, 128), ("bf16", 128, 128),
                                         ("f32", 64, 64)])
def test_weights_between_strong_decays(pattern, dtype, dk, dv):
    T, H = 640, 4
    dt = DT[dtype]
    gen = torch.Generator().manual_seed(dk)
    u = lambda *s: torch.rand(*s, generator=gen) + 0.25  # noqa: E731
    q, k = u(T, H, dk).to(dt), u(T, H, dk).to(dt)
    k[:] = k[:1]                                             # equal scores in a row: the terms cancel
    v = (u(1, H, dv).expand(T, H, dv) * (1.0 - 2.0 * (torch.arange(T) % 2))[:, None, None]).to(dt)
    g = decays(pattern, T, H)
    out = binding.hla_fwd(q.cuda(), k.cuda(), v.cuda(), g.cuda()).double().cpu()
    assert binding.device_status()[0] == 0
    q, k, v = (t.double() for t in (q, k, v))
    g = g.double().clamp(min=-110.0)
    # the weight of token j at token i from the sum of what lies between, in 64 bits
    G = g.cumsum(0)
    D = (G[:, None] - G[None]).permute(2, 0, 1)
    D = torch.where(torch.ones(T, T).tril().bool(), D, -math.inf).exp()
    P = torch.einsum("ihd,jhd->hij", q, k) * D
    ref = torch.einsum("hij,jhe->ihe", P, v)
    block = torch.arange(T) // 128
    near = block[:, None] == block[None]
    a_in = torch.einsum("hij,jhe->ihe", P * near, v.abs())
    a_out = torch.einsum("hij,jhe->ihe", P * ~near, v.abs())
    info = torch.finfo(dt)
    bound = 2 ** -16 * a_in + 2 ** -15 * a_out + info.eps / 2 * ref.abs().clamp(min=info.smallest_normal)
    worst = ((out - ref).abs() / bound).max().item()
    assert worst <= 1.0, worst
