"""Cases of the head-decay attention whose groups walk many blocks of tokens, the plan's
arithmetic (hla.cu, make_plan) and a chunked form in 64 bits, shared by CPU and GPU tests."""
import math
import random

import torch

SMS = 148


def lengths(seed, n, low, high):
    r = random.Random(seed)
    return [r.randint(low, high) for _ in range(n)]


# name: lengths, heads, key heads, dk, dv, type, gated, equal sequences without offsets
STEADY = {
    "f16-64-gated": (lengths(1, 16, 1100, 1500), 16, 4, 64, 64, "f16", True, False),
    "f16-64-plain": (lengths(2, 16, 1100, 1500), 16, 16, 64, 64, "f16", False, False),
    "f16-128-gated": (lengths(3, 16, 1100, 1500), 16, 4, 128, 128, "f16", True, False),
    "f16-128-plain": (lengths(4, 16, 1100, 1500), 16, 4, 128, 128, "f16", False, False),
    "f16-64x128-gated": (lengths(5, 16, 1100, 1500), 16, 4, 64, 128, "f16", True, False),
    "f16-128x64-gated": (lengths(6, 16, 1100, 1500), 16, 4, 128, 64, "f16", True, False),
    "bf16-64-gated": (lengths(7, 16, 1100, 1500), 16, 4, 64, 64, "bf16", True, False),
    "bf16-128-gated": (lengths(8, 16, 1100, 1500), 16, 4, 128, 128, "bf16", True, False),
    "bf16-128-plain": (lengths(9, 16, 1100, 1500), 16, 4, 128, 128, "bf16", False, False),
    "f16-64-equal": ([1408] * 16, 16, 4, 64, 64, "f16", True, True),
    "f16-128-equal": ([1400] * 16, 8, 2, 128, 128, "f16", True, True),
    "bf16-128-equal": ([1400] * 16, 8, 8, 128, 128, "bf16", False, True),
    "f16-64-40": (lengths(10, 38, 0, 900) + [0, 1], 16, 4, 64, 64, "f16", True, False),
    "f16-128-40": (lengths(11, 38, 0, 700) + [0, 1], 16, 8, 128, 128, "f16", True, False),
    "bf16-128-40": (lengths(12, 38, 0, 700) + [1, 0], 16, 8, 128, 128, "bf16", False, False),
    "bf16-64-1030": (lengths(13, 1030, 0, 70), 4, 4, 64, 64, "bf16", True, False),
    "f32-64-40": (lengths(14, 38, 0, 600) + [0, 1], 4, 2, 64, 64, "f32", True, False),
}


def plan(nseq, T, H, dk, dv, dtype, equal, sms=SMS):
    """(groups, cut, workspace bytes) of make_plan."""
    tc = dtype != "f32" and dk >= 64 and dv >= 64
    k_sum, k_extra = (0.35, 4.0) if tc else (0.5, 3.0)
    C = 128 if tc else 16
    slots = sms // (dv // 64) if tc else sms
    longest = -(-(T // nseq if equal else T) // C)
    B = H * (nseq * (longest + 1) if equal else T // C + 2 * nseq)
    items = nseq * H
    share = -(-B // slots) if tc else B / slots
    whole = -(-items // slots) * (longest + 1) if equal else max(share, longest)
    cut = longest > 1 and whole > share * (1 + k_sum) + k_extra
    most = slots if tc else 2 * slots if cut else 4 * slots
    if not cut:
        J = min(items, most)
    elif tc:
        J = -(-B // share)
    else:
        J = min(B, most)
    return J, cut, J * (2 * dk * dv * 4 + 16 + 4) if cut else 0


def longest_walk(lens, H, J, cut, C=128):
    """(most blocks in one group's walk, most blocks in one of its parts)."""
    nb = [-(-n // C) for n in lens]
    line = [(n, h, b) for n in range(len(lens)) for h in range(H) for b in range(nb[n] + 1)]
    B = len(line)
    J = min(J, B)
    most = part = 0
    for j in range(J):
        x0, x1 = (B // J * i + min(i, B % J) for i in (j, j + 1))
        runs = {}
        for n, h, b in line[x0:x1]:
            if cut:
                if b < nb[n]:
                    runs[n, h] = runs.get((n, h), 0) + 1
            elif b == 0:
                runs[n, h] = nb[n]
        most, part = max(most, sum(runs.values())), max(part, max(runs.values(), default=0))
    return most, part


def inputs(case, seed):
    """On the GPU: slow decays, and values that grow and shrink along a sequence."""
    lens, H, Hk, dk, dv, dtype, gated, equal = case
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    n = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    T = sum(lens)
    wave = torch.exp2(5.0 * torch.sin(torch.arange(T, device="cuda") / 130.0))[:, None, None]
    d = {"q": n(T, Hk, dk).to(dt), "k": n(T, Hk, dk).to(dt), "v": (n(T, H, dv) * wave).to(dt),
         "z": n(T, H, dv).to(dt) if gated else None, "w": 1 + 0.2 * n(dv) if gated else None,
         "g": torch.nn.functional.logsigmoid(n(T, H) + 2.0) / 64.0, "S": n(len(lens), H, dk, dv) * 4,
         "lens": lens, "scale": dk ** -0.5}
    d["cu"] = None if equal else torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    return d


def reference(d, chunk=64):
    """(outputs, final states) in 64 bits, `chunk` tokens of a sequence at a time: within a chunk the scores of
    earlier tokens weighted by their decays, across chunks the state."""
    H, Hk = d["v"].shape[1], d["q"].shape[1]
    wide = lambda t: t.double().repeat_interleave(H // Hk, 1)  # noqa: E731
    q, k, v, g = wide(d["q"]), wide(d["k"]), d["v"].double(), d["g"].double()
    out, finals, at = torch.empty_like(v), [], 0
    for n, length in enumerate(d["lens"]):
        S = d["S"][n].double()
        for a in range(at, at + length, chunk):
            b = min(a + chunk, at + length)
            G = g[a:b].cumsum(0)
            D = (G[:, None] - G[None]).permute(2, 0, 1)
            D = torch.where(torch.ones_like(D[0]).tril().bool(), D, -math.inf).exp()
            scores = torch.einsum("ihd,jhd->hij", q[a:b], k[a:b]) * D
            out[a:b] = torch.einsum("hij,jhe->ihe", scores, v[a:b])
            out[a:b] += G.exp()[..., None] * torch.einsum("ihd,hde->ihe", q[a:b], S)
            left = (G[-1] - G).exp()
            S = G[-1].exp()[:, None, None] * S + torch.einsum("jh,jhd,jhe->hde", left, k[a:b], v[a:b])
        finals.append(S)
        at += length
    out *= d["scale"]
    if d["z"] is not None:
        z = d["z"].double()
        out = out / (out.square().mean(-1, keepdim=True) + 1e-5).sqrt() * d["w"].double() * z / (1 + torch.exp(-z))
    return out.cpu().numpy(), torch.stack(finals).cpu().numpy()
