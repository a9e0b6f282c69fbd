"""The head-decay linear attention and the residual norm: cases, plain forms and exact values.

Three operators are timed and compared here: the prompt form of the linear
attention with one decay per head (``binding.hla_fwd``), its form for single
tokens (``binding.hla_step``) and the norms around a block with its gate and
residual scale (``binding.residual_norm``).
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
RMS_EPS = 1e-5


# --------------------------------------------------------------------- cases
def _prompt(name, lens, H, Hk, dk, dv, dtype, **more):
    case = {"op": "prompt", "lens": " ".join(map(str, lens)), "H": H, "Hk": Hk, "dk": dk, "dv": dv, "dtype": dtype,
            "gated": True,      # RMSNorm x SiLU(z) on the output
            "decay": "token",   # a log-decay per token and head; "head": one constant per head
            "gate_div": 16.0,   # log-decays are logsigmoid(N(2, 1)) / gate_div
            "start": False,     # sequences continue from a state
            "final": True}      # the states they end with are wanted
    case.update(more)
    return dict(case, name=name) if name else case


def _step(name, N, slots, H, Hk, dk, dv, dtype, **more):
    case = {"op": "step", "N": N, "slots": slots, "H": H, "Hk": Hk, "dk": dk, "dv": dv, "dtype": dtype,
            "gated": True, "decay": "token", "gate_div": 16.0}
    case.update(more)
    return dict(case, name=name) if name else case


def _norm(name, N, D, x_dtype, dtype, **more):
    case = {"op": "norm", "N": N, "D": D, "x_dtype": x_dtype, "dtype": dtype, "post": True, "gate": "none",
            "res_scale": True, "pre": True}
    case.update(more)
    return dict(case, name=name) if name else case


def _lens(case):
    return [int(n) for n in case["lens"].split()]


def _ragged(seed, n, low, high):
    """n lengths spread over the logarithm of [low, high]."""
    import random
    r = random.Random(seed)
    return [int(round(math.exp(r.uniform(math.log(low), math.log(high))))) for _ in range(n)]


def listed():
    return [
        # one long sequence, few heads: a 128 x 128 token grid read as a sequence, output gate on
        _prompt("prompt_16k", [16384], 6, 6, 64, 64, "f16"),
        # the longest: a 256 x 256 grid, four heads of 128 dims
        _prompt("prompt_64k", [65536], 4, 4, 128, 128, "bf16"),
        # a batch of equal sequences, constant decays per head
        _prompt("prompt_batch8", [1600] * 8, 6, 6, 64, 64, "bf16", decay="head"),
        # a serving batch: prompts of many lengths, key heads shared by four value heads,
        # some of it continuing from earlier states, raw output
        _prompt("prompt_packed", _ragged(7, 28, 3, 9000), 16, 4, 128, 128, "bf16", gated=False, start=True),
        # the smallest call: one short odd prompt
        _prompt("prompt_short", [77], 4, 4, 64, 64, "f16"),
        # full precision
        _prompt("prompt_f32", [1600], 6, 6, 64, 64, "f32", final=False),
        # one request's next token
        _step("step_1", 1, 4, 6, 6, 64, 64, "f16"),
        # a usual decoding batch
        _step("step_64", 64, 96, 16, 4, 128, 128, "bf16"),
        # the largest decoding batch, constant decays, raw output
        _step("step_500", 500, 512, 16, 16, 128, 128, "bf16", gated=False, decay="head"),
        # the residual stream of the 128 x 128 grid: fp32 stream, 16-bit branch
        _norm("norm_16k", 16384, 384, "f32", "f16", post=False),
        # rows of a decoding batch
        _norm("norm_9", 9, 4096, "bf16", "bf16", gate="sigmoid"),
        # a wide stream with both norms and an elementwise SiLU gate
        _norm("norm_wide", 8191, 5120, "bf16", "bf16", gate="silu"),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "step", "norm"])
    if op == "norm":
        N, D = _log_int(rng, 1, 20000), _log_int(rng, 40, 8192)
        D -= D % rng.choice([1, 2, 8, 64])
        while N * D > 40_000_000:
            N = max(1, N // 2)
        x_dtype = rng.choice(["f32", "f16", "bf16"])
        return _norm(None, N, D, x_dtype, x_dtype if x_dtype != "f32" else rng.choice(["f32", "f16", "bf16"]),
                     post=rng.random() < 0.6, gate=rng.choice(["none", "mul", "sigmoid", "silu"]),
                     res_scale=rng.random() < 0.6, pre=rng.random() < 0.8)
    Hk = rng.choice([1, 2, 3, 4, 6, 8])
    H = Hk * rng.choice([1, 1, 2, 4])
    H = min(H, 16) if min(H, 16) % Hk == 0 else Hk
    dk, dv = rng.choice([(64, 64), (64, 64), (128, 128), (128, 128), (64, 128), (128, 64)])
    dtype = rng.choice(["f16", "bf16", "bf16"])
    more = {"gated": rng.random() < 0.6, "decay": rng.choice(["token", "token", "head"]),
            "gate_div": rng.choice([1.0, 4.0, 16.0, 64.0])}
    if op == "step":
        N = _log_int(rng, 1, 480)
        if rng.random() < 0.2:
            dtype = "f32"
        return _step(None, N, N + rng.randrange(0, 30), H, Hk, dk, dv, dtype, **more)
    if rng.random() < 0.15:   # full precision, moderate lengths
        return _prompt(None, [_log_int(rng, 1, 3000) for _ in range(rng.randrange(1, 5))], H, Hk, dk, dv, "f32",
                       start=rng.random() < 0.5, final=rng.random() < 0.7, **more)
    total = _log_int(rng, 20, 40000)
    n = min(total, _log_int(rng, 1, 40))
    cuts = sorted(rng.sample(range(1, total), n - 1)) if n > 1 else []
    lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    return _prompt(None, lens, H, Hk, dk, dv, dtype, start=rng.random() < 0.5, final=rng.random() < 0.7, **more)


# -------------------------------------------------------------------- inputs
def _log_decay(case, rows, gen):
    if case["decay"] == "head":   # a geometric ladder of decay times, 16 tokens and up
        return torch.log1p(-torch.exp2(-4.0 - torch.arange(case["H"], device="cuda") / 2.0)).float()
    u = torch.randn(rows, case["H"], device="cuda", generator=gen) + 2.0
    return torch.nn.functional.logsigmoid(u) / case["gate_div"]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, device="cuda", generator=gen)  # noqa: E731
    dt = TYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "norm":
        N, D = case["N"], case["D"]
        s["x"] = normal(N, D).to(TYPES[case["x_dtype"]])
        s["y"] = (normal(N, D) * 0.7).to(dt)
        s["post_w"] = 1.0 + 0.2 * normal(D) if case["post"] else None
        s["gate"] = normal(N, D).to(dt) if case["gate"] != "none" else None
        s["res_scale"] = 0.5 * normal(D) if case["res_scale"] else None
        s["pre_w"] = 1.0 + 0.2 * normal(D) if case["pre"] else None
        s["x_out"] = torch.empty_like(s["x"])
        return s
    H, Hk, dk, dv = case["H"], case["Hk"], case["dk"], case["dv"]
    rows = sum(_lens(case)) if case["op"] == "prompt" else case["N"]
    s["q"], s["k"] = normal(rows, Hk, dk).to(dt), normal(rows, Hk, dk).to(dt)
    s["v"] = normal(rows, H, dv).to(dt)
    s["z"] = normal(rows, H, dv).to(dt) if case["gated"] else None
    s["w"] = 1.0 + 0.2 * normal(dv) if case["gated"] else None
    s["g"] = _log_decay(case, rows, gen)
    s["scale"] = dk ** -0.5
    if case["op"] == "prompt":
        lens = torch.tensor([0] + _lens(case))
        s["cu"] = torch.cumsum(lens, 0).to(torch.int32).cuda()
        n = len(_lens(case))
        s["state_in"] = normal(n, H, dk, dv) * 4.0 if case["start"] else None
        s["state_out"] = torch.zeros(n, H, dk, dv, device="cuda") if case["final"] else None
        # tokens that each sequence has already seen: none for every third, whose state is not read
        s["seen"] = torch.tensor([0 if i % 3 == 2 else 10 + i for i in range(n)], dtype=torch.int32).cuda() \
            if case["start"] else None
    else:
        s["state_in"] = normal(case["slots"], H, dk, dv) * 4.0
        s["state_out"] = torch.zeros(case["slots"], H, dk, dv, device="cuda")
        s["slots"] = torch.randperm(case["slots"], device="cuda", generator=gen)[:rows].to(torch.int32)
    return s


# --------------------------------------------------------------- plain forms
def _gate_norm(o, s):
    """RMSNorm over the head dim, its weight and the SiLU gate, in 32 bits."""
    if s["z"] is None:
        return o
    o = o * torch.rsqrt((o * o).mean(-1, keepdim=True) + RMS_EPS) * s["w"]
    z = s["z"].float()
    return o * z / (1.0 + torch.exp(-z))


def _plain_prompt(s, C=128):
    """Chunks of C tokens: masked scores within, a product with the decays between them across."""
    case, q = s["case"], s["q"]
    T, (H, Hk, dk, dv) = q.shape[0], (case["H"], case["Hk"], case["dk"], case["dv"])
    n = len(_lens(case))
    nc = T // C + n
    cu = s["cu"].long()
    lens = cu[1:] - cu[:-1]
    ends = torch.cumsum((lens + C - 1) // C, 0)
    chunk = torch.arange(nc, device=q.device)
    seq = torch.searchsorted(ends, chunk, right=True)
    live = seq < n
    seq = seq.clamp(max=n - 1)
    first = ends[seq] - (lens[seq] + C - 1) // C            # the sequence's first chunk
    pos = (chunk - first)[:, None] * C + torch.arange(C, device=q.device)
    valid = live[:, None] & (pos < lens[seq][:, None])       # [nc, C]
    row = torch.where(valid, cu[seq][:, None] + pos, 0)
    keep = valid[:, :, None, None].float()
    qc = q[row].float() * keep * s["scale"]
    kc = s["k"][row].float() * keep
    vc = s["v"][row].float() * keep                          # [nc, C, H, dv]
    g = s["g"].double()
    g = g[row] if g.dim() == 2 else g.expand(nc, C, H)
    G = torch.cumsum(g * valid[:, :, None], 1)               # [nc, C, H], 64 bits
    A = G[:, -1]                                             # [nc, H]
    r = H // Hk
    qh = qc.permute(0, 2, 1, 3).repeat_interleave(r, 1)      # [nc, H, C, dk]
    kh = kc.permute(0, 2, 1, 3).repeat_interleave(r, 1)
    vh = vc.permute(0, 2, 1, 3)
    Gh = G.permute(0, 2, 1)                                  # [nc, H, C]
    causal = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    D = torch.exp((Gh[:, :, :, None] - Gh[:, :, None, :]).float().masked_fill(~causal, -math.inf))
    o = ((qh @ kh.transpose(-1, -2)) * D) @ vh
    del D
    w = torch.exp((Gh[:, :, -1:] - Gh).float())
    dS = (kh * w[..., None]).transpose(-1, -2) @ vh          # [nc, H, dk, dv]
    E = torch.cumsum(A, 0) - A                               # log-decay before each chunk, from the first of all
    before = (seq[None, :] == seq[:, None]) & (chunk[None, :] < chunk[:, None]) & live[:, None] & live[None, :]
    M = (E.t()[:, :, None] - (E + A).t()[:, None, :]).float().masked_fill(~before, -math.inf).exp()
    S = torch.bmm(M, dS.permute(1, 0, 2, 3).reshape(H, nc, dk * dv)).view(H, nc, dk, dv).permute(1, 0, 2, 3)
    S0 = None
    if s["state_in"] is not None:
        S0 = s["state_in"] * (s["seen"] > 0)[:, None, None, None]
        S = S + torch.exp((E - E[first.clamp(max=nc - 1)]).float())[..., None, None] * S0[seq]
    o = o + torch.exp(Gh.float())[..., None] * (qh @ S)
    o = o.permute(0, 2, 1, 3)                                # [nc, C, H, dv]
    flat = torch.empty(T + 1, H, dv, device=q.device)
    flat[torch.where(valid, row, T)] = o
    out = _gate_norm(flat[:T], s).to(q.dtype)
    if s["state_out"] is None:
        return out
    last = (ends - 1).clamp(min=0)
    end = torch.exp(A[last].float())[..., None, None] * S[last] + dS[last]
    empty = (lens == 0)[:, None, None, None]
    s["state_out"].copy_(torch.where(empty, S0 if S0 is not None else torch.zeros_like(end), end))
    return out, s["state_out"]


def _plain_step(s):
    r = s["case"]["H"] // s["case"]["Hk"]
    at = s["slots"].long()
    q = s["q"].float().repeat_interleave(r, 1) * s["scale"]
    k = s["k"].float().repeat_interleave(r, 1)
    S = torch.exp(s["g"])[..., None, None] * s["state_in"][at] + k[..., None] * s["v"].float()[:, :, None, :]
    o = (q[:, :, None, :] @ S)[:, :, 0]
    s["state_out"].index_copy_(0, at, S)
    return _gate_norm(o, s).to(s["q"].dtype), s["state_out"]


def _plain_norm(s):
    x, r = s["x"].float(), s["y"].float()
    if s["post_w"] is not None:
        r = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + RMS_EPS) * s["post_w"]
    if s["gate"] is not None:
        gate, kind = s["gate"].float(), s["case"]["gate"]
        r = r * (gate if kind == "mul" else torch.sigmoid(gate) if kind == "sigmoid" else gate * torch.sigmoid(gate))
    if s["res_scale"] is not None:
        r = r * s["res_scale"]
    x = x + r
    s["x_out"].copy_(x)
    if s["pre_w"] is None:
        return s["x_out"]
    out = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + RMS_EPS) * s["pre_w"]
    return s["x_out"], out.to(s["y"].dtype)


def run(s):
    op = s["case"]["op"]
    if not own:
        return _plain_prompt(s) if op == "prompt" else _plain_step(s) if op == "step" else _plain_norm(s)
    from linear_vision_backbone_b200 import binding
    if op == "prompt":
        out = binding.hla_fwd(s["q"], s["k"], s["v"], s["g"], s["z"], s["w"], cu_seqlens=s["cu"], scale=s["scale"],
                              state_in=s["state_in"], state_out=s["state_out"], seen=s["seen"])
        return out if s["state_out"] is None else (out, s["state_out"])
    if op == "step":
        out = binding.hla_step(s["q"], s["k"], s["v"], s["g"], s["state_in"], s["z"], s["w"], slots=s["slots"],
                               scale=s["scale"], state_out=s["state_out"])
        return out, s["state_out"]
    out = binding.residual_norm(s["x"], s["y"], post_w=s["post_w"], gate=s["gate"], gate_act=s["case"]["gate"],
                                res_scale=s["res_scale"], pre_w=s["pre_w"], x_out=s["x_out"])
    return s["x_out"] if s["pre_w"] is None else (s["x_out"], out)


# ------------------------------------------------------------------ the work
def work(case):
    es = BYTES[case["dtype"]]
    if case["op"] == "norm":
        N, D = case["N"], case["D"]
        tensors = 1 + (case["gate"] != "none") + case["pre"]           # y, gate, out
        vectors = case["post"] + case["res_scale"] + case["pre"]
        per = 2 + 4 * case["post"] + 3 * (case["gate"] != "none") + case["res_scale"] + 4 * case["pre"]
        return {"bytes": N * D * (2 * BYTES[case["x_dtype"]] + tensors * es) + 4 * D * vectors, "flops": N * D * per}
    H, Hk, dk, dv = case["H"], case["Hk"], case["dk"], case["dv"]
    rows = sum(_lens(case)) if case["op"] == "prompt" else case["N"]
    b = rows * (2 * Hk * dk + (2 + case["gated"]) * H * dv) * es
    b += 4 * H * (rows if case["decay"] == "token" else 1)
    if case["op"] == "prompt":
        # every third sequence of a batch with states starts without one
        n = len(_lens(case))
        states = (n - n // 3 if case["start"] else 0) + (n if case["final"] else 0)
    else:
        states = 2 * rows
    b += 4 * states * H * dk * dv
    return {"bytes": b, "flops": rows * H * (5 if case["op"] == "step" else 4) * dk * dv}


# --------------------------------------------------------------- exact values
def _silu(t):
    return t * torch.sigmoid(t)


def _finish(o, s):
    if s["z"] is None:
        return o
    return o / torch.sqrt(o.square().mean(-1, keepdim=True) + 1e-5) * s["w"].double() * _silu(s["z"].double())


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        branch = s["y"].double()
        if case["post"]:
            branch = branch / torch.sqrt(branch.square().mean(-1, keepdim=True) + 1e-5) * s["post_w"].double()
        if case["gate"] == "mul":
            branch = branch * s["gate"].double()
        elif case["gate"] == "sigmoid":
            branch = branch * torch.sigmoid(s["gate"].double())
        elif case["gate"] == "silu":
            branch = branch * _silu(s["gate"].double())
        if case["res_scale"]:
            branch = branch * s["res_scale"].double()
        x = s["x"].double() + branch
        if not case["pre"]:
            return x
        return x, x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-5) * s["pre_w"].double()
    group = case["H"] // case["Hk"]
    spread = lambda t: t.double().repeat_interleave(group, dim=1)  # noqa: E731
    g = s["g"].double()
    if case["op"] == "step":
        at = s["slots"].long()
        states = s["state_out"].double()
        S = s["state_in"].double()[at] * torch.exp(g)[..., None, None]
        S = S + torch.einsum("nhi,nhj->nhij", spread(s["k"]), s["v"].double())
        states[at] = S
        return _finish(torch.einsum("nhi,nhij->nhj", spread(s["q"]), S) * s["scale"], s), states
    # the recurrence, 64 tokens of one sequence at a time
    out = torch.empty_like(s["v"], dtype=torch.float64)
    states, at = [], 0
    for i, length in enumerate(_lens(case)):
        S = torch.zeros(case["H"], case["dk"], case["dv"], dtype=torch.float64, device="cuda")
        if case["start"] and i % 3 != 2:
            S = s["state_in"][i].double()
        for a in range(at, at + length, 64):
            b = min(a + 64, at + length)
            q, k, v = (t.transpose(0, 1) for t in (spread(s["q"][a:b]), spread(s["k"][a:b]), s["v"][a:b].double()))
            G = torch.cumsum(g[a:b] if case["decay"] == "token" else g.expand(b - a, -1), 0).t()   # [H, n]
            weight = torch.exp(torch.tril(G[:, :, None] - G[:, None, :])).tril()
            out[a:b] = (torch.einsum("hij,hjd->hid", torch.einsum("hic,hjc->hij", q, k) * weight, v)
                        + torch.exp(G)[..., None] * torch.einsum("hic,hcd->hid", q, S)).transpose(0, 1)
            S = torch.exp(G[:, -1])[:, None, None] * S + torch.einsum(
                "hjc,hjd->hcd", k * torch.exp(G[:, -1:] - G)[..., None], v)
        states.append(S)
        at += length
    out = _finish(out * s["scale"], s)
    return (out, torch.stack(states)) if case["final"] else out
