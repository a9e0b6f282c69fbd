"""Calls of the head-decay attention that its documentation allows, in the settings a program makes them in.

Tolerances as in test_gpu_hla.py."""
import subprocess
import sys

import pytest
import torch

from linear_vision_backbone_b200 import binding, build
from tests.hla_steady import STEADY, inputs, reference
from tests.parity import assert_close
from tests.test_gpu_hla import DT, check_states, dev, make
from tests.test_gpu_hla import reference as oracle_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    build.build()
    binding.load()


FIRST = """
import sys, torch
sys.path.insert(0, {root!r})
from linear_vision_backbone_b200 import binding
torch.manual_seed(0)
q, k, v, z = (torch.randn(3000, 2, 64, device="cuda").{type}() for _ in range(4))
g = torch.full((3000, 2), -0.02, device="cuda")
pool, x = torch.zeros(1, 2, 64, 64, device="cuda"), torch.randn(3000, 128, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    y = binding.hla_fwd(q, k, v, g, z, state_in=pool, state_out=pool)
    one = binding.hla_step(q[:1], k[:1], v[:1], g[:1], pool, z[:1])
    h = binding.residual_norm(x, y.view(3000, 128), pre_norm=True)
pool.zero_()
x0 = x.clone()
graph.replay()
torch.cuda.synchronize()
p2, x2 = torch.zeros_like(pool), x0.clone()
y2 = binding.hla_fwd(q, k, v, g, z, state_in=p2, state_out=p2)
one2 = binding.hla_step(q[:1], k[:1], v[:1], g[:1], p2, z[:1])
h2 = binding.residual_norm(x2, y2.view(3000, 128), pre_norm=True)
for a, b in ((y, y2), (one, one2), (h, h2), (pool, p2), (x, x2)):
    assert torch.equal(a, b)
assert binding.device_status()[0] == 0
print("captured")
"""


@pytest.mark.parametrize("dtype", ["half", "bfloat16", "float"])
def test_a_process_whose_first_call_is_captured(dtype):
    code = FIRST.format(root=build.ROOT, type=dtype)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=180)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("dtype,dk", [("f16", 64), ("bf16", 128), ("f32", 32)])
def test_slots_without_states_skip_sequences(dtype, dk):
    lens = [40, 150, 3, 60]
    d = make(lens, 2, 2, dk, dk, dtype, seed=40)
    c = dev(d)
    out = torch.full_like(c["v"], 7.0)
    slots = torch.tensor([0, -1, 9, -3], dtype=torch.int32, device="cuda")       # no pool: only their signs count
    binding.hla_fwd(c["q"], c["k"], c["v"], c["g"], c["z"], c["w"], cu_seqlens=c["cu"], scale=d["scale"], slots=slots,
                    out=out)
    ref, _ = oracle_of(d)
    for n, (a, b) in enumerate(zip(d["cu"].tolist(), d["cu"].tolist()[1:])):
        if slots[n] < 0:
            assert (out[a:b] == 7).all()
        else:
            assert_close(out[a:b], ref[a:b], DT[dtype], f"sequence {n}")
    assert binding.device_status()[0] == 0


def test_two_graphs_replayed_at_the_same_time():
    made = []
    for n, name in enumerate(("f16-128-gated", "bf16-64-gated")):
        case = STEADY[name]
        d = inputs(case, seed=50 + n)
        fin, out = torch.empty_like(d["S"]), torch.empty_like(d["v"])
        call = lambda d=d, fin=fin, out=out: binding.hla_fwd(  # noqa: E731
            d["q"], d["k"], d["v"], d["g"], d["z"], d["w"], cu_seqlens=d["cu"], scale=d["scale"], state_in=d["S"],
            state_out=fin, out=out)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            call()
        graph.replay()
        torch.cuda.synchronize()
        ref, S = reference(d)
        assert_close(out, ref, d["v"].dtype, name)
        check_states(fin, S, name)
        made.append((graph, torch.cuda.Stream(), out, fin, out.clone(), fin.clone(), d))    # d: a graph owns no input
    for _ in range(10):
        for graph, stream, out, fin, *_ in made:
            with torch.cuda.stream(stream):
                out.fill_(7.0)
                fin.fill_(7.0)
                for _ in range(3):
                    graph.replay()
        torch.cuda.synchronize()
        for _, _, out, fin, out0, fin0, _ in made:
            assert torch.equal(out, out0) and torch.equal(fin, fin0)


@pytest.mark.parametrize("dtype,dk,block", [("f16", 64, 128), ("bf16", 128, 128), ("bf16", 32, 1), ("f32", 64, 1)])
def test_a_nan_value_leaves_earlier_blocks_alone(dtype, dk, block):
    # tensor cores: any output of its block of 128 tokens and what follows; CUDA cores: what follows
    d = make([400], 2, 2, dk, dk, dtype, seed=41, gated=False)
    ref, _ = oracle_of(d)
    at = 300
    d["v"][at, 1, 5] = float("nan")
    c = dev(d)
    out = binding.hla_fwd(c["q"], c["k"], c["v"], c["g"], scale=d["scale"])
    clean = at // block * block
    assert_close(out[:, 0], ref[:, 0], DT[dtype], "the other head")
    assert_close(out[:clean, 1], ref[:clean, 1], DT[dtype], "earlier blocks")
    assert torch.isnan(out[at:, 1, 5].float()).all()


@pytest.mark.parametrize("dtype,dk", [("f16", 64), ("bf16", 128), ("f32", 64)])
def test_batches_as_column_blocks_of_one_buffer(dtype, dk):
    # [B, T, width] with q, k, v, z and out beside each other: one pitch for all
    B, T, H = 3, 150, 2
    d = make([T] * B, H, H, dk, dk, dtype, seed=42)
    w = H * dk
    buf = torch.full((B, T, 5 * w + 16), 7.0, dtype=DT[dtype], device="cuda")
    q, k, v, z, out = (buf[..., 8 + i * w:8 + (i + 1) * w].unflatten(2, (H, dk)) for i in range(5))
    for n, t in (("q", q), ("k", k), ("v", v), ("z", z)):
        t.copy_(d[n].view(B, T, H, dk))
    fin = torch.empty(B, H, dk, dk, device="cuda")
    got = binding.hla_fwd(q, k, v, d["g"].view(B, T, H).cuda(), z, d["w"].cuda(), scale=d["scale"], state_out=fin, out=out)
    assert got is out
    ref, S = oracle_of(d)
    assert_close(out.reshape(B * T, H, dk), ref, DT[dtype], "columns")
    check_states(fin, S)
    assert (buf[..., :8] == 7).all() and (buf[..., 8 + 5 * w:] == 7).all()
    for n, t in (("q", q), ("k", k), ("v", v), ("z", z)):
        assert torch.equal(t.cpu(), d[n].view(B, T, H, dk))


@pytest.mark.parametrize("dk,dv", [(16, 16), (32, 64), (64, 32), (16, 128)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_long_walks_of_small_heads(dk, dv, dtype):
    # 16-bit heads of 16 and 32 dims: CUDA cores, many batches of tokens a group
    case = ([900, 0, 1, 1300, 700, 33], 6, 3, dk, dv, dtype, True, False)
    d = inputs(case, seed=60)
    fin = torch.empty_like(d["S"])
    call = lambda: binding.hla_fwd(d["q"], d["k"], d["v"], d["g"], d["z"], d["w"], cu_seqlens=d["cu"],  # noqa: E731
                                   scale=d["scale"], state_in=d["S"], state_out=fin)
    out = call()
    ref, S = reference(d)
    assert_close(out, ref, DT[dtype], "small heads")
    check_states(fin, S)
    assert torch.equal(call(), out)
