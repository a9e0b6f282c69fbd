"""Head-decay attention where a group walks many blocks of tokens: against 64 bits, and bit for bit again.

Tolerances as in test_gpu_hla.py: outputs by tests/parity.py, states 1e-5 relative L2.
"""
import pytest
import torch

import oracle
from linear_vision_backbone_b200 import binding, build
from tests.hla_steady import SMS, STEADY, inputs, plan, reference
from tests.parity import assert_close
from tests.test_gpu_hla import check_states

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    build.build()
    binding.load()


def run(d, case):
    equal = case[-1]
    n = len(d["lens"])
    shape = (lambda t: None if t is None else t.unflatten(0, (n, -1))) if equal else (lambda t: t)
    fin = torch.full_like(d["S"], 5.0)
    out = binding.hla_fwd(shape(d["q"]), shape(d["k"]), shape(d["v"]), shape(d["g"]), shape(d["z"]), d["w"],
                          cu_seqlens=d["cu"], scale=d["scale"], state_in=d["S"], state_out=fin)
    return out.view(d["v"].shape), fin


def test_reference_equals_the_oracle():
    d = inputs(([70, 0, 200], 4, 2, 16, 32, "f32", True, False), 1)
    out, S = reference(d)
    want, SW = oracle.hla_fwd(d["q"], d["k"], d["v"], d["g"], d["z"], d["w"], cu_seqlens=d["cu"].tolist(),
                              scale=d["scale"], states=d["S"])
    assert abs(out - want).max() < 1e-11 * abs(want).max() and abs(S - SW).max() < 1e-11 * abs(SW).max()


@pytest.mark.parametrize("name", STEADY)
def test_long_walks(name):
    case = STEADY[name]
    lens, H, Hk, dk, dv, dtype, gated, equal = case
    d = inputs(case, seed=len(name))
    if torch.cuda.get_device_properties(0).multi_processor_count == SMS and not equal:
        # the plan that the CPU test looks at is the library's
        ids = {"f32": 0, "f16": 1, "bf16": 2}
        need = binding.load().gtr_hla_workspace_bytes(len(lens), sum(lens), H, dk, dv, ids[dtype])
        sizes = [plan(len(lens), sum(lens), H, dk, dv, dtype, e)[2] for e in (False, True)]
        assert need == (max(sizes) if sum(lens) % len(lens) == 0 else sizes[0])
    out, fin = run(d, case)
    ref, S = reference(d)
    assert_close(out, ref, DT[dtype], name)
    check_states(fin, S, name)
    assert binding.device_status()[0] == 0
    for _ in range(6):
        again, fin2 = run(d, case)
        assert torch.equal(again, out) and torch.equal(fin2, fin), name
