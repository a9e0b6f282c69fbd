"""The gates of the residual norm over the whole range of their argument, element by element."""
import numpy as np
import pytest
import torch

from linear_vision_backbone_b200 import binding, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    build.build()
    binding.load()


def gated(z, act, dtype, D):
    x = torch.zeros(len(z) // D, D, device="cuda")
    y = torch.full_like(x, 3.0).to(dtype)
    binding.residual_norm(x, y, gate=z.to(dtype).cuda().view_as(x), gate_act=act)
    return x.double().cpu().numpy().ravel()


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("D", [64, 65])
def test_fp32_gates(act, D):
    """exp (2 ulp: 2^-22), a sum, a quotient and three products of 2^-24 each: within 2^-20 of the value; results
    below fp32's normal numbers are off by their step of 2^-149, twice that with the products behind."""
    z = torch.cat([torch.linspace(-104, 104, 64 * 65 * 4 - 7), torch.tensor([0.0, -0.0, 1e-30, -1e-30, -87.5, -88.8, 200.0])])
    got = gated(z, act, torch.float32, D)
    zd = z.double().numpy()
    sig = np.where(zd >= 0, 1 / (1 + np.exp(-np.abs(zd))), np.exp(-np.abs(zd)) / (1 + np.exp(-np.abs(zd))))
    want = 3.0 * sig * (zd if act == "silu" else 1.0)
    err = np.abs(got - want) / (np.abs(want) * 2 ** -20 + 2 ** -149 * 3 * np.maximum(np.abs(zd), 1))
    assert err.max() <= 1.0, (err.max(), z[err.argmax()])


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_16_bit_gates(act, dtype):
    """The short form for 16-bit branches: the rounding of z log2 e becomes |z| 2^-24 of e^-z, and with the two
    instructions (2^-22 each) and the products the value is within |z| 2^-24 + 2^-20; a sigmoid below 2^-126 is zero."""
    z = torch.cat([torch.linspace(-100, 100, 64 * 256 - 4), torch.tensor([0.0, -0.0, -87.0, -88.0])]).to(dtype)
    got = gated(z, act, dtype, 64)
    zd = z.double().numpy()
    want = 3.0 * np.exp(-np.logaddexp(0, -zd)) * (zd if act == "silu" else 1.0)
    err = np.abs(got - want) / (np.abs(want) * (np.abs(zd) * 2 ** -24 + 2 ** -20) + 2.0 ** -126 * 3 * np.maximum(np.abs(zd), 1))
    assert err.max() <= 1.0, (err.max(), z[err.argmax()])


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_infinite_gates(dtype):
    z = torch.tensor([float("inf"), -float("inf")] * 32)
    got = gated(z, "sigmoid", dtype, 64)
    assert (got[::2] == 3).all() and (got[1::2] == 0).all()
