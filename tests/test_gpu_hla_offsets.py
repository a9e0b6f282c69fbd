"""Offsets that are not those of packed sequences: nothing is computed, and the device status says so.

Their blocks could be more than 31 bits count, which is what the kernels number them with."""
import pytest
import torch

from linear_vision_backbone_b200 import binding, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    build.build()
    binding.load()


BAD = {"decreasing": [0, 40, 30, 70], "twice": [0, 70, 0, 70], "negative": [-1, 20, 40, 70], "past the end": [0, 20, 40, 71],
       "all past": [80, 90, 90, 100], "far": [0, 20, 40, 2 ** 31 - 1]}


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("dtype,dk", [(torch.float16, 64), (torch.bfloat16, 128), (torch.float32, 32)])
def test_invalid_offsets_compute_nothing(bad, many, dtype, dk):
    cu = BAD[bad]
    if many:                                # more than 32 sequences: the block-wide search
        cu = cu[:1] * 20 + cu + cu[-1:] * 20
    n, T, H = len(cu) - 1, 70, 2
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    q, k, v = (torch.randn(T, H, dk, device="cuda", generator=gen).to(dtype) for _ in range(3))
    g = torch.full((T, H), -0.1, device="cuda")
    S = torch.randn(n, H, dk, dk, device="cuda", generator=gen)
    fin, out = torch.full_like(S, 5.0), torch.full_like(v, 7.0)
    assert binding.device_status()[0] == 0
    call = lambda offsets: binding.hla_fwd(q, k, v, g, cu_seqlens=torch.tensor(offsets).int().cuda(), state_in=S,  # noqa: E731
                                           state_out=fin, out=out)
    call(cu)
    rc, bits, _ = binding.device_status()
    assert rc == -6 and bits == 2
    assert (out == 7).all() and (fin == 5).all()
    call([0] * n + [T])                     # and the next call is as ever
    assert binding.device_status()[0] == 0
    assert torch.equal(fin[:-1], S[:-1]) and not (out == 7).all(-1).any()   # every row is written


def test_invalid_offsets_of_a_call_with_cuts():
    T, H, d = 9000, 1, 64
    q, k, v = (torch.randn(T, H, d, device="cuda").half() for _ in range(3))
    g = torch.full((T, H), -0.01, device="cuda")
    S = torch.randn(2, H, d, d, device="cuda")
    for cu in ([0, 9000, 8000], [0, 8000, 9001]):
        pool, out = S.clone(), torch.full_like(v, 7.0)
        binding.hla_fwd(q, k, v, g, cu_seqlens=torch.tensor(cu).int().cuda(), state_in=pool, state_out=pool, out=out)
        rc, bits, _ = binding.device_status()
        assert rc == -6 and bits == 2 and torch.equal(pool, S) and (out == 7).all()
