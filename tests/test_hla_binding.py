"""What the binding of the head-decay attention and the residual norm sends to the C ABI, and what it
refuses, without a GPU: its checks run on CPU tensors, whose device is -1."""
import pytest
import torch

from linear_vision_backbone_b200 import binding


def pitch(t):
    return binding._pitch(t, "q", t.dtype, t.shape, -1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_row_pitches(dtype):
    e = lambda *s: torch.empty(*s, dtype=dtype)  # noqa: E731
    assert pitch(e(5, 2, 64)) == 0 and pitch(e(0, 2, 64)) == 0 and pitch(e(3, 5, 2, 64)) == 0      # dense
    assert pitch(e(5, 400)[:, 64:192].unflatten(1, (2, 64))) == 400
    assert pitch(e(3, 5, 400)[..., 64:192].unflatten(2, (2, 64))) == 400
    assert pitch(e(3, 1, 400)[..., 64:192].unflatten(2, (2, 64))) == 400    # one token a sequence
    assert pitch(e(1, 5, 400)[..., 64:192].unflatten(2, (2, 64))) == 400
    assert pitch(e(1, 400)[:, 64:192].unflatten(1, (2, 64))) == 0           # one row has no pitch
    assert pitch(e(1, 2, 64).expand(1, 2, 64)) == 0


@pytest.mark.parametrize("t", [
    torch.empty(1, 2, 64).expand(10, 2, 64),                  # one row for every token
    torch.empty(2, 64).expand(10, 2, 64),
    torch.empty(1, 1, 64).expand(10, 1, 64),
    torch.empty(1, 1, 2, 64).expand(3, 10, 2, 64),            # for every token of every sequence
    torch.empty(1, 1, 2, 64).expand(3, 1, 2, 64),             # one token, a batch
    torch.empty(1, 1, 2, 64).expand(1, 10, 2, 64),
    torch.empty(1, 10, 2, 64).expand(3, 10, 2, 64),           # one sequence for the batch
    torch.empty(3, 1, 2, 64).expand(3, 10, 2, 64),            # one token for each sequence
    torch.empty(1000).as_strided((10, 2, 64), (64, 64, 1)),   # rows that share columns
    torch.empty(1000).as_strided((3, 4, 2, 64), (256, 64, 64, 1)),
    torch.empty(10, 1, 64).expand(10, 2, 64),                 # one head for all
    torch.empty(10, 2, 1).expand(10, 2, 64),
])
def test_rows_that_share_memory_are_refused(t):
    # a pitch of zero stands for dense rows: a broadcast tensor would be read (or written) past its end
    with pytest.raises(ValueError):
        pitch(t)


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is on cuda:0, for the checks before a launch."""

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return 0


@pytest.fixture
def no_launch(monkeypatch):
    """The binding without a device: calls that reach the library fail the test."""
    monkeypatch.setattr(binding, "_elsewhere", lambda device, stream: False)
    monkeypatch.setattr(binding, "load", lambda: pytest.fail("reached the library"))
    monkeypatch.setattr(binding, "_lib", None)


def on_device(*shape, dtype=torch.float16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


def test_offsets_that_are_no_tensor_are_refused(no_launch):
    q, g = on_device(6, 2, 64), on_device(6, 2, dtype=torch.float32)
    for cu in ([0, 2, 6], (0, 6), 6):
        with pytest.raises(ValueError, match="cu_seqlens"):
            binding.hla_fwd(q, q, q, g, cu_seqlens=cu)


def test_a_gate_needs_its_kind(no_launch):
    # "none" is for calls without a gate: it would have multiplied by the raw gate
    x = on_device(4, 64)
    with pytest.raises(ValueError, match="gate_act"):
        binding.residual_norm(x, x, gate=x, gate_act="none")


def test_every_variant_of_the_norm_has_a_call():
    """The launch rule of residual_norm.cu over all widths and row counts reaches each kernel that it names."""
    import os
    import re
    src = open(os.path.join(os.path.dirname(binding.__file__), "csrc", "residual_norm.cu")).read()
    body = src[src.index("int launch_typed("):src.index("bool aligned(")]
    named = set(re.findall(r"launch_(warp|block)<TX, TY, ([\d, ]+)>", body))

    def rule(D, N, vec, sixteen, sms=148):
        up = lambda n: (n + 31) // 32 * 32  # noqa: E731
        if vec:
            nv, threads = D // 8, up((D // 8 + 1) // 2)
            if nv <= 64:
                return "warp", "8, 1" if nv <= 32 else "8, 2"
            if nv <= 512 and N * nv < sms * 1024:
                assert up(nv) <= 512
                return "block", "8, 1, 512"
            if sixteen and 128 < threads <= 320:
                return "block", "8, 2, 320, 4"
            assert threads <= 1024 and threads * 2 >= nv
            return "block", "8, 2, 512" if threads <= 512 else "8, 2, 1024"
        if D <= 256:
            return "warp", "1, 8"
        if D <= 4096:
            assert up((D + 7) // 8) <= 512
            return "block", "1, 8, 512"
        assert up((D + 15) // 16) <= (512 if D <= 8192 else 1024)
        return "block", "1, 16, 512" if D <= 8192 else "1, 16, 1024"

    for sixteen in (False, True):
        got = {rule(D, N, vec, sixteen) for D in range(1, 16385) for N in (1, 100000) for vec in ((False, True) if D % 8 == 0 else (False,))}
        assert got == (named if sixteen else named - {("block", "8, 2, 320, 4")})
