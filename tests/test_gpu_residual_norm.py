"""The norms around a residual branch on the GPU against the fp64 oracle.

fp32 results: the row sums are fp32 (relative error below D 2^-24 / 32 lanes, far
under 1e-5), everything else a handful of fp32 roundings: relative L2 1e-5.
16-bit results follow tests/parity.py (the oracle rounded to the type).
"""
import numpy as np
import pytest
import torch

import oracle
from linear_vision_backbone_b200 import binding, build
from tests.parity import assert_close

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    build.build()
    binding.load()


def make(N, D, xd, yd, seed, gate_rows=1):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return {"x": n(N, D).to(DT[xd]), "y": (n(N, D) * 0.7).to(DT[yd]), "post_w": 1 + 0.2 * n(D),
            "gate": n(N // gate_rows, D).to(DT[yd]), "res_scale": 0.5 * n(D), "pre_w": 1 + 0.2 * n(D)}


def run_both(d, use, xd, yd, what, **kw):
    d = {k: v for k, v in d.items() if k in ("x", "y") or k in use}
    c = {k: v.cuda() for k, v in d.items()}
    x_out = torch.empty_like(c["x"])
    post = "post_w" in use or kw.get("post_norm", False)
    pre = "pre_w" in use or kw.get("pre_norm", False)
    out = binding.residual_norm(c["x"], c["y"], x_out=x_out, **{k: c[k] for k in use}, **kw)
    ref_x, ref = oracle.residual_norm(d["x"], d["y"], post_norm=post, **{k: d[k] for k in use},
                                      **{k: v for k, v in kw.items() if k in ("gate_act", "alpha", "eps")}) \
        if "gate_act" in kw else oracle.residual_norm(d["x"], d["y"], post_norm=post, gate_act="sigmoid",
                                                      **{k: d[k] for k in use},
                                                      **{k: v for k, v in kw.items() if k in ("alpha", "eps")})
    torch.cuda.synchronize()
    assert torch.equal(c["x"].cpu(), d["x"]), "x is left alone"
    assert_close(x_out, ref_x, DT[xd], what + " x")
    assert (out is not None) == pre
    if pre:
        assert_close(out, ref, DT[yd], what + " out")
    # in place: the same bits
    binding.residual_norm(c["x"], c["y"], **{k: c[k] for k in use}, **kw)
    assert torch.equal(c["x"], x_out)


TYPES = [("f32", "f32"), ("f32", "f16"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "bf16")]
SIZES = [(1, 1), (3, 7), (2, 8), (5, 33), (300, 384), (7, 1000), (9, 1024), (2, 1032), (4, 2050), (3, 4096), (2, 5120),
         (1, 16383), (2, 16384)]


@pytest.mark.parametrize("N,D", SIZES)
@pytest.mark.parametrize("xd,yd", TYPES)
def test_every_part(N, D, xd, yd):
    d = make(N, D, xd, yd, seed=N + D)
    for use in ((), ("pre_w",), ("post_w",), ("gate",), ("res_scale", "pre_w"),
                ("post_w", "gate", "res_scale", "pre_w")):
        run_both(d, use, xd, yd, f"{N}x{D} {xd}/{yd} {use}")


@pytest.mark.parametrize("N,D", [(300, 4096), (600, 2056), (1200, 1032), (40, 8184)])
@pytest.mark.parametrize("xd,yd", [("f32", "f16"), ("bf16", "bf16")])
def test_many_rows(N, D, xd, yd):
    # two vectors a thread, whole and partly filled warps
    d = make(N, D, xd, yd, seed=N)
    run_both(d, ("post_w", "gate", "res_scale", "pre_w"), xd, yd, f"{N}x{D}", gate_act="silu", alpha=0.3)


def test_offsets_past_31_bits():
    # 2^31 + 16384 elements; the first and the last rows
    D = 16384
    N = (1 << 31) // D + 1
    x = torch.empty(N, D, device="cuda", dtype=torch.float16)
    y = torch.empty(N, D, device="cuda", dtype=torch.float16)
    gen = torch.Generator().manual_seed(9)
    rows = torch.tensor([0, 1, N - 2, N - 1])
    hx, hy = torch.randn(2, 4, D, generator=gen).half()
    x[rows.cuda()] = hx.cuda()
    y[rows.cuda()] = hy.cuda()
    out = binding.residual_norm(x, y, pre_norm=True)
    ref_x, ref = oracle.residual_norm(hx, hy)
    assert_close(x[rows.cuda()], ref_x, torch.float16, "x")
    assert_close(out[rows.cuda()], ref, torch.float16, "out")


@pytest.mark.parametrize("act", ["mul", "sigmoid", "silu"])
def test_gates_alpha_eps_and_norms_without_weights(act):
    d = make(20, 264, "f32", "bf16", seed=1)
    run_both(d, ("gate", "pre_w"), "f32", "bf16", act, gate_act=act, alpha=-0.25)
    run_both(d, ("gate",), "f32", "bf16", act, gate_act=act, post_norm=True, pre_norm=True, eps=1e-2)


@pytest.mark.parametrize("D", [48, 50])
def test_one_gate_row_for_a_sequence(D):
    d = make(24, D, "f16", "f16", seed=2, gate_rows=8)
    run_both(d, ("gate", "pre_w"), "f16", "f16", "gate rows", gate_act="silu")


def test_rows_at_odd_addresses():
    # element-aligned views: the 16-byte path does not apply
    d = make(6, 64, "f32", "bf16", seed=3)
    buf = torch.zeros(6 * 64 + 1, dtype=torch.bfloat16, device="cuda")
    y = buf[1:].view(6, 64)
    y.copy_(d["y"])
    x = d["x"].cuda()
    out = binding.residual_norm(x, y, pre_w=d["pre_w"].cuda())
    ref_x, ref = oracle.residual_norm(d["x"], d["y"], pre_w=d["pre_w"])
    assert_close(x, ref_x, torch.float32)
    assert_close(out, ref, torch.bfloat16)


def test_no_branch_zero_rows_and_large_rows():
    d = make(5, 96, "f32", "f16", seed=4)
    x = d["x"].cuda()
    out = binding.residual_norm(x, pre_w=d["pre_w"].cuda())
    assert out.dtype == torch.float32 and torch.equal(x.cpu(), d["x"])
    assert_close(out, oracle.residual_norm(d["x"], pre_w=d["pre_w"])[1], torch.float32)
    copy = torch.empty_like(x)
    assert binding.residual_norm(x, x_out=copy) is None and torch.equal(copy, x)
    # a zero row stays zero (0 / sqrt(eps)), and 16-bit rows at the type's largest values stay finite
    z = torch.zeros(2, 96, dtype=torch.float16, device="cuda")
    assert (binding.residual_norm(z, z.clone(), post_norm=True, pre_norm=True) == 0).all()
    big = torch.full((2, 96), 60000.0, dtype=torch.float16, device="cuda")
    out = binding.residual_norm(big, torch.zeros_like(big), pre_norm=True)
    assert_close(out, np.ones((2, 96)), torch.float16)
    assert binding.residual_norm(torch.empty(0, 64, device="cuda"), pre_norm=True).shape == (0, 64)


def test_non_finite_rows_stay_rows():
    d = make(10, 200, "f32", "bf16", seed=5)
    d["y"][4, 7] = float("inf")
    d["x"][8, 1] = float("nan")
    c = {k: v.cuda() for k, v in d.items()}
    out = binding.residual_norm(c["x"], c["y"], post_w=c["post_w"], gate=c["gate"], pre_w=c["pre_w"])
    keep = [0, 1, 2, 3, 5, 6, 7, 9]
    ref_x, ref = oracle.residual_norm(d["x"][keep], d["y"][keep], post_norm=True, post_w=d["post_w"],
                                      gate=d["gate"][keep], gate_act="sigmoid", pre_w=d["pre_w"])
    assert_close(c["x"][keep], ref_x, torch.float32)
    assert_close(out[keep], ref, torch.bfloat16)
    assert torch.isnan(out[4].float()).any() and torch.isnan(out[8].float()).all()


def test_captured_block_of_mixer_and_norms():
    """A mixer half as a user chains it: norm, projections, head-decay attention, output
    projection, norms around the branch; captured in a graph and replayed."""
    T, H, d, dm = 200, 4, 64, 256
    gen = torch.Generator().manual_seed(6)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = n(T, dm)
    w_in = (n(dm, 4 * H * d) / dm ** 0.5).bfloat16()
    w_out = (n(H * d, dm) / (H * d) ** 0.5).bfloat16()
    g = torch.nn.functional.logsigmoid(n(T, H)) / 16
    post_w, scale, pre_w = 1 + 0.2 * n(dm), 0.5 * n(dm), 1 + 0.2 * n(dm)
    c = [t.cuda() for t in (x, w_in, w_out, g, post_w, scale, pre_w)]
    xs = c[0].clone()

    def block():
        a = torch.empty(T, dm, dtype=torch.bfloat16, device="cuda")
        zero = torch.zeros(T, dm, dtype=torch.bfloat16, device="cuda")
        binding.residual_norm(xs, zero, pre_norm=True, out=a)
        q, k, v, z = binding.mixer_in_proj(a[None], c[1], H, d)
        y = binding.hla_fwd(q, k, v, c[3][None], z, scale=d ** -0.5)
        p = binding.mixer_out_proj(y.view(T, H * d), c[2])
        return a, binding.residual_norm(xs, p, post_w=c[4], res_scale=c[5], pre_w=c[6])
    block()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, out = block()
    xs.copy_(c[0])
    graph.replay()
    torch.cuda.synchronize()
    r16 = lambda t: torch.from_numpy(t).bfloat16()  # noqa: E731
    a_ref = r16(oracle.residual_norm(x, pre_w=None)[1])
    assert_close(a, a_ref.double().numpy(), torch.bfloat16, "first norm")
    a_ref = a.cpu()
    proj = [r16((a_ref.double() @ w.double()).numpy()).view(T, H, d) for w in w_in.split(H * d, 1)]
    y_ref = r16(oracle.hla_fwd(proj[0], proj[1], proj[2], g, proj[3], scale=d ** -0.5)[0])
    p_ref = r16((y_ref.view(T, H * d).double() @ w_out.double()).numpy())
    x_ref, out_ref = oracle.residual_norm(x, p_ref, post_norm=True, post_w=post_w, res_scale=scale, pre_w=pre_w)
    # three roundings to bf16 upstream (projections, y, p), each half a step 2^-9 of its row's scale and
    # partly averaged by the products: within 2^-7 of the result's norm
    for got, want in ((xs, x_ref), (out, out_ref)):
        e = np.linalg.norm(got.double().cpu().numpy() - want) / np.linalg.norm(want)
        assert e <= 2 ** -7, e


def test_binding_refuses_wrong_tensors():
    x = torch.zeros(4, 64, device="cuda")
    y = torch.zeros(4, 64, device="cuda", dtype=torch.float16)
    for kw in (dict(y=y[:3]), dict(y=y.t()), dict(y=y, gate=y.float()), dict(y=y, gate=y[:3]),
               dict(y=y, post_w=y[0]), dict(y=y, pre_w=x[0, :8]), dict(y=y, post_w=x[0], post_norm=False),
               dict(y=y, pre_w=x[0], pre_norm=False), dict(y=y.cpu()), dict(y=y, out=x)):
        with pytest.raises(ValueError):
            binding.residual_norm(x, **kw)
    with pytest.raises(KeyError):
        binding.residual_norm(x, y, gate=y, gate_act="tanh")
    with pytest.raises(binding.GtrError):
        binding.residual_norm(y, y.bfloat16())          # a 16-bit stream with another type's branch
    with pytest.raises(binding.GtrError):
        binding.residual_norm(x, y, x_out=x, out=None, gate=y, pre_norm=True, eps=-1.0)
