"""Head-decay linear attention on the GPU against the fp64 oracle.

Outputs follow the rules of tests/parity.py (fp32: relative L2 1e-5; 16-bit:
against the oracle rounded to the type).  Final states are fp32: the fp32
kernels round each operation (2^-24), and the tensor-core kernels carry at
least 16 significant bits of each inexact operand, an error of at most 2^-17 =
7.7e-6 of each term and so of the norm of their sum where terms do not cancel;
1e-5 relative L2 covers both.
"""
import numpy as np
import pytest
import torch

import oracle
from linear_vision_backbone_b200 import binding, build
from tests.parity import assert_close

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
STATE_REL = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_ok):
    build.build()
    binding.load()


def make(lens, H, Hk, dk, dv, dtype, *, seed, gated=True, per_head=False, div=16.0, lead=0, tail=0, states=False,
         mu=2.0):
    """Host inputs: `lead` and `tail` rows that belong to no sequence surround the sequences."""
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    T = lead + sum(lens) + tail
    dt = DT[dtype]
    d = {"q": n(T, Hk, dk).to(dt), "k": n(T, Hk, dk).to(dt), "v": n(T, H, dv).to(dt),
         "z": n(T, H, dv).to(dt) if gated else None, "w": 1 + 0.2 * n(dv) if gated else None,
         "g": torch.nn.functional.logsigmoid(n(*((H,) if per_head else (T, H))) + mu) / div,
         "S": n(len(lens), H, dk, dv) * 4 if states else None,
         "cu": (lead + torch.cumsum(torch.tensor([0] + list(lens)), 0)).to(torch.int32), "scale": dk ** -0.5}
    return d


def dev(d):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}


def reference(d):
    return oracle.hla_fwd(d["q"], d["k"], d["v"], d["g"], d["z"], d["w"], cu_seqlens=d["cu"], scale=d["scale"],
                          states=d["S"])


def check_states(got, want, what=""):
    got = got.double().cpu().numpy()
    assert np.all(np.isfinite(got)), what
    assert np.linalg.norm(got - want) <= STATE_REL * max(np.linalg.norm(want), 1e-30), \
        (what, np.linalg.norm(got - want) / np.linalg.norm(want))


def check(d, H, dtype, what):
    """One call with final states; the rows outside the sequences keep their mark."""
    c = dev(d)
    nseq = len(d["cu"]) - 1
    out = torch.full(d["v"].shape, 7.0, dtype=DT[dtype], device="cuda")
    fin = torch.full((nseq, H, d["q"].shape[2], d["v"].shape[2]), 5.0, device="cuda")
    binding.hla_fwd(c["q"], c["k"], c["v"], c["g"], c["z"], c["w"], cu_seqlens=c["cu"], scale=d["scale"],
                    state_in=c["S"], state_out=fin, out=out)
    torch.cuda.synchronize()
    ref, S = reference(d)
    a, b = int(d["cu"][0]), int(d["cu"][-1])
    assert (out[:a] == 7).all() and (out[b:] == 7).all(), what
    if b > a:
        assert_close(out[a:b], ref[a:b], DT[dtype], what)
    check_states(fin, S, what)
    rc, bits, _ = binding.device_status()
    assert rc == 0 and bits == 0, (what, rc, bits)


LENS = [[1], [2, 1, 3], [63, 64, 65], [127], [128], [129], [0, 5, 0, 200, 0], [385, 17, 256], [1100]]


@pytest.mark.parametrize("lens", LENS, ids=lambda v: "-".join(map(str, v)))
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
def test_prompt_16bit(lens, dtype, dk, dv):
    for gated, states in ((True, False), (False, True)):
        d = make(lens, 4, 2, dk, dv, dtype, seed=len(lens) + dk, gated=gated, states=states, lead=3, tail=2)
        check(d, 4, dtype, f"{lens} {dtype} {dk}x{dv} gated={gated}")


@pytest.mark.parametrize("lens", [[1], [0, 5, 0, 40], [129, 3], [700]], ids=lambda v: "-".join(map(str, v)))
@pytest.mark.parametrize("dtype,dk,dv", [("f32", 64, 64), ("f32", 128, 128), ("f32", 16, 32), ("f32", 32, 16),
                                         ("f16", 16, 16), ("bf16", 32, 128), ("bf16", 128, 16), ("f32", 64, 128)])
def test_prompt_cuda_core_shapes(lens, dtype, dk, dv):
    for gated, states in ((True, True), (False, False)):
        d = make(lens, 3, 3, dk, dv, dtype, seed=7 + dv, gated=gated, states=states, lead=1, tail=4)
        check(d, 3, dtype, f"{lens} {dtype} {dk}x{dv} gated={gated}")


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("div,mu", [(64.0, 2.0), (1.0, 2.0), (1.0, -3.0), (0.05, -3.0)])
def test_decays_from_slow_to_total(dtype, div, mu):
    # down to a mean log-decay of -60 per token: the state forgets everything at once
    d = make([300, 131], 2, 2, 64, 64, dtype, seed=11, div=div, mu=mu, states=True, gated=False)
    check(d, 2, dtype, f"div {div} mu {mu}")


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_zero_infinite_and_positive_log_decays(dtype):
    d = make([260], 2, 1, 64, 64, dtype, seed=12, gated=False, states=True)
    d["g"][:, 0] = 0.0                      # no decay at all
    d["g"][5::37, 1] = -float("inf")        # the state is reset at some tokens
    d["g"][7, 1] = -3e38
    check(d, 2, dtype, "infinite decays")
    e = dict(d, g=d["g"].clone())
    e["g"][9, 0] = 0.5                      # above zero counts as zero
    c = dev(e)
    got = binding.hla_fwd(c["q"], c["k"], c["v"], c["g"], cu_seqlens=c["cu"], scale=d["scale"], state_in=c["S"])
    c = dev(d)
    want = binding.hla_fwd(c["q"], c["k"], c["v"], c["g"], cu_seqlens=c["cu"], scale=d["scale"], state_in=c["S"])
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("H,Hk", [(1, 1), (6, 1), (6, 6), (8, 2)])
def test_head_groups_and_constant_decays(dtype, H, Hk):
    d = make([200, 77], H, Hk, 64, 64, dtype, seed=13, per_head=True)
    check(d, H, dtype, f"{H}/{Hk}")


@pytest.mark.parametrize("dtype,dk,dv", [("f16", 64, 64), ("bf16", 128, 128), ("f16", 128, 128), ("f32", 64, 64)])
def test_long_sequence_over_many_segments(dtype, dk, dv):
    d = make([9000, 333], 1, 1, dk, dv, dtype, seed=14, div=64.0, states=True)
    check(d, 1, dtype, "long")


@pytest.mark.parametrize("dtype,dk,dv", [("f16", 64, 64), ("bf16", 128, 128), ("f32", 32, 16)])
def test_states_in_place_over_many_segments(dtype, dk, dv):
    # a sequence's last segment may finish before its first one starts
    d = make([12000, 50, 7000], 1, 1, dk, dv, dtype, seed=30, div=64.0, states=True)
    c = dev(d)
    ref, S = reference(d)
    for _ in range(5):
        pool = c["S"].clone()
        out = binding.hla_fwd(c["q"], c["k"], c["v"], c["g"], c["z"], c["w"], cu_seqlens=c["cu"], scale=d["scale"],
                              state_in=pool, state_out=pool)
        assert_close(out, ref, DT[dtype], "in place")
        check_states(pool, S)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", [1e-3, 300.0])
def test_small_and_large_values(dtype, size):
    # states and scores far outside fp16's range or near its smallest numbers;
    # the norm brings the outputs back
    d = make([300], 2, 2, 64, 64, dtype, seed=15, div=64.0)
    for n in ("q", "k", "v"):
        d[n] = (d[n].float() * size).to(DT[dtype])
    d["scale"] = 1.0 if size > 1 else 1e6
    check(d, 2, dtype, f"size {size}")


@pytest.mark.parametrize("dtype,dk", [("bf16", 64), ("f16", 128), ("f32", 64)])
def test_output_between_the_inputs_columns(dtype, dk):
    # v, out and z as column blocks of one buffer, in this order
    d = make([150, 33], 4, 2, dk, dk, dtype, seed=31)
    c = dev(d)
    want = binding.hla_fwd(c["q"], c["k"], c["v"], c["g"], c["z"], c["w"], cu_seqlens=c["cu"], scale=d["scale"])
    T = c["v"].shape[0]
    buf = torch.full((T, 4 * dk * 3), 7.0, device="cuda", dtype=DT[dtype])
    v, out, z = (buf[:, i * 4 * dk:(i + 1) * 4 * dk].unflatten(1, (4, dk)) for i in range(3))
    v.copy_(c["v"])
    z.copy_(c["z"])
    got = binding.hla_fwd(c["q"], c["k"], v, c["g"], z, c["w"], cu_seqlens=c["cu"], scale=d["scale"], out=out)
    assert got.data_ptr() == out.data_ptr()
    assert torch.equal(out, want) and torch.equal(v, c["v"]) and torch.equal(z, c["z"])
    with pytest.raises(binding.GtrError):
        binding.hla_fwd(c["q"], c["k"], v, c["g"], z, c["w"], cu_seqlens=c["cu"], scale=d["scale"], out=z)


@pytest.mark.parametrize("dtype,dk,dv", [("f16", 64, 64), ("bf16", 128, 128), ("f32", 64, 32)])
def test_non_finite_rows_stay_in_their_sequence_and_head(dtype, dk, dv):
    d = make([70, 130, 60], 2, 2, dk, dv, dtype, seed=16, lead=5, tail=9, gated=False)
    clean = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in d.items()}
    bad = float("nan")
    for n in ("q", "k", "v"):
        d[n][:5] = bad                        # rows outside the sequences
        d[n][-9:] = float("inf")
        d[n][75 + 20, 1] = bad                # a token of sequence 1, head 1
    d["g"][:5] = bad
    d["g"][-9:] = bad
    c = dev(d)
    fin = torch.zeros(3, 2, dk, dv, device="cuda")
    out = binding.hla_fwd(c["q"], c["k"], c["v"], c["g"], cu_seqlens=c["cu"], scale=d["scale"], state_out=fin)
    ref, S = reference(clean)
    for a, b, h in ((5, 75, 0), (5, 75, 1), (75, 205, 0), (205, 265, 0), (205, 265, 1)):
        assert_close(out[a:b, h], ref[a:b, h], DT[dtype], f"rows {a}..{b} head {h}")
    assert torch.isnan(out[95:205, 1].float()).all()     # the token itself and what follows
    check_states(fin[[0, 0, 1, 2, 2], [0, 1, 0, 0, 1]], S[[0, 0, 1, 2, 2], [0, 1, 0, 0, 1]])
    assert torch.isnan(fin[1, 1]).any()


@pytest.mark.parametrize("dtype,dk,dv", [("f16", 64, 64), ("bf16", 128, 128), ("f32", 32, 64)])
def test_slots_seen_and_skipped_sequences(dtype, dk, dv):
    lens, H = [40, 150, 1, 0, 64, 33], 2
    d = make(lens, H, 1, dk, dv, dtype, seed=17, states=True)
    slots = torch.tensor([7, 2, -1, 4, 0, 5], dtype=torch.int32)
    seen = torch.tensor([3, 0, 9, 2, 1, -4], dtype=torch.int32)
    pool = torch.randn(9, H, dk, dv, generator=torch.Generator().manual_seed(3))
    starts = torch.stack([pool[s] if s >= 0 and n > 0 else torch.zeros(H, dk, dv)
                          for s, n in zip(slots.tolist(), seen.tolist())])
    ref, S = reference(dict(d, S=starts))
    c = dev(d)
    for in_place in (True, False):
        src = pool.cuda()
        dst = src if in_place else torch.full_like(src, 3.0)
        out = torch.full_like(c["v"], 7.0)
        binding.hla_fwd(c["q"], c["k"], c["v"], c["g"], c["z"], c["w"], cu_seqlens=c["cu"], scale=d["scale"],
                        state_in=src, state_out=dst, slots=slots.cuda(), seen=seen.cuda(), out=out)
        for n, (s, length) in enumerate(zip(slots.tolist(), lens)):
            a, b = int(d["cu"][n]), int(d["cu"][n + 1])
            if s < 0:
                assert (out[a:b] == 7).all()
                continue
            if length:
                assert_close(out[a:b], ref[a:b], DT[dtype], f"sequence {n}")
            check_states(dst[s], S[n], f"state {n}")
        for s in set(range(9)) - set(slots.tolist()):      # states of no sequence
            assert torch.equal(dst[s].cpu(), pool[s] if in_place else torch.full_like(pool[s], 3.0))
    assert binding.device_status()[0] == 0
    # a slot outside the pool: skipped, and recorded
    bad = slots.clone()
    bad[1] = 9
    out = torch.full_like(c["v"], 7.0)
    dst = pool.cuda()
    binding.hla_fwd(c["q"], c["k"], c["v"], c["g"], c["z"], c["w"], cu_seqlens=c["cu"], scale=d["scale"],
                    state_in=dst, state_out=dst, slots=bad.cuda(), out=out)
    rc, bits, _ = binding.device_status()
    assert rc == -6 and bits == 16
    assert (out[40:190] == 7).all() and torch.equal(dst[2].cpu(), pool[2])
    assert binding.device_status()[0] == 0


@pytest.mark.parametrize("dtype,dk,dv", [("f16", 64, 64), ("bf16", 64, 128), ("f32", 16, 16)])
def test_column_blocks_of_one_projection(dtype, dk, dv):
    H, Hk, T = 4, 2, 190
    d = make([T], H, Hk, dk, dv, dtype, seed=18)
    width = 2 * Hk * dk + 2 * H * dv + 16
    block = torch.full((T, width), float("nan"), dtype=DT[dtype])
    views, at = {}, 8
    for n, heads, w in (("q", Hk, dk), ("k", Hk, dk), ("v", H, dv), ("z", H, dv)):
        block[:, at:at + heads * w] = d[n].reshape(T, -1)
        views[n] = (at, heads, w)
        at += heads * w
    b = block.cuda()
    c = {n: b[:, a:a + h * w].unflatten(1, (h, w)) for n, (a, h, w) in views.items()}
    outs = torch.full((T, H * dv + 8), 7.0, dtype=DT[dtype], device="cuda")
    o = outs[:, 8:].unflatten(1, (H, dv))
    binding.hla_fwd(c["q"], c["k"], c["v"], d["g"].cuda(), c["z"], d["w"].cuda(), scale=d["scale"], out=o)
    ref, _ = reference(d)
    assert_close(o, ref, DT[dtype], "strided")
    assert (outs[:, :8] == 7).all()


def test_batched_tensors_are_sequences():
    d = make([50, 50, 50], 2, 2, 64, 64, "bf16", seed=19, states=True)
    c = dev(d)
    ref, S = reference(d)
    v4 = {n: c[n].view(3, 50, *c[n].shape[1:]) for n in ("q", "k", "v", "z", "g")}
    fin = torch.empty_like(c["S"])
    out = binding.hla_fwd(v4["q"], v4["k"], v4["v"], v4["g"], v4["z"], c["w"], scale=d["scale"], state_in=c["S"],
                          state_out=fin)
    assert out.shape == (3, 50, 2, 64)
    assert_close(out.reshape(150, 2, 64), ref, torch.bfloat16)
    check_states(fin, S)
    # many equal sequences of several segments each
    d = make([700] * 2, 1, 1, 64, 64, "f16", seed=20)
    c = dev(d)
    v4 = {n: c[n].view(2, 700, *c[n].shape[1:]) for n in ("q", "k", "v", "z", "g")}
    out = binding.hla_fwd(v4["q"], v4["k"], v4["v"], v4["g"], v4["z"], c["w"], scale=d["scale"])
    assert_close(out.reshape(1400, 1, 64), reference(d)[0], torch.float16)


# ------------------------------------------------------------- single tokens
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128), (128, 64), (16, 16), (32, 64), (16, 128),
                                   (128, 16)])
def test_step(dtype, dk, dv):
    for N, H, Hk, gated, per_head in ((1, 1, 1, True, False), (5, 4, 2, False, True), (33, 6, 6, True, False)):
        d = make([1] * N, H, Hk, dk, dv, dtype, seed=N + dk, gated=gated, per_head=per_head, states=True)
        ref, S = reference(d)
        c = dev(d)
        slots = torch.randperm(N + 3, generator=torch.Generator().manual_seed(N))[:N].to(torch.int32)
        pool = torch.full((N + 3, H, dk, dv), 2.0)
        pool[slots.long()] = d["S"]
        src = pool.cuda()
        out = binding.hla_step(c["q"], c["k"], c["v"], c["g"], src, c["z"], c["w"], slots=slots.cuda(),
                               scale=d["scale"])
        assert_close(out, ref, DT[dtype], f"{N} {H}/{Hk}")
        check_states(src[slots.long().cuda()], S)
        free = [s for s in range(N + 3) if s not in slots.tolist()]
        assert (src[free] == 2).all()
        # into another pool, identity slots
        dst = torch.zeros(N, H, dk, dv, device="cuda")
        again = binding.hla_step(c["q"], c["k"], c["v"], c["g"], c["S"], c["z"], c["w"], scale=d["scale"],
                                 state_out=dst)
        assert torch.equal(again, out)
        check_states(dst, S)


def test_step_skips_padding_rows_and_bad_slots():
    d = make([1] * 6, 2, 2, 64, 64, "bf16", seed=21, states=True)
    c = dev(d)
    slots = torch.tensor([4, -1, 0, 6, -7, 2], dtype=torch.int32)
    pool = torch.randn(6, 2, 64, 64, device="cuda")
    before = pool.clone()
    out = torch.full_like(c["v"], 7.0)
    binding.hla_step(c["q"], c["k"], c["v"], c["g"], pool, c["z"], c["w"], slots=slots.cuda(), out=out)
    rc, bits, _ = binding.device_status()
    assert rc == -6 and bits == 16                  # slot 6 of 6
    assert (out[[1, 3, 4]] == 7).all() and not (out[[0, 2, 5]] == 7).all()
    assert torch.equal(pool[[1, 3, 5]], before[[1, 3, 5]])
    assert not torch.equal(pool[[4, 0, 2]], before[[4, 0, 2]])


@pytest.mark.parametrize("dtype,dk,dv", [("f16", 64, 64), ("bf16", 128, 128), ("f32", 64, 64)])
def test_prompt_then_steps_equal_one_prompt(dtype, dk, dv):
    """A prompt, a second prompt on its states, then token by token: the states and the
    outputs are those of the whole sequences at once."""
    lens, H, Hk = [150, 41], 4, 2
    d = make(lens, H, Hk, dk, dv, dtype, seed=22)
    ref, S = reference(d)
    c = dev(d)
    pool = torch.full((3, H, dk, dv), float("nan"), device="cuda")
    slots = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    at = [int(x) for x in d["cu"]]
    cuts = [(0, 100, 130, 150), (0, 30, 38, 41)]
    got = torch.empty_like(c["v"])
    seen = torch.zeros(2, dtype=torch.int32, device="cuda")
    for part in range(2):
        rows = [range(at[n] + cuts[n][part], at[n] + cuts[n][part + 1]) for n in range(2)]
        idx = torch.tensor([r for rr in rows for r in rr], device="cuda")
        cu = torch.tensor([0, len(rows[0]), len(rows[0]) + len(rows[1])], dtype=torch.int32, device="cuda")
        got[idx] = binding.hla_fwd(c["q"][idx], c["k"][idx], c["v"][idx], c["g"][idx], c["z"][idx], c["w"],
                                   cu_seqlens=cu, scale=d["scale"], state_in=pool, state_out=pool, slots=slots,
                                   seen=seen)
        seen += cu[1:] - cu[:-1]
    for t in range(20):
        rows = torch.tensor([at[0] + 130 + t, at[1] + min(38 + t, 40)], device="cuda")
        live = torch.tensor([2, 0 if t < 3 else -1], dtype=torch.int32, device="cuda")   # the second ends earlier
        step = binding.hla_step(c["q"][rows], c["k"][rows], c["v"][rows], c["g"][rows], pool, c["z"][rows], c["w"],
                                slots=live, scale=d["scale"])
        got[rows[0]] = step[0]
        if t < 3:
            got[rows[1]] = step[1]
    assert_close(got, ref, DT[dtype], "prompt, prompt, steps")
    check_states(pool[[2, 0]], S)
    assert torch.isnan(pool[1]).all()


@pytest.mark.parametrize("dtype,dk", [("bf16", 64), ("f16", 128), ("f32", 64)])
def test_offsets_past_31_bits(dtype, dk):
    # 70 rows 2^25 elements apart, and states behind 2^31 elements of a pool
    d = make([40, 29], 2, 2, dk, dk, dtype, seed=32, states=True)
    c = dev(d)
    T, w = 69, 2 * dk
    buf = torch.empty(T, 1 << 25, device="cuda", dtype=DT[dtype])
    q, k, v, z, out = (buf[:, i * w:(i + 1) * w].unflatten(1, (2, dk)) for i in range(5))
    for n, t in (("q", q), ("k", k), ("v", v), ("z", z)):
        t.copy_(c[n])
    far = (1 << 31) // (2 * dk * dk) + 1
    pool = torch.empty(far + 1, 2, dk, dk, device="cuda")
    slots = torch.tensor([far, 3], dtype=torch.int32, device="cuda")
    pool[slots.long()] = c["S"]
    binding.hla_fwd(q, k, v, c["g"], z, c["w"], cu_seqlens=c["cu"], scale=d["scale"], state_in=pool, state_out=pool,
                    slots=slots, out=out)
    ref, S = reference(d)
    assert_close(out, ref, DT[dtype], "far rows")
    check_states(pool[slots.long()], S)
    rows = slice(T - 2, T)                    # the last two rows, a token of each state
    one = dict(d, cu=torch.tensor([0, 1, 2], dtype=torch.int32), S=torch.from_numpy(S),
               **{n: d[n][rows] for n in ("q", "k", "v", "z", "g")})
    binding.hla_step(q[rows], k[rows], v[rows], c["g"][rows], pool, z[rows], c["w"], scale=d["scale"], slots=slots,
                     out=out[rows])
    ref, S = reference(one)
    assert_close(out[rows], ref, DT[dtype], "far rows, step")
    check_states(pool[slots.long()], S)


def test_sequences_without_a_token_only():
    # rows, but every sequence is empty: no row is written, the states are the initial ones
    for dtype, dk in (("bf16", 64), ("f16", 128), ("f32", 64)):
        d = make([70], 2, 2, dk, dk, dtype, seed=33)
        c = dev(d)
        S = torch.randn(3, 2, dk, dk, device="cuda")
        fin = torch.zeros_like(S)
        out = torch.full_like(c["v"], 7.0)
        cu = torch.tensor([5, 5, 5, 5], dtype=torch.int32, device="cuda")
        seen = torch.tensor([1, 0, 4], dtype=torch.int32, device="cuda")
        binding.hla_fwd(c["q"], c["k"], c["v"], c["g"], c["z"], c["w"], cu_seqlens=cu, scale=d["scale"], state_in=S,
                        state_out=fin, seen=seen, out=out)
        assert (out == 7).all()
        assert torch.equal(fin[[0, 2]], S[[0, 2]]) and (fin[1] == 0).all()


# ------------------------------------------------- streams, graphs, repetition
@pytest.mark.parametrize("dtype,dk,dv", [("f16", 64, 64), ("bf16", 128, 128), ("f32", 64, 64)])
def test_captured_and_replayed_on_new_inputs(dtype, dk, dv):
    H = 2
    a = make([1400, 70, 300], H, 1, dk, dv, dtype, seed=23, states=True)
    b = make([20, 1500, 250], H, 1, dk, dv, dtype, seed=24, states=True)     # other lengths, the same rows
    c = dev(a)
    fin = torch.empty_like(c["S"])
    out = torch.empty_like(c["v"])
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call = lambda: binding.hla_fwd(c["q"], c["k"], c["v"], c["g"], c["z"], c["w"], cu_seqlens=c["cu"],  # noqa: E731
                                       scale=a["scale"], state_in=c["S"], state_out=fin, out=out)
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
            binding.hla_step(c["q"][:3], c["k"][:3], c["v"][:3], c["g"][:3], fin, c["z"][:3], c["w"],
                             scale=a["scale"])
    for d in (a, b, a):
        for n, t in dev(d).items():
            if isinstance(t, torch.Tensor):
                c[n].copy_(t)
        out.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ref, S = reference(d)
        assert_close(out, ref, DT[dtype], "replayed")
        first = dict(d, cu=torch.tensor([0, 1, 2, 3], dtype=torch.int32), S=torch.from_numpy(S))
        for n in ("q", "k", "v", "z", "g"):
            first[n] = d[n][:3]
        check_states(fin, reference(first)[1], "stepped state")


def test_two_calls_at_once_and_a_stream_of_the_callers():
    d1 = make([3000], 2, 2, 64, 64, "f16", seed=25)
    d2 = make([2900, 40], 2, 2, 64, 64, "bf16", seed=26)
    c1, c2 = dev(d1), dev(d2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(8):
        o1 = binding.hla_fwd(c1["q"], c1["k"], c1["v"], c1["g"], c1["z"], c1["w"], scale=d1["scale"], stream=s1)
        o2 = binding.hla_fwd(c2["q"], c2["k"], c2["v"], c2["g"], c2["z"], c2["w"], cu_seqlens=c2["cu"],
                             scale=d2["scale"], stream=s2)
        outs.append((o1, o2))
    torch.cuda.synchronize()
    assert_close(outs[0][0], reference(d1)[0], torch.float16)
    assert_close(outs[0][1], reference(d2)[0], torch.bfloat16)
    for o1, o2 in outs[1:]:                     # and the same bits every time
        assert torch.equal(o1, outs[0][0]) and torch.equal(o2, outs[0][1])


def test_binding_refuses_wrong_tensors():
    d = dev(make([8], 4, 2, 64, 64, "f16", seed=27, states=True))
    ok = dict(q=d["q"], k=d["k"], v=d["v"], g=d["g"])
    for name, bad in (("k", d["k"].bfloat16()), ("k", d["k"][:7]), ("v", d["v"][..., :32]), ("g", d["g"].double()),
                      ("g", d["g"][:, :2]), ("q", d["q"].double()), ("q", d["q"].transpose(0, 1)),
                      ("k", d["k"].cpu())):
        with pytest.raises(ValueError):
            binding.hla_fwd(**dict(ok, **{name: bad}))
    for kw in (dict(w=d["w"]), dict(z=d["z"], w=d["w"][:8]), dict(cu_seqlens=d["cu"].long()),
               dict(state_in=d["S"].half()), dict(state_in=d["S"][:, :2]), dict(state_in=d["S"], state_out=d["S"][:0]),
               dict(slots=torch.zeros(2, dtype=torch.int32, device="cuda")),
               dict(cu_seqlens=torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda"), state_in=d["S"]),
               dict(out=torch.empty(8, 4, 64, device="cuda"))):
        with pytest.raises(ValueError):
            binding.hla_fwd(**ok, **kw)
    with pytest.raises(binding.GtrError):         # head dims the kernels do not have
        binding.hla_fwd(*(torch.zeros(4, 2, 48, device="cuda", dtype=torch.float16) for _ in range(3)),
                        torch.zeros(4, 2, device="cuda"))
    with pytest.raises(ValueError):
        binding.hla_step(d["q"], d["k"], d["v"], d["g"], d["S"])    # 8 rows, one state


def test_empty_calls():
    e = torch.empty(0, 2, 64, device="cuda", dtype=torch.float16)
    g = torch.empty(0, 2, device="cuda")
    S = torch.randn(2, 2, 64, 64, device="cuda")
    assert binding.hla_fwd(e, e, e, g).shape == (0, 2, 64)
    fin = torch.zeros_like(S)
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    binding.hla_fwd(e, e, e, g, cu_seqlens=cu, state_in=S, state_out=fin)
    assert torch.equal(fin, S)                    # two sequences of length zero
    assert binding.hla_step(e, e, e, g, S).shape == (0, 2, 64)
    torch.cuda.synchronize()
