"""Head-decay linear attention and residual norm without a GPU: the oracle against
other forms, the refusals of the C ABI and of the binding, the segment arithmetic."""
import ctypes
import random

import numpy as np
import pytest
import torch

import oracle
from linear_vision_backbone_b200 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


# ------------------------------------------------------------------- oracle
def test_oracle_hla_equals_the_quadratic_form():
    rng = np.random.default_rng(0)
    T, Hk, H, dk, dv = 23, 2, 4, 5, 7
    q, k = rng.normal(size=(2, T, Hk, dk))
    v = rng.normal(size=(T, H, dv))
    g = -rng.random((T, H))
    S0 = rng.normal(size=(2, H, dk, dv))
    cu = [2, 11, 20]                      # rows 0, 1 and 20.. belong to no sequence
    out, final = oracle.hla_fwd(q, k, v, g, cu_seqlens=cu, scale=0.3, states=S0)
    assert np.isnan(out[:2]).all() and np.isnan(out[20:]).all()
    for n in range(2):
        a, b = cu[n], cu[n + 1]
        for h in range(H):
            G = np.cumsum(g[a:b, h])
            D = np.tril(np.exp(G[:, None] - G[None, :]))
            want = 0.3 * ((q[a:b, h // 2] @ k[a:b, h // 2].T * D) @ v[a:b, h]
                          + np.exp(G)[:, None] * (q[a:b, h // 2] @ S0[n, h]))
            np.testing.assert_allclose(out[a:b, h], want, rtol=1e-12, atol=1e-12)
            S = np.exp(G[-1]) * S0[n, h] + (k[a:b, h // 2] * np.exp(G[-1] - G)[:, None]).T @ v[a:b, h]
            np.testing.assert_allclose(final[n, h], S, rtol=1e-12, atol=1e-12)


def test_oracle_hla_equals_the_key_decay_oracle_with_equal_decays():
    rng = np.random.default_rng(1)
    T, H, d = 12, 2, 16
    q, k, v, z = rng.normal(size=(4, 1, T, H, d))
    g = -rng.random((1, T, H))
    f = torch.from_numpy
    full = oracle.gla_fwd(f(q).float(), f(k).float(), f(v).float(), f(np.repeat(g[..., None], d, -1)).float(),
                          f(z).float(), None, gh=3, gw=4, direction="LR")
    t32 = lambda a: a[0].astype(np.float32)  # noqa: E731
    out, _ = oracle.hla_fwd(t32(q), t32(k), t32(v), t32(g), t32(z))
    np.testing.assert_allclose(out, np.asarray(full)[0], rtol=1e-6, atol=1e-6)


def test_oracle_residual_norm_equals_torch():
    g = torch.Generator().manual_seed(2)
    x, y = torch.randn(2, 6, 10, generator=g, dtype=torch.float64)
    w1, w2, s = torch.randn(3, 10, generator=g, dtype=torch.float64)
    gate = torch.randn(3, 10, generator=g, dtype=torch.float64)
    xo, out = oracle.residual_norm(x, y, post_norm=True, post_w=w1, gate=gate, gate_act="silu", res_scale=s, alpha=0.5,
                                   pre_w=w2)
    rms = lambda t, w: torch.nn.functional.rms_norm(t, (10,), w, 1e-5)  # noqa: E731
    want = x + 0.5 * s * rms(y, w1) * torch.nn.functional.silu(gate.repeat_interleave(2, 0))
    np.testing.assert_allclose(xo, want.numpy(), rtol=1e-12)
    np.testing.assert_allclose(out, rms(want, w2).numpy(), rtol=1e-12)


# ----------------------------------------------------------------- refusals
FIELDS = ["q", "k", "v", "g", "outgate", "rms_w", "out", "state_in", "state_out", "slots", "seen", "cu_seqlens",
          "workspace", "workspace_bytes", "ldq", "ldk", "ldv", "ldz", "ldo", "nseq", "T", "Hk", "H", "dk", "dv",
          "nslots", "g_per_head", "dtype", "scale"]


def hla_args(**kw):
    a = dict(q=4096, k=4096, v=4096, g=4096, outgate=0, rms_w=0, out=4096, state_in=0, state_out=0, slots=0, seen=0,
             cu_seqlens=0, workspace=0, workspace_bytes=0, ldq=0, ldk=0, ldv=0, ldz=0, ldo=0, nseq=1, T=4, Hk=2, H=4,
             dk=64, dv=64, nslots=0, g_per_head=0, dtype=1, scale=1.0)
    a.update(kw)
    return binding._HLA_ARGS.pack(*[a[n] for n in FIELDS])


def test_hla_fwd_rejects_invalid_arguments_before_any_launch(lib):
    call = lambda **kw: lib.gtr_hla_fwd(hla_args(**kw), None)  # noqa: E731
    assert lib.gtr_hla_fwd(None, None) == -1
    assert call(dtype=3) == -1
    assert call(nseq=-1) == -1 and call(T=-1) == -1 and call(H=-1) == -1 and call(nslots=-1) == -1
    assert call(dk=48) == -2 and call(dv=256) == -2
    assert call(Hk=3) == -1 and call(Hk=0) == -1          # key heads must divide the heads
    assert call(H=131072, Hk=1) == -2
    assert call(nseq=3) == -1                             # equal sequences: nseq divides T
    for name in ("q", "k", "v", "g", "out"):
        assert call(**{name: 0}) == -1, name
    assert call(rms_w=4096) == -1                         # a norm weight without a gate
    assert call(state_in=4096, nslots=0) == -1            # a state per sequence
    assert call(state_out=4096, nslots=0) == -1
    assert call(state_in=1 << 20, state_out=(1 << 20) + 1024, nslots=1) == -1   # overlapping states
    assert call(ldq=64) == -1                             # a pitch below the heads' width
    assert call(ldv=260) == -3 and call(ldk=2 * 64 + 4) == -3   # pitch not a multiple of 16 bytes
    assert call(ldo=1 << 40) == -1
    for name in ("q", "k", "v", "outgate", "out", "workspace"):
        assert call(**{name: 4104}) == -3, name
    assert call(g=4098) == -3 and call(cu_seqlens=4097) == -3
    # empty problems: pointers unused
    assert call(nseq=0) == 0 and call(H=0, Hk=0) == 0
    assert call(T=0, q=0, k=0, v=0, g=0, out=0) == 0


@pytest.mark.parametrize("kw", [
    dict(q=1 << 20), dict(k=(1 << 20) + 1024 - 16), dict(v=(1 << 20) - 16), dict(outgate=1 << 20),
    dict(g=(1 << 20) + 4), dict(state_in=(1 << 20) + 16, nslots=1),
    dict(state_out=(1 << 20) - 65536 + 16, nslots=1),   # of 65536 bytes
    dict(v=(1 << 20) + 256, ldv=512, ldo=512),            # columns 128 .. 383 on 0 .. 255
    dict(v=(1 << 20) + 768, ldv=512, ldo=512),            # columns 384 .. 511 and the next row's 0 .. 127
    dict(q=(1 << 20) + 512, ldq=256, ldo=512),            # other pitches: whole ranges count
])
def test_hla_output_over_an_input_is_refused(lib, kw):
    # q, k: 2 heads, v, g, out: 4 heads, 4 tokens, bf16
    ptrs = {n: (i + 2) << 24 for i, n in enumerate(["q", "k", "v", "g"])}
    assert lib.gtr_hla_fwd(hla_args(**{**ptrs, "out": 1 << 20, **kw}), None) == -1
    if "ldv" not in kw and "ldq" not in kw:               # the same for single tokens: four rows, dense
        step = {"state_in": 1 << 27, "state_out": 1 << 27, "nslots": 4, "nseq": 4}
        kw = {n: a for n, a in kw.items() if n != "nslots"}
        if "state_in" in kw:
            kw["state_out"] = kw["state_in"]
        if "state_out" in kw:
            kw["state_in"] = kw["state_out"]
        assert lib.gtr_hla_step(hla_args(**{**ptrs, "out": 1 << 20, **step, **kw}), None) == -1


def test_hla_step_rejects_invalid_arguments_before_any_launch(lib):
    def call(**kw):
        return lib.gtr_hla_step(hla_args(**dict(dict(nseq=4, state_in=1 << 20, state_out=1 << 20, nslots=4), **kw)),
                                None)
    assert call(nseq=3) == -1                             # one row per sequence
    assert call(cu_seqlens=4096) == -1 and call(seen=4096) == -1
    assert call(state_in=0) == -1 and call(state_out=0) == -1
    assert call(nslots=3) == -1
    assert call(dk=8) == -2
    assert call(state_in=(1 << 20) + 8) == -3
    assert call(nseq=0, T=0) == 0


def test_hla_workspace_size(lib):
    ws = lib.gtr_hla_workspace_bytes
    bad = ctypes.c_size_t(-1).value
    assert ws(-1, 4, 4, 64, 64, 1) == bad and ws(1, 4, 4, 48, 64, 1) == bad and ws(1, 4, 4, 64, 64, 7) == bad
    assert ws(0, 4, 4, 64, 64, 1) == 0 and ws(1, 0, 4, 64, 64, 1) == 0 and ws(1, 4, 0, 64, 64, 1) == 0


def test_residual_norm_rejects_invalid_arguments_before_any_launch(lib):
    base = dict(x=1 << 20, x_out=1 << 20, y=2 << 20, post_w=0, gate=0, res_scale=0, pre_w=0, out=3 << 20, N=4,
                gate_rows=1, D=64, x_dtype=0, dtype=1, post_norm=0, gate_act=0, alpha=1.0, eps=1e-5)

    def call(**kw):
        return lib.gtr_residual_norm(binding._NORM_ARGS.pack(*dict(base, **kw).values()), None)
    assert lib.gtr_residual_norm(None, None) == -1
    assert call(x_dtype=5) == -1 and call(dtype=-1) == -1
    assert call(N=-1) == -1 and call(D=-1) == -1 and call(N=1 << 32) == -1
    assert call(D=0) == -2 and call(D=16385) == -2
    assert call(x_dtype=1, dtype=2) == -2                 # a 16-bit stream has its branch's type
    assert call(gate_act=3) == -1
    assert call(eps=-1.0) == -1 and call(eps=float("nan")) == -1
    assert call(x=0) == -1 and call(x_out=0) == -1
    assert call(post_w=4 << 20) == -1                     # a weight without its norm
    assert call(pre_w=4 << 20, out=0) == -1
    assert call(y=0, post_norm=1) == -1 and call(y=0, gate=4 << 20) == -1 and call(y=0, res_scale=4 << 20) == -1
    assert call(gate=4 << 20, gate_rows=3) == -1 and call(gate=4 << 20, gate_rows=0) == -1
    assert call(x=(1 << 20) + 2, x_out=(1 << 20) + 2) == -3 and call(y=(2 << 20) + 1) == -3
    assert call(x_out=(1 << 20) + 256) == -1              # x_out over part of x
    assert call(out=1 << 20) == -1 and call(out=2 << 20) == -1
    assert call(gate=3 << 20) == -1                       # out over the gate
    assert call(N=0, x=0, x_out=0) == 0


def test_binding_refuses_what_is_not_a_cuda_tensor():
    t = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError, match="q must be"):
        binding.hla_fwd(t, t, t, torch.zeros(4, 2))
    with pytest.raises(ValueError, match="q must be"):
        binding.hla_step(t, t, t, torch.zeros(4, 2), torch.zeros(4, 2, 64, 64))
    with pytest.raises(ValueError, match="state_in"):
        binding.hla_step(t, t, t, torch.zeros(4, 2), None)
    with pytest.raises(ValueError, match="x must be"):
        binding.residual_norm(torch.zeros(4, 64))


def test_argument_structs_have_the_headers_sizes(tmp_path):
    import subprocess
    src = tmp_path / "s.c"
    src.write_text(f'#include "{build.INCLUDE}/gtr_gla.h"\n#include <stdio.h>\n'
                   'int main(void) { printf("%zu %zu %zu", sizeof(gtr_hla_args), offsetof(gtr_hla_args, nseq),'
                   ' sizeof(gtr_residual_norm_args)); }\n')
    subprocess.run(["gcc", str(src), "-o", str(tmp_path / "s")], check=True)
    size, nseq, norm = map(int, subprocess.run([str(tmp_path / "s")], check=True, capture_output=True).stdout.split())
    assert size == binding._HLA_ARGS.size
    # C pads the struct to its 8-byte alignment
    assert norm == -(-binding._NORM_ARGS.size // 8) * 8
    assert nseq == 13 * 8 + 8 + 5 * 8


# --------------------------------------------------- the split of the work
def _ranges(lens, H, C, groups):
    """The kernels' arithmetic (hla_common.cuh): the parts of every group and the cuts."""
    nb = [-(-n // C) for n in lens]
    B = H * sum(n + 1 for n in nb)
    J = min(groups, B)
    starts, x = [], 0                               # first unit of each sequence
    for n in nb:
        starts.append(x)
        x += (n + 1) * H
    at = lambda x: (max(i for i, s in enumerate(starts) if s <= x),)  # noqa: E731
    start = lambda j: B if j >= J else B // J * j + min(j, B % J)  # noqa: E731
    parts, cuts = [], []
    for j in range(groups):
        x0, x1 = start(j), start(j + 1)
        mine, x = [], x0
        while x < x1:
            n, = at(x)
            h, b0 = divmod(x - starts[n], nb[n] + 1)
            units = min(nb[n] + 1 - b0, x1 - x)
            end = min(b0 + units, nb[n])
            if b0 == 0 or b0 < nb[n]:
                mine.append((n, h, b0, end - b0, end == nb[n]))
            x += units
        parts.append(mine)
        if x0 < x1 < B:
            n, = at(x1)
            h, e = divmod(x1 - starts[n], nb[n] + 1)
            if 0 < e < nb[n]:
                b0 = max(0, e - (x1 - x0))
                m = 0
                if b0 == 0:                          # the scan's walk from here
                    end, m = x1 - e + nb[n], 1
                    while j + m < J and start(j + m + 1) < end:
                        m += 1
                cuts.append((j, n, h, b0, e - b0, m))
    return nb, J, parts, cuts


def test_every_block_is_in_one_part_and_every_cut_is_scanned():
    rng = random.Random(3)
    for _ in range(300):
        C = rng.choice([16, 128])
        lens = [rng.choice([0, 1, C - 1, C, C + 1, rng.randrange(9 * C)]) for _ in range(rng.randrange(1, 9))]
        H, groups = rng.choice([1, 3, 8]), rng.choice([1, 5, 74, 148])
        nb, J, parts, cuts = _ranges(lens, H, C, groups)
        seen = [(n, h, b) for mine in parts for n, h, b0, k, _ in mine for b in range(b0, b0 + k)]
        assert seen == [(n, h, b) for n in range(len(lens)) for h in range(H) for b in range(nb[n])]
        # the state of every (sequence, head), empty ones too, is started once and ended once
        heads = [(n, h) for n in range(len(lens)) for h in range(H)]
        assert [(n, h) for mine in parts for n, h, b0, k, last in mine if b0 == 0] == heads
        assert [(n, h) for mine in parts for n, h, b0, k, last in mine if last] == heads
        # a part that does not start its (sequence, head) starts its group, and the group before has its summary
        entry = {j: (n, h, b0 + k) for j, n, h, b0, k, _ in cuts}
        for j, mine in enumerate(parts):
            for x, (n, h, b0, k, last) in enumerate(mine):
                if b0:
                    assert x == 0 and entry[j - 1] == (n, h, b0)
                if not last:
                    assert [(c[1], c[2], c[3], c[4]) for c in cuts if c[0] == j] == [(n, h, b0, k)] and k > 0
        assert sum(not p[4] for mine in parts for p in mine) == len(cuts)
        # each cut is walked by exactly one scan, from its (sequence, head)'s first group on
        walked = [j + u for j, *_, m in cuts for u in range(m)]
        assert sorted(walked) == sorted(c[0] for c in cuts)
        for j, n, h, b0, k, m in cuts:
            for u in range(m):
                assert entry[j + u][:2] == (n, h)


@pytest.mark.parametrize("kw", [
    dict(rms_w=(1 << 20) + 16, outgate=9 << 24), dict(cu_seqlens=(1 << 20) + 4), dict(slots=1 << 20), dict(seen=(1 << 20) + 2044),
    dict(workspace=(1 << 20) - 64, workspace_bytes=128),
])
def test_hla_output_over_what_steers_the_call_is_refused(lib, kw):
    # out: 4 tokens, 4 heads of 64, bf16 (2048 bytes)
    ptrs = {n: (i + 2) << 24 for i, n in enumerate(["q", "k", "v", "g"])}
    assert lib.gtr_hla_fwd(hla_args(**{**ptrs, "out": 1 << 20, **kw}), None) == -1


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "outgate", "rms_w", "slots", "seen", "cu_seqlens", "workspace"])
def test_hla_states_over_an_input_are_refused(lib, name):
    # state_out: one state of 65536 bytes
    ptrs = {n: (i + 2) << 24 for i, n in enumerate(["q", "k", "v", "g", "out"])}
    at = (1 << 20) + 65536 - 16
    more = {"rms_w": dict(outgate=9 << 24), "workspace": dict(workspace_bytes=64)}.get(name, {})
    assert lib.gtr_hla_fwd(hla_args(**{**ptrs, **more, "state_out": 1 << 20, "nslots": 1, name: at}), None) == -1
