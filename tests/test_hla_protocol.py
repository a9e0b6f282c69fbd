"""The order of the tensor-core prompt kernel's reads and writes (hla_tc.cuh), without a GPU.

Its roles share ring buffers, tensor memory and small per-block values, and
meet only at mbarriers.  The model below writes down each role's waits,
accesses and arrivals for a walk over several (sequence, head)s, builds the
order that the barriers enforce, and asks of every buffer that what is read
has been written, and that nothing is overwritten before its last reader is
done, whatever the roles' speeds.
"""
import os
import re

import pytest

from tests.hla_steady import STEADY, longest_walk, plan

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = open(os.path.join(ROOT, "linear_vision_backbone_b200", "csrc", "hla_tc.cuh")).read()


class Order:
    """Events of sequential agents, the edges that barriers add, and the accesses."""

    def __init__(self):
        self.before = []                      # direct predecessors of each event
        self.last = {}                        # the agent's latest event
        self.arrivals = {}                    # barrier -> agent -> its arrivals in order
        self.waits = []                       # (event, barrier, phase)
        self.writes, self.reads = {}, {}      # buffer -> version -> events

    def event(self, agent, *after):
        self.before.append([e for e in (self.last.get(agent), *after) if e is not None])
        self.last[agent] = len(self.before) - 1
        return self.last[agent]

    def arrive(self, agent, barrier, *after):
        e = self.event(agent, *after)
        self.arrivals.setdefault(barrier, {}).setdefault(agent, []).append(e)

    def wait(self, agent, barrier, phase):
        e = self.event(agent)
        if phase >= 0:                        # a fresh barrier passes its first wait
            self.waits.append((e, barrier, phase))

    def write(self, agent, buffer, version, *after):
        self.writes.setdefault(buffer, {}).setdefault(version, []).append(self.event(agent, *after))

    def read(self, agent, buffer, version, *after):
        self.reads.setdefault(buffer, {}).setdefault(version, []).append(self.event(agent, *after))

    def faults(self):
        for e, barrier, phase in self.waits:  # a phase ends with the arrival of each of its agents
            for mine in self.arrivals[barrier].values():
                self.before[e].append(mine[phase])
        done, state = [0] * len(self.before), [0] * len(self.before)
        for root in range(len(self.before)):
            stack = [root]
            while stack:
                e = stack[-1]
                if state[e] == 2:
                    stack.pop()
                    continue
                if state[e] == 0:
                    state[e] = 1
                    todo = [p for p in self.before[e] if state[p] != 2]
                    assert not any(state[p] == 1 for p in todo), "the roles wait for one another"
                    stack.extend(todo)
                if all(state[p] == 2 for p in self.before[e]):
                    for p in self.before[e]:
                        done[e] |= done[p] | 1 << p
                    state[e] = 2
                    stack.pop()
        early = []
        for buffer, versions in self.writes.items():
            names = sorted(versions)
            for x, v in enumerate(names):
                for r in self.reads.get(buffer, {}).get(v, []):
                    if not all(done[r] >> w & 1 for w in versions[v]):
                        early.append(f"{buffer}: version {v} is read before it is written")
                if x + 1 < len(names):
                    for w in versions[names[x + 1]]:
                        old = versions[v] + self.reads.get(buffer, {}).get(v, [])
                        if not all(done[w] >> o & 1 for o in old):
                            early.append(f"{buffer}: version {v} is overwritten while in use")
        for buffer, versions in self.reads.items():
            for v in versions:
                assert v in self.writes.get(buffer, {}), (buffer, v)
        return sorted(set(early))


def _exponent_behind_wait():
    """Whether the state warps store their exponent behind the wait for the terms' last reader."""
    put = SOURCE[SOURCE.index("auto put = [&]()"):SOURCE.index("warp_arrive(kSF);")]
    return put.index("es[is & 1] = ") > put.index("wait(kSE, (is & 1) ^ 1)")


def outputs_kernel(parts, NQ, NK, NV, NZ, gated, partial, exponent_behind_wait):
    """parts: (blocks, starts from a state, its last state is wanted)."""
    o = Order()
    blocks = []                               # (index, part's first, part's last, state before it, state behind it)
    for nb, start, end in parts:
        for c in range(nb):
            blocks.append((len(blocks), c == 0, c + 1 == nb, c > 0 or start, c + 1 < nb or end))
    # what the tensor cores do runs in the order of its issue; a commit arrives behind all of it
    tc, mma = "tc", "mma"

    def commit(barrier):
        o.arrive(tc, barrier, o.last[mma])

    for i, *_ in blocks:
        o.wait("load", ("KE", i % NK), i // NK - 1)
        o.write("load", ("K", i % NK), (i, 0))
        o.arrive("load", ("KF", i % NK))
        o.wait("load", ("VE", i % NV), i // NV - 1)
        o.write("load", ("V", i % NV), (i, 0))
        o.arrive("load", ("VF", i % NV))
        o.wait("loadq", ("QE", i % NQ), i // NQ - 1)
        o.write("loadq", ("Q", i % NQ), i)
        o.arrive("loadq", ("QF", i % NQ))

    def finish(i):
        o.wait("loadz", ("OS", i % NZ), i // NZ)
        o.read("loadz", ("Z", i % NZ), (i, 1))
    for i, *_ in blocks:
        if i >= NZ:
            finish(i - NZ)
        if gated:
            o.write("loadz", ("Z", i % NZ), (i, 0))
        o.arrive("loadz", ("ZF", i % NZ))
    for i in range(max(0, len(blocks) - NZ), len(blocks)):
        finish(i)

    m = 0                                     # states used so far
    for i, _, _, state, behind in blocks:
        tail = partial and not behind
        o.wait(mma, ("KF", i % NK), i // NK)
        o.wait(mma, ("QF", i % NQ), i // NQ)
        issue = o.event(mma)
        o.read(tc, ("Q", i % NQ), i, issue)
        if not tail:                          # (the columns behind the last token are zeroed meanwhile, and masked)
            o.read(tc, ("K", i % NK), (i, 0), issue)
        o.write(tc, "scores", (i, 0), issue)
        commit("ScF")
        o.wait(mma, "WF", i)
        o.wait(mma, "KvE", i - 1)
        if behind:
            issue = o.event(mma)
            o.read(tc, ("K", i % NK), (i, int(tail)), issue)
            o.read(tc, "W", i, issue)
            o.write(tc, "KV", i, issue)
        for b in ("KvF", "WE", ("KE", i % NK)):
            commit(b)
        if state:
            o.wait(mma, "SF", m)
        o.wait(mma, "OE", i - 1)
        if state:
            issue = o.event(mma)
            o.read(tc, ("Q", i % NQ), i, issue)
            o.read(tc, "S", m, issue)
            o.write(tc, "QS", m, issue)
            commit("SE")
            m += 1
        commit(("QE", i % NQ))
        o.wait(mma, "PF", i)
        issue = o.event(mma)
        o.read(tc, "scores", (i, 1), issue)
        o.read(tc, ("V", i % NV), (i, int(tail)), issue)
        o.write(tc, "PV", i, issue)
        commit("PvF")
        commit(("VE", i % NV))

    for i, _, _, state, behind in blocks:
        tail = partial and not behind
        o.wait("build", ("GE", i & 1), (i >> 1) - 1)
        o.write("build", ("L", i & 1), (i, 0))
        o.write("build", ("U", i & 1), (i, 0))
        o.write("build", ("wsum", i & 1), i)
        o.read("build", ("wsum", i & 1), i)
        o.arrive("build", ("GF", i & 1))
        o.wait("build", ("VF", i % NV), i // NV)
        o.read("build", ("V", i % NV), (i, 0))
        o.wait("build", "WE", i - 1)
        if behind:
            o.write("build", ("ew", i & 3), i)
            o.write("build", "W", i)
        if tail:
            o.wait("build", ("KF", i % NK), i // NK)
            o.write("build", ("K", i % NK), (i, 1))
            o.write("build", ("V", i % NV), (i, 1))
        o.arrive("build", "WF")

    m = 0

    def put():
        nonlocal m
        if not exponent_behind_wait:
            o.write("state", ("es", m & 1), m)
        o.wait("state", "SE", m - 1)
        if exponent_behind_wait:
            o.write("state", ("es", m & 1), m)
        o.write("state", "S", m)
        o.arrive("state", "SF")
        m += 1
    for i, first, last, state, behind in blocks:
        if first and state:
            put()
        o.wait("state", ("GF", i & 1), i >> 1)
        o.wait("state", "KvF", i)
        o.read("state", ("wsum", i & 1), i)
        o.arrive("state", ("GE", i & 1))
        if behind:
            o.read("state", ("ew", i & 3), i)
            o.read("state", "KV", i)
        o.arrive("state", "KvE")
        if not last:
            put()

    for i, *_ in blocks:
        o.wait("p", ("GF", i & 1), i >> 1)
        o.read("p", ("L", i & 1), (i, 0))
        o.write("p", ("L", i & 1), (i, 1))
        o.read("p", ("wsum", i & 1), i)
        o.read("p", ("U", i & 1), (i, 0))
        o.wait("p", "ScF", i)
        o.write("p", ("pexp", i & 1), i)
        o.read("p", "scores", (i, 0))
        o.write("p", "scores", (i, 1))
        o.arrive("p", "PF")
        o.arrive("p", ("GE", i & 1))

    m = 0
    for i, _, _, state, _ in blocks:
        o.wait("out", ("ZF", i % NZ), i // NZ)
        o.wait("out", "PvF", i)
        o.read("out", ("L", i & 1), (i, 1))
        o.read("out", ("pexp", i & 1), i)
        if state:
            o.read("out", ("es", m & 1), m)
            o.read("out", "QS", m)
            m += 1
        o.read("out", "PV", i)
        o.arrive("out", "OE")
        if gated:
            o.write("out", ("U", i & 1), (i, 1))          # the row's sum of squares
            o.read("out", ("U", i & 1), (i, 1))
            o.read("out", ("Z", i % NZ), (i, 0))
        o.arrive("out", ("GE", i & 1))
        o.write("out", ("Z", i % NZ), (i, 1))
        o.arrive("out", ("OS", i % NZ))
    return o


def summary_kernel(nb, NK, NV, NW):
    """The summaries: one part, wv tiles and kv accumulators in turn."""
    o = Order()
    for i in range(nb):
        o.wait("load", ("KE", i % NK), i // NK - 1)
        o.write("load", ("K", i % NK), i)
        o.arrive("load", ("KF", i % NK))
        o.wait("load", ("VE", i % NV), i // NV - 1)
        o.write("load", ("V", i % NV), i)
        o.arrive("load", ("VF", i % NV))
        o.wait("mma", ("KF", i % NK), i // NK)
        o.wait("mma", ("WF", i % NW), i // NW)
        o.wait("mma", ("KvE", i % NW), i // NW - 1)
        issue = o.event("mma")
        o.read("tc", ("K", i % NK), i, issue)
        o.read("tc", ("W", i % NW), i, issue)
        o.write("tc", ("KV", i % NW), i, issue)
        for b in (("KvF", i % NW), ("WE", i % NW), ("KE", i % NK), ("VE", i % NV)):
            o.arrive("tc", b, o.last["mma"])
        o.wait("build", ("GE", i & 1), (i >> 1) - 1)
        o.write("build", ("wsum", i & 1), i)
        o.arrive("build", ("GF", i & 1))
        o.wait("build", ("VF", i % NV), i // NV)
        o.read("build", ("V", i % NV), i)
        o.wait("build", ("WE", i % NW), i // NW - 1)
        o.write("build", ("ew", i & 3), i)
        o.write("build", ("W", i % NW), i)
        o.arrive("build", ("WF", i % NW))
        o.wait("state", ("GF", i & 1), i >> 1)
        o.wait("state", ("KvF", i % NW), i // NW)
        o.read("state", ("wsum", i & 1), i)
        o.arrive("state", ("GE", i & 1))
        o.read("state", ("ew", i & 3), i)
        o.read("state", ("KV", i % NW), i)
        o.arrive("state", ("KvE", i % NW))
    return o


PARTS = [[(9, True, True)], [(1, True, True), (1, False, True), (6, True, False), (1, False, False), (5, False, True)],
         [(2, False, False)] * 4]
RINGS = {64: dict(NQ=2, NK=2, NV=2, NZ=2), 128: dict(NQ=1, NK=2, NV=2, NZ=1)}


@pytest.mark.parametrize("parts", PARTS, ids=["one", "mixed", "short"])
@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("partial", [True, False])
def test_no_buffer_of_the_outputs_kernel_is_reused_early(parts, dk, gated, partial):
    o = outputs_kernel(parts, **RINGS[dk], gated=gated, partial=partial,
                       exponent_behind_wait=_exponent_behind_wait())
    assert o.faults() == []


def test_an_exponent_stored_before_the_wait_would_be_early():
    o = outputs_kernel([(9, True, True)], **RINGS[128], gated=True, partial=False, exponent_behind_wait=False)
    assert any("es" in f for f in o.faults())


@pytest.mark.parametrize("nk", [2, 3])
def test_no_buffer_of_the_summary_kernel_is_reused_early(nk):
    assert summary_kernel(12, nk, nk, 2).faults() == []


def test_the_models_rings_are_the_kernels():
    for name, text in (("kNQ", "kSum ? 0 : DK == 64 ? 2 : 1"), ("kNK", "kSum && DK == 64 ? 3 : 2"), ("kNV", "kNK"),
                       ("kNW", "kSum ? 2 : 1"), ("kNZ", "DK == 64 ? 2 : 1")):
        got = re.search(rf"static constexpr int {name} = ([^;]*);", SOURCE).group(1)
        assert got == text, name


# ------------------------------------------------ the GPU tests' long walks
@pytest.mark.parametrize("name", STEADY)
def test_steady_cases_walk_many_blocks(name):
    lens, H, Hk, dk, dv, dtype, gated, equal = STEADY[name]
    J, cut, _ = plan(len(lens), sum(lens), H, dk, dv, dtype, equal)
    tc = dtype != "f32"
    walk, part = longest_walk(lens, H, J, cut, 128 if tc else 16)
    # every ring of the kernel wraps and every barrier takes both parities, more than once
    assert walk >= 8
    if len(lens) < 32:
        assert part >= 8                      # and with one state behind another in a single part
    assert cut != equal


# ------------------------------------------------------ waits that run out
def _role(name, following):
    a = SOURCE.index(f"role == {name}) {{", SOURCE.index("if (role == kLoad) {"))
    return SOURCE[a:SOURCE.index(following, a)]


@pytest.mark.parametrize("name,following", [("kMma", "role == kBuild"), ("kBuild", "role == kState"),
                                            ("kState", "} else if constexpr (!kSum)"), ("kP", "role == kOut"),
                                            ("kOut", "role == kLoadQ")])
def test_a_wait_that_ran_out_skips_no_barrier_of_its_group(name, following):
    """bar.sync and the warp-wide instructions have no limit, so no thread of these groups may leave its walk, or take
    another way through it, because a bounded wait of its own ran out: it may only leave out arrivals and issues."""
    body = re.sub(r"//[^\n]*", "", _role(name, following))
    body = body.replace("if (!more) break;", "")       # the end of the walk, the same for the whole group
    assert "break" not in body and "return false" not in body and "continue" not in body
    for line in body.splitlines():
        if re.search(r"\bok\b", line):
            assert re.search(r"if \((lead|row == 0|\(c \+ 1 < nb \|\| want_end\) && lead) && ok\)|if \(ok\) peer_|cluster_wait\(",
                             line), line
    for _, guarded in re.findall(r"^( *)if \([^\n]*\bok\b[^\n]*\) \{\n(.*?)^\1\}", body, re.S | re.M):
        assert "named_barrier" not in guarded and "_arrive(" not in guarded and "sync" not in guarded
    # the waits give nothing back that a caller could branch on
    assert not re.search(r"=\s*wait2?\(", body) and not re.search(r"(if|while) \(!?wait2?\(", body)


def test_every_wait_has_a_limit_and_the_walk_does_not_depend_on_it():
    text = re.sub(r"//[^\n]*", "", SOURCE)
    assert len(re.findall(r"mbarrier\.try_wait", text)) == 1 and "mbar_wait(" not in text
    # both loops that probe, and end for a thread that gave up before
    assert len(re.findall(r"uint32_t n = ok \? kProbes : 0;", text)) == 2
    assert len(re.findall(r"if \(n == 0\) \{\s*ok = false;\s*return;\s*\}\s*--n;", text)) == 2
    assert "while (next_part<kC" in text and "ok && next_part" not in text
