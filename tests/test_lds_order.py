"""LDS ordering of the attention kernels, read from the gfx950 assembly that the compiler makes of the sources here (CPU).

A copy from global memory into LDS is not ordered behind a wave's earlier LDS reads: an instruction has to wait for them
(lgkmcnt).  The check follows every path of a kernel and carries how many LDS operations came after the newest read of a
staged tile, until a wait covers that read.  The other way round, a wave waits for a staged tile by the number of vector
memory operations that may still be in flight (vmcnt): those have to be copies, whose number the source fixes, and no
loads, whose number the compiler chooses.
"""
import os
import re
import subprocess

import pytest

from gated_short_causal_amd import build

CSRC = build.CSRC
READ = re.compile(r"ds_read_(b128|b64)")                   # tiles are read 16 bytes at a time, or transposed 8
QUEUED = re.compile(r"ds_|s_load|s_buffer_load")           # what lgkmcnt counts
COPY = re.compile(r"global_load_lds|buffer_load\S*\s.*\blds\b")
BARRIER = re.compile(r"s_barrier")
VMEM = re.compile(r"global_(load|store)|buffer_(load|store)|flat_")
VMWAIT = re.compile(r"s_waitcnt\b.*vmcnt\((\d+)\)")
WAIT = re.compile(r"s_waitcnt\b.*lgkmcnt\((\d+)\)")


def _kernels(asm):
    """{mangled name: {label: (instructions, successors)}} of every function."""
    out = {}
    for name, body in re.findall(r"^(_Z\w+):(.*?)^\.Lfunc_end", asm, re.M | re.S):
        blocks, label = {"entry": []}, "entry"
        for line in body.splitlines():
            line = line.split(";")[0].strip()
            mark = re.match(r"(\.LBB\w+):", line)
            if mark or re.match(r"s_c?branch", blocks[label][-1] if blocks[label] else ""):
                new = mark.group(1) if mark else f"{label}+"
                blocks[new], label = [], new
            if line and not mark and not line.startswith("."):
                blocks[label].append(line)
        names, graph = list(blocks), {}
        for here, after in zip(names, names[1:] + [None]):
            last = blocks[here][-1] if blocks[here] else ""
            jump = re.match(r"s_(c?)branch\S*\s+(\S+)", last)
            if jump:
                to = [jump.group(2)] + ([after] if jump.group(1) else [])
            else:
                to = [] if last.startswith("s_endpgm") else [after]
            graph[here] = (blocks[here], [t for t in to if t is not None])
        out[name] = graph
    return out


def _step(newer, instruction):
    """newer: LDS operations since the newest tile read that nothing waited for; None: none such."""
    if READ.match(instruction):
        return 0
    if newer is None:
        return None
    if QUEUED.match(instruction):
        return newer + 1
    wait = WAIT.match(instruction)
    return None if wait and int(wait.group(1)) <= newer else newer


def _flow(graph, start, step):
    """The least state (None: above all) in which some path reaches each instruction: (label, instruction, state)."""
    state, work = {"entry": start}, ["entry"]
    while work:
        here = work.pop()
        now = state[here]
        for i in graph[here][0]:
            now = step(now, i)
        for to in graph[here][1]:
            old = state.get(to, "new")
            joined = now if old == "new" else min((x for x in (old, now) if x is not None), default=None)
            if joined != old:
                state[to] = joined
                work.append(to)
    out = []
    for here, now in state.items():
        for i in graph[here][0]:
            out.append((here, i, now))
            now = step(now, i)
    return out


def _unwaited(graph, what):
    """The instructions matching `what` that some path reaches with a tile read in flight."""
    return [(here, i) for here, i, newer in _flow(graph, None, _step) if newer is not None and what.match(i)]


def _counts_a_load(graph, least):
    """The waits that leave `least` or more operations in flight which on some path are not all copies."""
    def step(run, i):                                # copies since the last other vector memory operation, at most 64
        return min(run + 1, 64) if COPY.match(i) else 0 if VMEM.match(i) else run
    return [(here, i) for here, i, run in _flow(graph, 0, step)
            for n in VMWAIT.findall(i) if int(n) >= least and int(n) > run]


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    try:
        hipcc = build.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not found")
    out, runs = {}, []
    for src in ("attn_fwd", "attn_bwd", "attn_cached"):
        asm = str(tmp_path_factory.mktemp("asm") / (src + ".s"))
        cmd = [hipcc, *build.compile_flags(), "--cuda-device-only", "-S", "-x", "hip", os.path.join(CSRC, src + ".hip"), "-o", asm]
        runs.append((asm, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)))
    for asm, p in runs:
        _, err = p.communicate(timeout=600)
        assert p.returncode == 0, err[-3000:]
        with open(asm) as f:
            out.update(_kernels(f.read()))
    # kernels that stage tiles in LDS
    return {n: g for n, g in out.items() if any(COPY.match(i) for b, _ in g.values() for i in b)}


def test_the_check_sees_a_read_in_flight():
    """The check itself: one read under a copy, one that a count of 1 covers, one that only a branch leaves open."""
    asm = """_Zone:
 ds_read_b128 v[0:3], v9
 ds_bpermute_b32 v4, v5, v6
 global_load_lds_dwordx4 v[7:8], off
 s_endpgm
.Lfunc_end0:
_Ztwo:
 ds_read_b64_tr_b16 v[0:1], v9
 ds_bpermute_b32 v4, v5, v6
 s_waitcnt lgkmcnt(1)
 buffer_load_dwordx4 v9, s[0:3], 0 offen lds
 s_endpgm
.Lfunc_end1:
_Zthree:
 s_waitcnt lgkmcnt(0)
.LBB2_1:
 global_load_lds_dwordx4 v[7:8], off
 s_cbranch_scc1 .LBB2_3
 ds_read_b128 v[0:3], v9
 s_branch .LBB2_1
.LBB2_3:
 s_endpgm
.Lfunc_end2:
"""
    k = _kernels(asm)
    assert [len(_unwaited(k[n], COPY)) for n in ("_Zone", "_Ztwo", "_Zthree")] == [1, 0, 1]


def test_the_check_sees_a_counted_load():
    asm = """_Zone:
 global_load_dword v0, v[1:2], off
 global_load_lds_dwordx4 v[7:8], off
 global_load_lds_dwordx4 v[7:8], off
 s_waitcnt vmcnt(2)
 s_waitcnt vmcnt(3) lgkmcnt(0)
 s_endpgm
.Lfunc_end0:
"""
    assert _counts_a_load(_kernels(asm)["_Zone"], 2) == [("entry", "s_waitcnt vmcnt(3) lgkmcnt(0)")]


def _named(kernels, part):
    hits = {n: g for n, g in kernels.items() if part in n}
    assert hits, part
    return hits


@pytest.mark.parametrize("part", ["attn_cached_direct_kernel", "attn_cached_kernel"])
def test_refills_wait_for_the_reads_of_the_tile(kernels, part):
    """A wave refills its own staging buffer: no copy may start while one of its tile reads is in flight."""
    for name, graph in _named(kernels, part).items():
        assert not _unwaited(graph, COPY), name


def test_barriers_wait_for_the_reads_of_the_tile(kernels):
    """Behind a barrier any wave of the workgroup refills the shared slot: every wave's reads have to be back."""
    assert {p for p in ("attn_fwd", "attn_grad", "attn_cached") for n in kernels if p in n} == {"attn_fwd", "attn_grad", "attn_cached"}
    for name, graph in kernels.items():
        assert not _unwaited(graph, BARRIER), name


@pytest.mark.parametrize("part", ["attn_cached_direct_kernel", "attn_cached_kernel"])
def test_waits_for_a_tile_count_copies_only(kernels, part):
    """The smallest tile is 4 copies: waits that leave 4 or more operations in flight are the kernels' own."""
    for name, graph in _named(kernels, part).items():
        assert not _counts_a_load(graph, 4), name
