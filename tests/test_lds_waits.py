"""CPU check of the attention kernels' waits, as compiled for gfx950.  Their tiles are moved by
buffer -> LDS loads that run ahead, so what keeps a read from a tile that is not there yet, and a
load from a tile that is still read, are waits alone:
  - in the optimised LLVM code no hand-written wait may be marked as not concerning memory that
    the function around it takes by restrict pointers: accesses could then move across it;
  - in the compiled code every LDS read is waited for before a later LDS-bound load is issued;
  - in the kernels whose waves wait for their own loads only (few rows) a tile is read only after a
    wait that leaves no more than the next block's loads under way."""

import os
import re
import subprocess

import pytest

from deformable_convolution_vision_amd import build as libbuild

SOURCES = ("dcn_attention.hip", "dcn_attention_grad.hip")
NOTHING = 1 << 10   # loads under way when none has been waited for


@pytest.fixture(scope="module")
def compiled(tmp_path_factory):
    if not os.path.exists(libbuild.hipcc()):
        pytest.skip("hipcc not found")
    at, jobs, texts = tmp_path_factory.mktemp("waits"), [], {}
    for src in SOURCES:
        for kind, flags in (("s", ("-S",)), ("ll", ("-S", "-emit-llvm"))):
            out = str(at / f"{src}.{kind}")
            cmd = [libbuild.hipcc(), *libbuild.HIPCC_FLAGS, "--cuda-device-only", *flags,
                   os.path.join(libbuild.CSRC, src), "-o", out]
            jobs.append((src, kind, out, subprocess.Popen(cmd, stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)))
    for src, kind, out, job in jobs:
        assert job.wait() == 0, f"hipcc failed on {src}"
        texts[src, kind] = open(out).read()
    return texts


def kernels(text):
    """(name, instructions and labels) of each kernel of an assembly file."""
    for m in re.finditer(r"^(_Z\S+):.*\n((?:.*\n)*?)\s*\.section", text, re.M):
        yield m.group(1), [s for s in (line.split(";")[0].strip() for line in m.group(2).splitlines()) if s]


def blocks(body):
    """Basic blocks: name -> (instructions, names of the blocks that may follow)."""
    out, name = {"entry": ([], [])}, "entry"
    for s in body:
        code, then = out[name]
        label = re.match(r"(\.LBB\w+):", s)
        if label:
            if not (code and re.match(r"s_branch|s_endpgm", code[-1])):
                then.append(label.group(1))
            name = label.group(1)
            out[name] = ([], [])
        elif not s.startswith("."):
            code.append(s)
            if re.match(r"s_c?branch", s):
                then.append(s.split()[-1])
                name = f"after {len(out)}"
                if s.startswith("s_cbranch"):
                    then.append(name)
                out[name] = ([], [])
    return out


def faults(body, most):
    """Walks every path: whether an LDS read may be under way, and how many loads the waits since the
    last LDS-bound load allow.  most: what a read of a tile may find (None: not checked)."""
    bs, known, todo, bad = blocks(body), {"entry": (False, 0)}, ["entry"], set()
    while todo:
        name = todo.pop()
        reading, under_way = known[name]
        for s in bs[name][0]:
            op = s.split()[0]
            if op.startswith("buffer_load") and s.endswith(" lds"):
                if reading:
                    bad.add(f"{name}: {s} while an LDS read is under way")
                under_way = NOTHING
            elif op.startswith("ds_read"):
                reading = True
                if most is not None and under_way > most:
                    bad.add(f"{name}: {s} with {under_way} loads under way")
            elif op == "s_waitcnt":
                reading = reading and "lgkmcnt(0)" not in s
                n = re.search(r"vmcnt\((\d+)\)", s)
                under_way = min(under_way, int(n.group(1))) if n else under_way
        for n in bs[name][1]:
            if n not in bs:
                continue
            old = known.get(n)
            new = (reading, under_way) if old is None else (old[0] or reading, max(old[1], under_way))
            if new != old:
                known[n] = new
                todo.append(n)
    return bad


def test_no_wait_is_marked_as_concerning_other_memory(compiled):
    n = 0
    for src in SOURCES:
        for line in compiled[src, "ll"].splitlines():
            if re.search(r'asm sideeffect "s_(waitcnt|barrier)', line):
                n += 1
                assert "!noalias" not in line, f"{src}: {line.strip()}"
    assert n > 0


def test_lds_reads_and_lds_bound_loads_wait_for_each_other(compiled):
    loads = few = 0
    for src in SOURCES:
        for name, body in kernels(compiled[src, "s"]):
            loads += sum(s.endswith(" lds") for s in body)
            # (element by element: rows come through registers)
            m = re.search(r"attn_few_rows_kernelI(t|f)Li(\d+)ELi\d+ELb1", name)
            row = int(m.group(2)) * (2 if m.group(1) == "t" else 4) if m else 0   # bytes
            few += m is not None
            # a block of 32 keys: 16 bytes a load of each lane for the keys, and as many values
            bad = faults(body, 2 * 32 * row // 16 // 64 if m else None)
            assert not bad, name + "\n" + "\n".join(sorted(bad)[:10])
    assert loads > 100 and few == 6


def test_the_walk_finds_what_it_looks_for():
    lds = "buffer_load_dwordx4 v1, s[0:3], 0 offen lds"
    ok = [lds, ".LBB0_1:", lds, "s_waitcnt vmcnt(1)", "ds_read_b128 v[0:3], v4", "s_waitcnt lgkmcnt(0)",
          "s_cbranch_scc1 .LBB0_1", "s_endpgm"]
    assert not faults(ok, 1)
    assert faults([s for s in ok if "lgkmcnt" not in s], 1)           # the loop's load may find the read under way
    assert faults([s for s in ok if "vmcnt" not in s], 1)             # the read finds loads that were not waited for
    assert faults([s.replace("vmcnt(1)", "vmcnt(2)") for s in ok], 1)
