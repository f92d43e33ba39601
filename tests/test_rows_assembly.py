"""What the attention kernels' inline assembly owes the processor, from the listings that the compiler makes of them here:
host only."""

import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from layout_permuting_copy_amd import build as B

SOURCES = [s for s in B.SOURCES if s.startswith("prompt_attention") or s.startswith("tree_attention_")]


@pytest.fixture(scope="module")
def listings(tmp_path_factory):
    if not os.path.exists(B.HIPCC):
        pytest.skip("no compiler")
    folder = tmp_path_factory.mktemp("listings")

    def lines(source):
        out = str(folder / (source + ".s"))
        B._run([B.HIPCC, B.ARCH, *B.NO_PK, *B.COMMON, "--cuda-device-only", "-S", os.path.join(B.CSRC, source), "-o", out])
        with open(out) as f:
            return [x for x in (line.split(";")[0].strip() for line in f) if x and not x.startswith(".") and not x.endswith(":")]

    with ThreadPoolExecutor(len(SOURCES)) as pool:
        return dict(zip(SOURCES, pool.map(lines, SOURCES)))


def _operands(line):
    return re.split(r"[ ,]+", line)[1:]


def _scalars(operand):
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m[1]), int(m[2]) + 1))
    m = re.fullmatch(r"s(\d+)", operand)
    return {int(m[1])} if m else set()


def _written(line):
    """Scalar registers that a vector instruction writes: its first operand, and the carry of those that have one."""
    o = _operands(line)
    return set().union(*(_scalars(x) for x in o[:2 if "_co_" in line or "div_scale" in line else 1]))


def test_loads_wait_for_scalars_from_vector_instructions(listings):
    """A memory instruction reads a scalar register that a vector instruction wrote five wait states later at least."""
    loads, early = 0, []
    for source, lines in listings.items():
        for i, line in enumerate(lines):
            if not re.match(r"(buffer|global|flat|scratch)_", line):
                continue
            read = set().union(*map(_scalars, _operands(line)))
            if not read:
                continue
            loads += 1
            states, j = 0, i - 1
            while j >= 0 and states < 5:
                if lines[j].startswith("v_") and _written(lines[j]) & read:
                    early.append((source, lines[j], line, states))
                    break
                states += int(_operands(lines[j])[0], 0) + 1 if lines[j].startswith("s_nop") else 1
                j -= 1
    assert loads > 500
    assert not early, (len(early), early[:3])


def test_assembly_names_the_registers_that_it_writes():
    """Scalar registers that a statement's instructions write by name are among its clobbers, m0 and the condition code too."""
    with open(os.path.join(B.CSRC, "rows_attention.hpp")) as f:
        text = f.read()
    written = 0
    for statement in re.findall(r"\basm(?: volatile)?\s*\(.*?\)\s*;", text, re.S):
        clobbers = statement.rsplit(":", 1)[1]
        for pattern, name in ((r"s_mov_b32 m0", "m0"), (r"s_cmp_", "scc")):
            if re.search(pattern, statement):
                written += 1
                assert f'"{name}"' in clobbers, statement[:120]
    assert written >= 4
