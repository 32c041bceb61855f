"""CPU test of the inline assembly in the kernels: what a statement writes, it
names, so that the compiler keeps nothing of its own there."""

import glob
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "tree_allreduce_algorithms_amd", "csrc")
FILES = sorted(f for e in ("hip", "hpp") for f in glob.glob(f"{CSRC}/**/*.{e}", recursive=True))


def statements(text):
    """(instructions, what follows them) of each asm statement."""
    for s in re.findall(r"\basm(?:\s+volatile)?\s*\((.*?)\)\s*;", text, re.S):
        template = re.match(r'\s*((?:"(?:[^"\\]|\\.)*"\s*)+)', s)
        code = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', template.group(1)))
        yield re.split(r"\\n(?:\\t)?", code), s[template.end():]


@pytest.mark.parametrize("path", FILES, ids=[os.path.relpath(f, CSRC) for f in FILES])
def test_written_scalar_registers_are_named(path):
    for code, rest in statements(open(path, encoding="utf-8").read()):
        for line in code:
            written = re.match(r"s_\w+\s+(m0|vcc\w*|exec\w*|s\d+|s\[\d+:\d+\])\s*,", line.strip())
            if written:
                assert f'"{written.group(1)}"' in rest.rsplit(":", 1)[-1], f"{line.strip()!r} in {path}"


def test_the_reader_finds_what_is_written():
    found = list(statements('asm volatile("s_mov_b32 m0, %0\\n\\ts_nop 0" ::"s"(f(x)) : "m0", "memory");'))
    assert found == [(["s_mov_b32 m0, %0", "s_nop 0"], '::"s"(f(x)) : "m0", "memory"')]
