"""Inline assembly in the HIP sources: a register that an instruction names in
the text is the compiler's to use unless the statement declares it as clobbered."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "decode_moe_mul_amd", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.h*")))
NAMED = re.compile(r"\b(m0|vcc|exec|scc|[vsa]\d+|[vsa]\[\d+:\d+\])\b")


def _statements(text):
    """(template, everything after it) of each asm statement of a source."""
    text = re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)
    for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\(((?:\s*\"(?:[^\"\\]|\\.)*\")+)([^;]*)\);", text):
        yield "".join(re.findall(r"\"((?:[^\"\\]|\\.)*)\"", m.group(1))), m.group(2)


def _undeclared(text):
    bad = []
    for template, rest in _statements(text):
        clobbers = rest.split(":")[3] if rest.count(":") >= 3 else ""
        for line in re.split(r"\\n|;", template):
            named = set(NAMED.findall(re.sub(r"\\t", " ", line)))
            bad += [(line, r) for r in named if f'"{r}"' not in clobbers]
    return bad


def test_the_search_finds_an_undeclared_register():
    text = 'asm volatile("s_mov_b32 m0, %0\\n\\ts_nop 0" : : "s"(x) : "memory");'
    assert [r for _, r in _undeclared(text)] == ["m0"]
    assert not _undeclared(text.replace('"memory"', '"m0", "memory"'))
    assert not _undeclared('asm("v_and_or_b32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "s"(b), "v"(c));')


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_registers_named_in_inline_assembly_are_declared(path):
    text = open(path).read()
    assert len(list(_statements(text))) == len(re.findall(r"\basm\b(?:\s+volatile)?\s*\(", text))
    assert not _undeclared(text)
