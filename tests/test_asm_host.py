"""Inline assembly names what it overwrites.  A register that a statement
writes by name is one that the compiler may hold a value in; without a word in
the list of clobbers it relies on nothing else using it."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_gemv_gemm_amd", "csrc")
WRITES = re.compile(r"\b[sv]_\w+\s+(m0|vcc|exec|[sv]\d+|[sv]\[\d+:\d+\])\s*,")


def unnamed(source):
    """(register, statement) of every one written and not in the clobbers."""
    found = []
    for m in re.finditer(r"\basm\s*(?:volatile\s*)?\(", source):
        depth, end = 1, m.end()
        while depth:  # (to the closing bracket; none of the strings holds one alone)
            depth += {"(": 1, ")": -1}.get(source[end], 0)
            end += 1
        body = source[m.end():end - 1]
        template = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', re.split(r'"\s*:', body)[0] + '"'))
        clobbers = body.rsplit(":", 1)[-1]
        found += [(r, body) for r in WRITES.findall(template.replace("\\n", "\n").replace("\\t", " ")) if f'"{r}"' not in clobbers]
    return found


def test_named_registers_are_clobbers():
    assert unnamed('asm volatile("s_mov_b32 m0, %0\\n\\ts_nop 0" ::"s"(to) : "memory");')
    assert not unnamed('asm volatile("s_mov_b32 m0, %0" ::"s"(to) : "memory", "m0");')
    sources = glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC, "*.h"))
    assert len(sources) > 10
    for path in sources:
        with open(path) as f:
            assert not unnamed(f.read()), path
