"""Registers that the kernels' inline assembly writes by name are in its list
of clobbered ones: the compiler keeps values in them otherwise."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "lossless_bf16_tensor_exp_amd", "csrc")


def statements(text):
    """Every asm statement, up to the semicolon behind its closing parenthesis."""
    for m in re.finditer(r"\basm\s+(?:volatile\s*)?\(", text):
        depth, at, quoted = 1, m.end(), False
        while depth:
            c = text[at]
            if c == '"' and text[at - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            at += 1
        yield text[m.end():at - 1]


def written(body):
    """The named registers that the instructions of an asm statement write."""
    code = "\n".join(re.findall(r'"((?:[^"\\]|\\.)*)"', body.split(":")[0])).replace("\\n", "\n").replace("\\t", " ")
    names = set()
    for line in code.split("\n"):
        m = re.match(r"\s*(?:s|v)_\w+\s+(m0|vcc|exec|scc|[sv]\d+|[sv]\[\d+:\d+\])\b", line)
        if m:
            names.add(m.group(1))
    return names


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.hip"))), ids=os.path.basename)
def test_named_registers_are_declared(path):
    for body in statements(open(path).read()):
        clobbers = body.rsplit(":", 1)[-1]
        for name in written(body):
            assert f'"{name}"' in clobbers, body


def test_the_check_finds_one():
    body, = statements('asm volatile("s_mov_b32 m0, %0\\n\\ts_nop 0" :: "s"(a) : "memory");')
    assert written(body) == {"m0"} and '"m0"' not in body.rsplit(":", 1)[-1]
