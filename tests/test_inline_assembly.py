"""Inline assembly of several instructions: an output that is written before the last
input is read must not share a register with an input, so it is tied to one of its own
("+") or marked early-clobber ("=&")."""
import glob
import os
import re

import pytest

import attention_attn_varlen_gb300 as av

FILES = sorted(f for e in ("cu", "cuh") for f in glob.glob(os.path.join(os.path.dirname(av.__file__), "csrc", "*." + e)))


def statements(code):
    """The text between the parentheses of each asm(...)."""
    for m in re.finditer(r"\basm\s*(?:volatile\s*)?\(", code):
        depth, i, text = 1, m.end(), False
        while depth:
            c = code[i]
            if c == '"' and code[i - 1] != "\\":
                text = not text
            elif not text:
                depth += (c == "(") - (c == ")")
            i += 1
        yield code[m.end():i - 1]


def fields(body):
    """(template, outputs, inputs) of a statement: constraints in order."""
    parts, at, text, depth = [""], 0, False, 0
    while at < len(body):
        c = body[at]
        if c == '"' and body[at - 1] != "\\":
            text = not text
        if not text:
            depth += (c in "([") - (c in ")]")
        if c == ":" and not text and depth == 0:
            if body[at:at + 2] == "::":                      # no outputs, or a name's scope
                if re.match(r"::\s*\"", body[at:]) or re.match(r"::\s*$", body[at:]):
                    parts += ["", ""]
                    at += 2
                    continue
                parts[-1] += "::"
                at += 2
                continue
            parts.append("")
        else:
            parts[-1] += c
        at += 1
    template = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', parts[0])).replace("\\n", "\n").replace("\\t", "\t")
    constraints = [re.findall(r'"([^"]*)"\s*\(', p) for p in parts[1:3]] + [[], []]
    return template, constraints[0], constraints[1]


def at_risk(template, outputs, inputs):
    """Outputs that an instruction writes while a later one still reads an input."""
    lines = [x.strip() for x in re.split(r"[;\n]", template.replace("{", " ").replace("}", " }")) if x.strip()]
    n = len(outputs)
    writes, last_read = {}, -1
    for i, line in enumerate(lines):
        if line.startswith("."):
            continue
        operands = [int(x) for x in re.findall(r"%(\d+)", line)]
        # the first operand of an instruction (or of a vector of them) is its destination
        head = re.match(r"(?:@!?\w+\s+)?[\w.:]+\s+(%\d+)", line)
        for x in operands:
            if x < n and head and head.group(1) == f"%{x}":
                writes.setdefault(x, i)
            elif x >= n and x < n + len(inputs):
                last_read = max(last_read, i)
    return [x for x, i in writes.items() if i < last_read and outputs[x].startswith("=") and "&" not in outputs[x]]


def test_the_reader_sees_the_hazard():
    take = ('"{\\n\\t.reg .b16 l, u, m;\\n\\tmov.b32 {l, u}, %2;\\n\\tfma.rn.f32.bf16 %0, l, m, %3;\\n\\t'
            'fma.rn.f32.bf16 %1, u, m, %4;\\n\\t}" : "={}f"(r0), "={}f"(r1) : "r"(h), "f"(x0), "f"(x1)')
    assert at_risk(*fields(take.replace("{}", ""))) == [0]
    assert at_risk(*fields(take.replace("{}", "&"))) == []
    assert at_risk(*fields('"mov.u32 %0, %1;" : "=r"(a) : "r"(b)')) == []
    assert at_risk(*fields('"mov.u32 %0, %1;\\n\\tadd.u32 %0, %0, %1;" : "=r"(a) : "r"(b)')) == [0]


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_no_output_is_written_before_the_last_input_is_read(path):
    code = re.sub(r"//[^\n]*", "", open(path).read())
    found = 0
    for body in statements(code):
        found += 1
        assert not at_risk(*fields(body)), body
    assert found == len(re.findall(r"\basm\b", code))
