"""The kernels' inline assembly (no GPU: the sources are read): what a block
writes beside its outputs is among its clobbers, so that the compiler keeps
nothing there across it."""
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "combine_router_topk_amd", "csrc")
SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith((".hip", ".hpp")))


def blocks(text):
    """(instructions, clobbers) of every asm statement."""
    for m in re.finditer(r"\b(?:__asm__|asm)\s*(?:volatile)?\s*\(", text):
        depth, i = 1, m.end()
        while depth:
            quoted = re.match(r'"(?:[^"\\]|\\.)*"', text[i:])
            if quoted:
                i += quoted.end()
                continue
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        body = text[m.end():i - 1]
        parts, depth, last = [], 0, 0  # at colons outside of quotes and parentheses
        for q in re.finditer(r'"(?:[^"\\]|\\.)*"|[():]', body):
            t = q.group()
            depth += {"(": 1, ")": -1}.get(t, 0)
            if depth == 0 and t == ":":
                parts.append(body[last:q.start()])
                last = q.end()
        parts.append(body[last:])
        strings = lambda s: "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', s))  # noqa: E731
        yield strings(parts[0]).replace("\\n", "\n").replace("\\t", "\t"), \
            re.findall(r'"([^"]*)"', parts[3]) if len(parts) > 3 else []


def test_the_blocks_are_found():
    found = {f: list(blocks(open(os.path.join(CSRC, f)).read())) for f in SOURCES}
    loads = [b for b in found["expert_gemm.hip"] if "global_load_lds" in b[0]]
    assert len(loads) == 2 and all("memory" in c for _, c in loads), loads
    assert any("s_barrier" in b for b, _ in found["expert_gemm.hip"])
    assert list(blocks('asm volatile("s_mov_b32 m0, %0" ::"s"(f(a, b ? 1 : 2)), "n"(P) : "memory", "m0");')) \
        == [("s_mov_b32 m0, %0", ["memory", "m0"])]
    assert list(blocks('asm("s_barrier" ::: "memory"); asm volatile("" : "+v"(a[b::c]));')) \
        == [("s_barrier", ["memory"]), ("", [])]


@pytest.mark.parametrize("name", SOURCES)
def test_written_registers_are_clobbers(name):
    text = open(os.path.join(CSRC, name)).read()
    for body, clobbers in blocks(text):
        for line in filter(None, (l.strip() for l in body.split("\n"))):
            op, _, args = line.partition(" ")
            first = args.split(",")[0].strip()
            if first in ("m0", "exec", "vcc", "scc"):
                assert first in clobbers, (name, line, clobbers)
            if re.match(r"s_(add|sub|and|or|xor|lsh|ash|cmp)", op):
                assert "scc" in clobbers, (name, line, clobbers)
            if re.match(r"(global|buffer|flat|ds|s)_(load|store|read|write|atomic|barrier|waitcnt)", op):
                assert "memory" in clobbers, (name, line, clobbers)
