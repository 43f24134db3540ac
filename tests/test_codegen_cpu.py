"""Code generation of the HIP kernels for gfx950 (no GPU: hipcc emits device
assembly here). Two properties that the kernels' speed depends on and that a
small source change can silently break:

- no out-of-line device calls: a shared device function the compiler stops
  inlining is compiled with generic pointers, so its global and LDS accesses
  become flat instructions (one such call slowed the layout plan kernel by
  6 us);
- no flat memory instructions and no register spills to scratch memory.
"""
import os
import re
import shutil
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "combine_router_topk_amd", "csrc")
HIPCC = "/opt/rocm/bin/hipcc"
# kernel -> allowed private segment bytes (none at present)
SCRATCH_ALLOWED: dict[str, int] = {}


def compile_asm(src: str, out_dir: str) -> str:
    out = os.path.join(out_dir, os.path.basename(src)[:-4] + ".s")
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang",
                    "-target-feature", "-Xclang", "-packed-fp32-ops",
                    f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", "--cuda-device-only", "-S",
                    src, "-o", out], check=True, capture_output=True, timeout=300)
    return out


@pytest.fixture(scope="module")
def device_asm():
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not installed")
    srcs = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".hip"))
    d = tempfile.mkdtemp(prefix="moe_asm_")
    try:
        with ThreadPoolExecutor(max_workers=8) as ex:
            outs = list(ex.map(lambda s: compile_asm(s, d), srcs))
        yield {os.path.basename(o): open(o).read() for o in outs}
    finally:
        shutil.rmtree(d, ignore_errors=True)


def kernels(asm: str):
    """(kernel name, its instruction text, private segment bytes) per kernel."""
    out = []
    for m in re.finditer(r"^(_Z\S+):\s*;\s*@\S+\n(.*?)^\.Lfunc_end", asm, re.S | re.M):
        name = m.group(1)
        body = m.group(2)
        priv = re.search(rf"\.amdhsa_kernel {re.escape(name)}\n(?:.*\n)*?\s*\.amdhsa_private_segment_fixed_size (\d+)", asm)
        out.append((name, body, int(priv.group(1)) if priv else 0))
    return out


def short(name: str) -> str:
    m = re.search(r"N_1\d+(\w+?kernel)", name) or re.search(r"(\w+kernel)", name)
    return m.group(1) if m else name


def test_every_source_compiles_to_kernels(device_asm):
    found = {f: len(kernels(a)) for f, a in device_asm.items()}
    assert all(n > 0 for f, n in found.items() if f != "abi.s"), found


def test_no_out_of_line_calls_or_flat_accesses(device_asm):
    bad = []
    for f, asm in device_asm.items():
        for name, body, _ in kernels(asm):
            if "s_swappc" in body:
                bad.append((f, short(name), "call"))
            if re.search(r"\bflat_(load|store|atomic)", body):
                bad.append((f, short(name), "flat"))
    assert not bad, bad


def test_no_unexpected_scratch(device_asm):
    bad = []
    for f, asm in device_asm.items():
        for name, _, priv in kernels(asm):
            if priv > SCRATCH_ALLOWED.get(short(name), 0):
                bad.append((f, short(name), priv))
    assert not bad, bad


# ---- wait states around inline assembly ---------------------------------------
# The compiler inserts the wait states that gfx9 instructions need, but does not
# look into inline assembly. A vector memory instruction may read a scalar
# register no sooner than 5 wait states after a vector instruction (readfirstlane,
# readlane, a compare) wrote it, and an LDS load its M0 no sooner than 1 after
# any write.
VMEM_AFTER_VALU, LDS_AFTER_M0 = 5, 1


def lines_of(body: str):
    """(instruction, its labels before it) in order."""
    out, labels = [], []
    for raw in body.split("\n"):
        t = raw.split(";")[0].split("//")[0].strip()
        if t.endswith(":"):
            labels.append(t[:-1])
        elif t and not t.startswith("."):
            out.append((t, labels))
            labels = []
    return out


def scalar_regs(text: str):
    """Numbers of the scalar registers named in `text` ("m0" as it is)."""
    regs = set()
    for m in re.finditer(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b|\b(m0|vcc)\b", text):
        if m[1]:
            regs |= set(range(int(m[1]), int(m[2]) + 1))
        else:
            regs.add(int(m[3]) if m[3] else m[4])
    return regs


def too_soon(body: str):
    """(reader, writer, wait states between) of every vector memory
    instruction that reads scalar registers too soon, over all ways there."""
    ins = lines_of(body)
    jumps: dict[str, list[int]] = {}
    for i, (t, _) in enumerate(ins):
        m = re.match(r"s_c?branch\w* (\S+)", t)
        if m:
            jumps.setdefault(m[1], []).append(i)
    bad = []

    def back(i, waited, needs, reader):
        """Walks back from before instruction i."""
        for label in ins[i][1]:
            for j in jumps.get(label, []):
                look(j, waited, needs, reader)
        if i > 0 and not re.match(r"s_branch|s_endpgm|s_setpc", ins[i - 1][0]):
            look(i - 1, waited, needs, reader)

    def look(i, waited, needs, reader):
        needs = {r: n for r, n in needs.items() if n[0] > waited or n[1] > waited}
        if not needs:
            return
        t = ins[i][0]
        op, _, args = t.partition(" ")
        first = scalar_regs(args.split(",")[0])
        for r in first & set(needs):
            valu, salu = needs[r]
            if op.startswith("v_") and waited < valu or op.startswith("s_") and waited < salu:
                bad.append((reader, t, waited))
        left = {r: n for r, n in needs.items() if r not in first}
        nop = re.match(r"s_nop (\d+)", t)
        back(i, waited + (int(nop[1]) + 1 if nop else 1), left, reader)

    for i, (t, _) in enumerate(ins):
        m = re.match(r"(global|buffer|flat|scratch)_(load|store|atomic)", t)
        if m:
            needs = {r: (VMEM_AFTER_VALU, 0) for r in scalar_regs(t.partition(" ")[2])}
            if "_lds_" in t:
                needs["m0"] = (VMEM_AFTER_VALU, LDS_AFTER_M0)
            back(i, 0, needs, t)
    return bad


def test_the_wait_states_are_counted():
    load = "\tglobal_load_lds_dword v1, s[0:1]\n"
    assert too_soon("\tv_readfirstlane_b32 s1, v3\n\ts_mov_b32 m0, s2\n\ts_nop 0\n" + load) \
        == [(load.strip(), "v_readfirstlane_b32 s1, v3", 2)]
    assert not too_soon("\tv_readfirstlane_b32 s1, v3\n\ts_mov_b32 m0, s2\n\ts_nop 3\n" + load)
    assert too_soon("\ts_mov_b32 m0, s2\n" + load) and not too_soon("\ts_mov_b32 m0, s2\n\ts_nop 0\n" + load)
    assert too_soon("\tv_readfirstlane_b32 m0, v2\n\ts_nop 3\n" + load)
    # a later write of the register is the one that counts, and ways over branches too
    assert not too_soon("\tv_readfirstlane_b32 s1, v3\n\ts_mov_b32 s1, s2\n" + load.replace("_lds", ""))
    way = "\ts_nop 7\n\ts_branch .L1\n.L0:\n\tv_readlane_b32 s0, v3, 1\n\ts_cbranch_vccnz .L2\n\ts_endpgm\n.L1:\n.L2:\n"
    assert ("v_readlane_b32 s0, v3, 1", 1) in [b[1:] for b in too_soon(way + load)]


def test_scalar_operands_of_memory_instructions_are_not_read_too_soon(device_asm):
    bad = []
    for f, asm in device_asm.items():
        for name, body, _ in kernels(asm):
            for reader, writer, waited in too_soon(body):
                bad.append((f, short(name), reader, writer, waited))
    assert not bad, (len(bad), bad[:5])
