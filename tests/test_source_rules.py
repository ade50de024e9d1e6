"""Rules on the HIP sources that no compiler check enforces.

Every inline-asm statement that writes M0 (the LDS base of gfx950's
global -> LDS copies) must name it in its clobber list, so that the compiler
orders the statement against its own uses of M0. No hand-written packed FP32
arithmetic appears anywhere (the build also turns the compiler's own off).
"""

import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int8_hadamard_domain_amd", "csrc")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC, "*.hpp")))


def _asm_statements(text):
    """Every `asm volatile(...)` / `asm(...)` statement of a source, whole."""
    out = []
    for m in re.finditer(r"\basm\s*(volatile\s*)?\(", text):
        i, depth = m.end() - 1, 0
        while True:
            c = text[i]
            if c == '"':                       # skip string literals (may hold parentheses)
                i += 1
                while text[i] != '"':
                    i += 2 if text[i] == "\\" else 1
            elif c == "(":
                depth += 1
            elif c == ")":
                depth -= 1
                if depth == 0:
                    break
            i += 1
        out.append(text[m.start():i + 1])
    return out


def _writes_m0(stmt):
    # the template strings: an instruction whose destination (first operand) is m0
    tmpl = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', stmt.split(":")[0]))
    return re.search(r"\b[sv]_\w+\s+m0\s*,", tmpl.replace("\\n", "\n").replace("\\t", " ")) is not None


def test_asm_writing_m0_declares_the_clobber():
    found = 0
    for path in _sources():
        with open(path) as f:
            text = f.read()
        for stmt in _asm_statements(text):
            if _writes_m0(stmt):
                found += 1
                clobbers = stmt.split(":")[-1]
                assert '"m0"' in clobbers, f"{os.path.basename(path)}: asm writes m0 without declaring it: {stmt}"
    assert found > 0   # the copy helpers exist, so the check is not vacuous


def test_checker_sees_a_missing_clobber():
    bad = 'asm volatile("s_mov_b32 m0, %1\\n\\tglobal_load_lds_dword %0, off" ::"v"(p), "s"(l) : "memory");'
    good = bad.replace(': "memory")', ': "memory", "m0")')
    (sb,), (sg,) = _asm_statements(bad), _asm_statements(good)
    assert _writes_m0(sb) and '"m0"' not in sb.split(":")[-1]
    assert _writes_m0(sg) and '"m0"' in sg.split(":")[-1]
    assert not _writes_m0('asm volatile("" : "+v"(x));')


def test_no_hand_written_packed_fp32():
    for path in _sources():
        with open(path) as f:
            text = f.read()
        assert not re.search(r"v_pk_(add|mul|fma)_f32", text), os.path.basename(path)


def test_asm_of_several_instructions_keeps_outputs_apart_from_inputs():
    """An output that an instruction writes while a later one still reads an input may not share a register with that
    input: in statements of more than one vector instruction every output is early-clobber (&)."""
    found = 0
    for path in _sources():
        with open(path) as f:
            text = f.read()
        macros = dict(re.findall(r"#define (I8H_\w+)[ \\\n]+((?:[^\n]*\\\n)*[^\n]*)", text))
        for stmt in _asm_statements(text):
            for name in re.findall(r"\bI8H_\w+", stmt):
                stmt = stmt.replace(name, macros.get(name, name))
            template, *operands = stmt.split(":")
            if operands and len(re.findall(r"I8H_SEL\(|\bv_\w+", template)) > 1:
                for constraint in re.findall(r'"([=+][^"]*)"', operands[0]):
                    found += 1
                    assert "&" in constraint, f"{os.path.basename(path)}: output {constraint} without & in {stmt}"
    assert found > 0


def test_lds_that_lanes_of_a_wave_hand_on_is_ordered():
    """LDS that a wave's lanes write for its other lanes, without a workgroup barrier: wave_lds_order() stands between
    the write and the reads, and between the reads and the next write."""
    with open(os.path.join(CSRC, "moe_mx.hip")) as f:
        text = f.read()
    calls = [m.start() for m in re.finditer(r"^\s*store_sc\(\);", text, flags=re.M)]
    assert calls
    for at in calls:
        before, after = text[:at].rstrip().split("\n")[-1], text[at:].strip().split("\n")[1]
        assert "wave_lds_order();" in before and "wave_lds_order();" in after
    with open(os.path.join(CSRC, "moe_mx_few.hip")) as f:
        text = f.read()
    body = text[text.index("for (int j = wave; j < k; j += waves) {"):text.index("part[j][4 * g + i]")]
    write, read = body.index("*reinterpret_cast<uint32_t*>(&row["), body.index("reinterpret_cast<const u32x4*>(&row[")
    assert "wave_lds_order();" in body[:write] and "wave_lds_order();" in body[write:read]
