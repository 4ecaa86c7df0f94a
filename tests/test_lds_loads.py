"""Loads from memory straight into LDS that the kernels write in inline asm, where the compiler neither sees the load nor
what it needs before it:
  * an SGPR that a vector instruction wrote (v_readlane, as for a spilled SGPR) may be read by a memory instruction only
    five wait states later;
  * m0, the LDS address, may be read by the load only one wait state after it was written, and the compiler has to know
    that it was overwritten.
An instruction is one wait state, s_nop N is N + 1.  Each asm statement has to hold them itself: what stands before it is
the register allocator's choice."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dynamic_vocab_draft_amd", "csrc")


def asm_statements(text):
    """(instructions, what follows the asm's text) of each asm statement."""
    for m in re.finditer(r'\basm\s*(?:volatile)?\s*\(\s*((?:"(?:[^"\\]|\\.)*"\s*)+)(.*?)\)\s*;', text, re.S):
        code = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', m[1]))
        yield [i.strip() for i in re.split(r"\\n|;", code.replace("\\t", " ")) if i.strip()], m[2]


def statements():
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            for code, rest in asm_statements(f.read()):
                yield name, code, rest


def wait_states(code):
    return sum(int(i.split()[1], 0) + 1 if i.startswith("s_nop") else 1 for i in code)


def test_parser():
    text = 'asm volatile("s_mov_b32 m0, %3\\n\\ts_nop 2\\n\\t"\n "buffer_load_dword %0, off lds" : : "v"(a), "s"(f(b)) : "memory", "m0");'
    (code, rest), = asm_statements(text)
    assert code == ["s_mov_b32 m0, %3", "s_nop 2", "buffer_load_dword %0, off lds"]
    assert wait_states(code[:2]) == 4 and '"m0"' in rest


def test_memory_instructions_wait_for_scalar_registers():
    found = 0
    for name, code, rest in statements():
        for at, i in enumerate(code):
            if re.match(r"(buffer|global|flat|scratch)_", i):
                found += 1
                assert wait_states(code[:at]) >= 5, f"{name}: {code}"
    assert found >= 3


def test_written_m0_is_declared():
    found = 0
    for name, code, rest in statements():
        if any(re.match(r"\w+ m0,", i) for i in code):
            found += 1
            assert re.search(r':[^:]*"m0"', rest), f"{name}: {code}"
            at = next(n for n, i in enumerate(code) if re.match(r"\w+ m0,", i))
            assert at + 2 < len(code) and wait_states(code[at + 1:-1]) >= 1, f"{name}: {code}"
    assert found >= 3
