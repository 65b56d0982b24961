"""Inline assembly of the kernels: registers that it writes are operands or named as clobbered, so that the
compiler knows what they hold."""
import glob
import os
import re

from conftest import ROOT

CSRC = os.path.join(ROOT, "post_weight_quantization_30_amd", "csrc")
FIXED = r"(m0|vcc|exec|scc|s\[?\d|v\[?\d|a\[?\d)"


def statements(text):
    """(instructions, what follows them) of every asm statement."""
    text = re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)
    for m in re.finditer(r"\basm\s*(?:volatile)?\s*\(", text):
        depth, i, quoted = 1, m.end(), False
        while depth:
            c = text[i]
            if c == '"' and text[i - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            i += 1
        body = text[m.end():i - 1]
        code = re.match(r'(\s*"(?:[^"\\]|\\.)*")*', body).group(0)
        yield "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', code)), body[len(code):]


def hidden_writes(text):
    """Fixed registers that an instruction names first, its destination, without a mention in the
    operands or clobbers."""
    out = []
    for code, rest in statements(text):
        for line in re.split(r"\\n|;", code.replace("\\t", " ")):
            m = re.match(r"\s*[a-z]\w+\s+" + FIXED, line)
            if m and not re.match(r"\s*(s_waitcnt|s_nop|s_barrier|s_setprio)", line) and m.group(1) not in rest:
                out.append(line.strip())
    return out


def test_the_check_finds_what_it_looks_for():
    assert hidden_writes('asm volatile("s_mov_b32 m0, %0\\n\\ts_nop 0" ::"s"(x) : "memory");') == ["s_mov_b32 m0, %0"]
    assert not hidden_writes('asm volatile("s_mov_b32 m0, %0" ::"s"(x) : "memory", "m0");')
    assert not hidden_writes('asm volatile("s_nop 0\\n\\tglobal_load_lds_dwordx4 %0, off" ::"v"(x), "{m0}"(y) : "memory");')
    assert not hidden_writes('asm volatile("s_waitcnt vmcnt(0)" ::: "memory");')


def test_no_hidden_writes():
    files = sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.hip")))
    assert files
    for f in files:
        assert not hidden_writes(open(f).read()), f
