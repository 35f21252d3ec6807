"""Matrix instructions written in inline asm are invisible to the compiler's
hazard handling: whatever it places behind the asm statement (a copy, a spill
or a reload of an accumulator) may come before their results are written.  So
every asm statement that holds one waits for them itself.  Read from the
sources; nothing is run."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_grouped_gemm_gmm_amd", "csrc")
# wait states between a matrix instruction and the first read or overwrite of its result by anything else:
# what the compiler keeps for its own builtin of a 32 x 32 x 16 bf16 product on gfx950 (s_nop 11)
RESULT = 12
# between a vector write of an operand and the matrix instruction
OPERAND = 2


def statements():
    """(file, line, instructions) of every asm statement that holds a matrix instruction."""
    out = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC, "*.hpp"))):
        text = open(path).read()
        for m in re.finditer(r"\basm\s+volatile\s*\(", text):
            body = text[m.end():]
            end = re.search(r"\n?\s*:(?=[\s\"])", re.sub(r'"(?:[^"\\]|\\.)*"', lambda s: "_" * len(s.group()), body))
            code = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', body[:end.start()]))
            lines = [i.strip() for i in re.split(r"\\n\\t|\\n", code) if i.strip()]
            if any("mfma" in i for i in lines):
                out.append((os.path.basename(path), text.count("\n", 0, m.start()) + 1, lines))
    return out


def states(lines):
    """Wait states that the instructions are certain to take."""
    return sum(int(i.split()[1]) + 1 if i.startswith("s_nop") else 1 for i in lines)


def test_there_are_some():
    assert len(statements()) >= 6


@pytest.mark.parametrize("where,line,code", statements(), ids=["%s:%d" % s[:2] for s in statements()])
def test_results_and_operands(where, line, code):
    mfma = [i for i, c in enumerate(code) if "mfma" in c]
    nops = [c for c in code[mfma[-1] + 1:] if c.startswith("s_nop")]
    assert states(nops) >= RESULT, "%s:%d ends before its last result is written" % (where, line)
    assert states(code[:mfma[0]]) >= OPERAND, "%s:%d starts before its operands are written" % (where, line)
    # operands loaded by the statement itself are not used by it: a load's result needs a wait first
    loaded = {c.split()[1].rstrip(",") for c in code if c.startswith("ds_read")}
    for i in mfma:
        assert not loaded & {a.strip() for a in code[i].split(None, 1)[1].split(",")}
    if loaded:
        assert code[-1] == "s_waitcnt lgkmcnt(0)"
