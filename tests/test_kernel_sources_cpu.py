"""What the kernels' sources may not hold: inline assembly with instructions.  The
compiler places the wait states that matrix instructions, scalar loads and LDS
transfers require before their results are read, but not for the operands of an
inline assembly statement, so every instruction comes from an operation it knows.
(A statement with an empty template, which only hides a value from the optimiser,
holds none.)"""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ASM = re.compile(r"\b(?:asm|__asm__|__asm)\b(?:\s+(?:volatile|__volatile__))?\s*\(\s*((?:\"(?:[^\"\\]|\\.)*\"\s*)*)")


def test_no_instruction_in_inline_assembly():
    files = sorted(glob.glob(os.path.join(ROOT, "segmented_gather_rank_amd", "csrc", "*")))
    assert len(files) > 10
    for path in files:
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in ASM.finditer(text):
            assert m.group(1).strip() == '""', f"{os.path.basename(path)}: {m.group(0)}"
