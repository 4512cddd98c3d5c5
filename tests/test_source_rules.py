"""Rules of the kernels' sources that no run would show."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "compressed_index_matmul_amd", "csrc")


def asm_statements():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.hip"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"\basm\s*(?:volatile\s*)?\((.*?)\)\s*;", text, re.S):
            yield os.path.basename(path), m.group(1)


def test_inline_assembly_names_the_scalar_registers_it_writes():
    """A statement whose text writes m0, vcc or exec has to say so, or the
    compiler may keep a value of its own there."""
    seen = 0
    for path, body in asm_statements():
        text, _, rest = body.partition("::") if "::" in body else body.partition(":")
        for reg in re.findall(r"\b(?:s|v)_\w+\s+(m0|vcc|exec)\b", text):
            seen += 1
            assert f'"{reg}"' in rest, f"{path}: {reg} is written and not named: {body}"
    assert seen >= 1
