"""CPU test of the kernel sources' inline asm: a statement that writes a fixed
register names it as clobbered, so that the compiler keeps no value there."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dequantize_amax_reduce_amd", "csrc")
FIXED = r"m0|vcc|exec|scc|[sv]\d+|[sv]\[\d+:\d+\]"


def asm_statements():
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"\basm\s+(?:volatile\s*)?\(", text):
            depth, i = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(text[i], 0)
                i += 1
            yield os.path.basename(path), text[m.end():i - 1]


def test_written_registers_are_clobbers():
    seen = 0
    for name, stmt in asm_statements():
        parts = re.split(r":(?=(?:[^\"]*\"[^\"]*\")*[^\"]*$)", stmt)      # colons outside strings
        code = "".join(re.findall(r'"([^"]*)"', parts[0]))
        clobbers = re.findall(r'"([^"]*)"', parts[3]) if len(parts) > 3 else []
        for ins in re.split(r"\\n|;", code):
            m = re.match(r"(?:\\t|\s)*[sv]_\w+\s+(" + FIXED + r")\s*,", ins)
            if m:
                seen += 1
                assert m.group(1) in clobbers, f"{name}: asm writes {m.group(1)} and does not name it: {stmt.strip()}"
    assert seen >= 2                                        # the two loads to LDS write m0
