"""Inline assembly in the device sources against the hardware's rules that the compiler does not apply inside it (no GPU)."""
import glob
import os
import re

import mxfp8_quantized_moe_amd

CSRC = os.path.join(os.path.dirname(mxfp8_quantized_moe_amd.__file__), "csrc")
ASM = re.compile(r'\basm\s*(?:volatile)?\s*\(\s*((?:"[^"]*"\s*)+)')


def statements():
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        with open(path) as f:
            for m in ASM.finditer(f.read()):
                yield os.path.basename(path), "".join(re.findall(r'"([^"]*)"', m.group(1))).replace("\\n", "\n").replace("\\t", " ")


def test_wide_stores_keep_their_data():
    """A vector instruction may overwrite the data of a store of more than 64 bits two wait states after it, not sooner; around
    inline assembly the compiler does not see the store, so the wait states stand behind it in the same block."""
    found = list(statements())
    assert found, "no inline assembly was found: the pattern no longer fits the sources"
    for name, text in found:
        lines = [l.strip() for l in text.split("\n") if l.strip()]
        for i, line in enumerate(lines):
            if re.match(r"(global|flat|buffer|scratch)_store_dwordx[34]\b", line):
                nop = re.match(r"s_nop (\d+)", lines[i + 1]) if i + 1 < len(lines) else None
                assert nop and int(nop.group(1)) >= 1, (name, line)
