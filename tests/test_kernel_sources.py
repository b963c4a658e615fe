"""What the kernels' inline assembly has to declare, read from the sources (no GPU needed)."""
import glob
import os
import re

import grouped_gemm_expert_router_amd.build as build


def asm_statements():
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*.h*"))):
        with open(path) as f:
            text = f.read()
        for m in re.finditer(r"\basm\s+volatile\s*\((.*?)\);", text, re.S):
            yield f"{os.path.basename(path)}:{text.count(chr(10), 0, m.start()) + 1}", m.group(1)


def test_assembly_that_writes_m0_says_so():
    """Otherwise the compiler may keep a value of its own there across the statement."""
    seen = 0
    for where, text in asm_statements():
        if re.search(r"\bm0\s*,", text):
            seen += 1
            assert '"m0"' in text.rsplit(":", 1)[1], where
    assert seen >= 4
