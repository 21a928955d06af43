"""Inline assembly of the kernels: what it changes behind the compiler's back (read from the sources)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int8_matmul_amd", "csrc")
FILES = sorted(glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC, "*.h")))


def statements(src):
    """The asm statements, from the keyword to the semicolon that ends them outside of quotes."""
    for m in re.finditer(r"\basm\b[^(;{]*\(", src):
        i, quoted = m.end(), False
        while quoted or src[i] != ";":
            quoted ^= src[i] == '"' and src[i - 1] != "\\"
            i += 1
        yield src[m.start():i]


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_m0_is_an_operand_where_it_is_used(path):
    """M0, which the compiler's own LDS loads use too, is set by an operand's constraint and never inside the text."""
    for st in statements(re.sub(r"//[^\n]*", "", open(path).read())):
        text = " ".join(re.findall(r'"((?:[^"\\]|\\.)*)"', st.split(":")[0]))
        assert not re.search(r"\bm0\b", text), st
        if re.search(r"\blds\b", text):
            assert '"{m0}"(' in st, st
