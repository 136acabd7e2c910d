"""The bounds-checked build reports failed checks in the 8-bit cache's and the prompt attention's kernels
as in the others: declared codes are distinct, of the file's own number, and used."""
import os
import re

import pytest

import nvfp4_block_sparse_gb300 as qsa

CSRC = os.path.join(os.path.dirname(qsa.__file__), "csrc")
CHECKS = {"qsa_cache8.cu": ("B", {"Row", "Load"}), "qsa_dense8.cu": ("C", {"Chunk", "Out", "Join"}),
          "qsa_prompt.cu": ("D", {"Unit", "Out"})}


@pytest.mark.parametrize("name", sorted(CHECKS))
def test_kernels_check_what_the_header_names(name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    number, kinds = CHECKS[name]
    codes = dict(re.findall(r"constexpr int kChk(\w+) = 0x(\w+)", text))
    assert set(codes) == kinds and len(set(codes.values())) == len(codes)
    assert all(c.startswith(number + "0") for c in codes.values())
    uses = text.replace("constexpr int kChk", "")
    for code in codes:
        assert re.search(r"\bkChk%s\b" % code, uses), (name, code)
    assert "QSA_BOUNDS_READER(" in text
