"""The bounds-checked build reports failed checks of every kind that the header
names: in each kernel source that copies pages, the copies' page ids and token
offsets; in each that writes attention outputs or records, their rows and units."""
import os
import re

import pytest

import nvfp4_block_sparse_gb300 as qsa

CSRC = os.path.join(os.path.dirname(qsa.__file__), "csrc")
CHECKS = {
    "qsa_attend.cu": {"Chunk", "Record", "Unit"}, "qsa_sparse_decode.cu": {"Chunk", "Unit"},
    "qsa_sparse_prefill.cu": {"Chunk", "Out"}, "qsa_dense.cu": {"Chunk", "Out", "Join"},
    "qsa_dense_tile.cu": {"Chunk", "Out", "Record"}, "qsa_prologue.cu": {"Row", "Load"},
    "qsa_store_tokens.cu": {"Row"},
}


@pytest.mark.parametrize("name", sorted(CHECKS))
def test_kernels_check_what_the_header_names(name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    codes = dict(re.findall(r"constexpr int kChk(\w+) = (0x[0-9A-Fa-f]+)", text))
    assert CHECKS[name] <= set(codes), name
    assert len(set(codes.values())) == len(codes)
    uses = text.replace("constexpr int kChk", "")
    for code in codes:       # declared codes are reported somewhere
        assert re.search(r"\bkChk%s\b" % code, uses), (name, code)
