"""Every wait for tensor-memory loads takes the loaded values through it, so
that no use of them can be scheduled ahead of the wait (a bare wait orders
memory accesses, not arithmetic on registers)."""
import glob
import os
import re

import nvfp4_block_sparse_gb300 as qsa

CSRC = os.path.join(os.path.dirname(qsa.__file__), "csrc")


def test_no_bare_waits_for_tensor_memory_loads():
    waits = 0
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        bare = len(re.findall(r"\btmem_wait_ld\(\);", text))
        # the one in the helper itself
        assert bare == (1 if "void tmem_wait_ld_of(" in text else 0), path
        waits += len(re.findall(r"\btmem_wait_ld_of\(", text))
        assert text.count("tcgen05.wait::ld") == (1 if path.endswith("qsa_tc.cuh") else 0), path
    assert waits > 10
