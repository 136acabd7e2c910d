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


def test_the_last_commits_are_waited_for():
    """An arrival that a commit sends may not be on its way when its block ends (the shared memory is then another
    block's): each barrier that MMAs are committed to is waited for to its last phase, the ones that no role waits for
    at the end by a lane each."""
    def text(name):
        return re.sub(r"\s+", " ", re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read()))
    prompt, tile = text("qsa_prompt.cu"), text("qsa_dense_tile.cu")
    committed = [set(re.findall(r"commit<CG>\((?:one|elect_one\(\)), &?(\w+)", t)) for t in (prompt, tile)]
    assert committed[0] == {"barS", "barO", "partO", "free_", "qfree", "mdone"}
    assert committed[1] == {"barS", "barO", "partO", "kfree", "vfree", "mdone"}
    tail = prompt[prompt.index("if (!dead) units.put(Unit{});"):prompt.index("warp == T::kRelay)")]
    for part in ("uint64_t* bar = stage ? &free_[lane] : o ? barO : qfree;",
                 "const int last = stage ? (pos - 1 - lane) / T::kStages : o ? pos / 2 - 1 : parts - 1;",
                 "dead = lanes_gave_up(bar, last,"):
        assert part in tail, part
    tail = tile[tile.index("any_dead = __syncthreads_or"):tile.index("tcgen05.dealloc")]
    for part in ("uint64_t* bar = o ? barO : lane & 2 ? &vfree[x] : &kfree[x];",
                 "lanes_gave_up(bar, o ? chunks - 1 : (chunks - 1 - x) >> 1,"):
        assert part in tail, part


def test_which_phases_are_the_last():
    """The phases waited for at the end: of 10 or 5 stages that chunks' K and V take in turn, and of two tiles."""
    for stages in (5, 10):
        for pos in range(0, 60, 2):
            uses = [sum(1 for p in range(pos) if p % stages == s) for s in range(stages)]
            for s in range(stages):
                assert (s < pos) == (uses[s] > 0)
                if s < pos:
                    assert (pos - 1 - s) // stages == uses[s] - 1
    for chunks in range(30):
        for x in range(2):
            uses = sum(1 for c in range(chunks) if c & 1 == x)
            assert (x < chunks) == (uses > 0) and (x >= chunks or (chunks - 1 - x) >> 1 == uses - 1)
