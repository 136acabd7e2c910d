"""What attention over the 8-bit cache and over whole prompts refuse before anything touches a GPU, and
the steps' own checks."""
import ctypes
import math

import pytest

import nvfp4_block_sparse_gb300 as qsa
from test_abi_cpu import FAKE, geom, lib  # noqa: F401  (lib: a fixture)
from test_dense_abi_cpu import at

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4


def ref(g):
    return None if g is None else ctypes.byref(g)


def dense(lib, g, **bad):  # noqa: F811
    a = dict(q=FAKE, kp=FAKE, ke=FAKE, vp=FAKE, ve=FAKE, sm=0.1, pt=FAKE, sl=FAKE, window=0, sinks=None, out=FAKE,
             lse=FAKE, ws=FAKE, n=lib.qsa_dense_attention_fp8_workspace_bytes(ref(g))) | bad
    return lib.qsa_dense_attention_fp8(ref(g), a["q"], a["kp"], a["ke"], a["vp"], a["ve"], a["sm"], a["pt"], a["sl"],
                                       a["window"], a["sinks"], a["out"], a["lse"], a["ws"], a["n"], None)


@pytest.mark.parametrize("bad", [dict([(n, None)]) for n in ("q", "kp", "ke", "vp", "ve", "pt", "sl", "out", "lse")]
                         + [dict([(n, at(264))]) for n in ("q", "kp", "ke", "vp", "ve", "out")]
                         + [dict(window=-1), dict(sm=0.0), dict(sm=-1.0), dict(sm=math.inf), dict(sm=math.nan)])
@pytest.mark.parametrize("rows", [1, 40])
def test_dense_refused(lib, bad, rows):  # noqa: F811
    assert dense(lib, geom(rows_per_req=rows), **bad) == INVALID


def test_dense_workspace_and_geometry(lib):  # noqa: F811
    for g in (geom(), geom(rows_per_req=5), geom(rows_per_req=4096), geom(head_dim=256, rows_per_req=77)):
        need = lib.qsa_dense_attention_fp8_workspace_bytes(ref(g))
        assert need > 0 and need % 256 == 0
        assert dense(lib, g, n=need - 1) == WORKSPACE
        assert dense(lib, g, ws=None) == WORKSPACE and dense(lib, g, ws=at(256 + 128)) == WORKSPACE
    wide = geom(num_q_heads=129, num_kv_heads=1)
    assert lib.qsa_dense_attention_fp8_workspace_bytes(ref(wide)) == 0
    assert dense(lib, wide, n=1 << 30) == UNSUPPORTED
    assert dense(lib, None) == INVALID and lib.qsa_dense_attention_fp8_workspace_bytes(None) == 0


def prompt(lib, g, **bad):  # noqa: F811
    a = dict(q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, cu=FAKE, T=100, sm=0.1, window=0, sinks=None, out=FAKE,
             lse=FAKE, ws=FAKE, n=256) | bad
    return lib.qsa_prompt_attention(ref(g), a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["cu"], a["T"],
                                    a["sm"], a["window"], a["sinks"], a["out"], a["lse"], a["ws"], a["n"], None)


@pytest.mark.parametrize("bad", [dict([(n, None)]) for n in ("q", "k", "v", "cu", "out", "lse")]
                         + [dict([(n, at(264))]) for n in ("q", "k", "v", "out")]
                         + [dict(qs=1016), dict(ks=248), dict(vs=260), dict(qs=1 << 39), dict(ks=1 << 39),
                            dict(vs=1 << 39), dict(qs=-1024), dict(T=-1), dict(T=(1 << 24) + 1), dict(window=-1),
                            dict(sm=0.0), dict(sm=math.inf), dict(sm=math.nan)])
def test_prompt_refused(lib, bad):  # noqa: F811
    assert prompt(lib, geom(), **bad) == INVALID


def test_prompt_workspace_and_geometry(lib):  # noqa: F811
    assert lib.qsa_prompt_attention_workspace_bytes(ref(geom()), 100) == 256
    for g, rows in ((None, 100), (geom(), -1), (geom(), (1 << 24) + 1), (geom(num_q_heads=129, num_kv_heads=1), 5),
                    (geom(head_dim=64), 5)):
        assert lib.qsa_prompt_attention_workspace_bytes(ref(g), rows) == 0
    assert prompt(lib, geom(), n=255) == WORKSPACE and prompt(lib, geom(), ws=None) == WORKSPACE
    assert prompt(lib, geom(), ws=at(128)) == WORKSPACE
    assert prompt(lib, geom(num_q_heads=129, num_kv_heads=1), qs=129 * 128, ks=128, vs=128) == UNSUPPORTED
    assert prompt(lib, geom(head_dim=192)) == UNSUPPORTED and prompt(lib, None) == INVALID


def test_steps_refused():
    g = dict(batch=2, rows_per_req=1, num_q_heads=8, num_kv_heads=2, head_dim=128, index_dim=64, page_size=64,
             max_blocks=16, num_pages=32)
    with pytest.raises(ValueError):
        qsa.DenseStep(g, cache="bf16", device="cpu")
    with pytest.raises(qsa.QsaError):
        qsa.PromptStep(dict(g, head_dim=64), 10, device="cpu")
    with pytest.raises(qsa.QsaError):
        qsa.PromptStep(dict(g, num_kv_heads=3), 10, device="cpu")
