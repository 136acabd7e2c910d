"""What the calls on several-axes rotations and on the 8-bit cache's rows refuse
before anything touches a GPU, and the rotation plans of several axes."""
import ctypes

import numpy as np
import pytest

import cache8_reference as c8
from nvfp4_block_sparse_gb300 import binding
from test_abi_cpu import FAKE, geom, lib  # noqa: F401  (lib: a fixture)
from test_dense_abi_cpu import at, config, turns

INVALID, UNSUPPORTED = 1, 2


def axes(lib, pairs, layout=0, n=None, plan=None, **kw):  # noqa: F811
    plan = binding.qsa_rope_axes_t() if plan is None else plan
    kw.setdefault("rotary_dim", 2 * sum(pairs))
    st = lib.qsa_rope_axes_init(ctypes.byref(config(**kw)), len(pairs) if n is None else n,
                                (ctypes.c_int * 8)(*pairs), layout, ctypes.byref(plan))
    return st, plan


@pytest.mark.parametrize("layout,name", [(0, "sections"), (1, "interleaved"), (2, "spectra")])
@pytest.mark.parametrize("pairs", [[64], [32, 32], [16, 24, 24], [24, 20, 20], [1, 3, 3, 1], [125, 1, 1, 1]])
def test_axes_plans(lib, layout, name, pairs):  # noqa: F811
    st, plan = axes(lib, pairs, layout)
    axis = c8.axis_of(pairs, name)
    if [axis.count(a) for a in range(len(pairs))] != pairs:      # these counts do not interleave
        assert st == INVALID
        return
    assert st == 0 and plan.axes == len(pairs) and list(plan.axis) == axis + [0] * (128 - len(axis))
    if name == "spectra":
        theta, i = 1e6, 0
        for n in pairs:
            f = theta ** (-np.arange(n) / n) / (2 * np.pi)
            got = np.array([t / 2.0**64 for t in plan.rope.turns[i:i + n]])
            assert np.abs(got - f).max() <= 16 * 2.0**-53
            i += n
    else:
        assert list(plan.rope.turns) == list(turns(lib, rotary_dim=2 * sum(pairs)).turns)


@pytest.mark.parametrize("bad", [
    dict(pairs=[64], n=0), dict(pairs=[64], n=5), dict(pairs=[32, 31]), dict(pairs=[32, 33], rotary_dim=128),
    dict(pairs=[64, 0]), dict(pairs=[65, -1], rotary_dim=128), dict(pairs=[60]), dict(pairs=[10, 27, 27], layout=1),
    dict(pairs=[64], layout=3), dict(pairs=[64], layout=-1), dict(pairs=[64], theta=1.0),
    dict(pairs=[2**31 - 1, 65], rotary_dim=128), dict(pairs=[64], scaling=2, low=0.0)])
def test_axes_plans_refused(lib, bad):  # noqa: F811
    plan = binding.qsa_rope_axes_t()
    plan.axes = 77
    assert axes(lib, plan=plan, **bad)[0] == INVALID
    assert plan.axes == 77                                       # left as it was


def test_axes_null(lib):  # noqa: F811
    plan, three = binding.qsa_rope_axes_t(), (ctypes.c_int * 1)(32)
    c = config(rotary_dim=64)
    assert lib.qsa_rope_axes_init(None, 1, three, 0, ctypes.byref(plan)) == INVALID
    assert lib.qsa_rope_axes_init(ctypes.byref(c), 1, None, 0, ctypes.byref(plan)) == INVALID
    assert lib.qsa_rope_axes_init(ctypes.byref(c), 1, three, 0, None) == INVALID


def test_axes_rows_refused(lib):  # noqa: F811
    plan = axes(lib, [16, 24, 24])[1]
    call = lambda p=plan, x=FAKE, n=5, c=FAKE: lib.qsa_rope_axes_rows(  # noqa: E731
        None if p is None else ctypes.byref(p), x, n, c, None)
    assert call(p=None) == INVALID and call(x=None) == INVALID and call(c=None) == INVALID
    assert call(n=-1) == INVALID and call(n=(1 << 24) + 1) == INVALID and call(c=at(264)) == INVALID
    assert call(p=binding.qsa_rope_axes_t()) == INVALID          # never filled
    for field, value in (("axes", 0), ("axes", 5), ("axes", 2)):  # axes its pairs do not have
        p = axes(lib, [16, 24, 24])[1]
        setattr(p, field, value)
        assert call(p=p) == INVALID


ROWS = dict(k=FAKE, ks=256, v=FAKE, vs=256, cu=None, n=0, table=FAKE, lens=FAKE, kp=FAKE, ke=FAKE, vp=FAKE, ve=FAKE)


@pytest.mark.parametrize("bad,want", [
    (dict(g=None), INVALID), (dict(g=dict(rows_per_req=4097)), UNSUPPORTED), (dict(g=dict(head_dim=64)), UNSUPPORTED),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(ks=128), INVALID), (dict(vs=260), INVALID),
    (dict(k=at(264)), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(kp=None), INVALID),
    (dict(ke=None), INVALID), (dict(vp=None), INVALID), (dict(ve=None), INVALID), (dict(kp=at(264)), INVALID),
    (dict(vp=at(264)), INVALID), (dict(cu=FAKE, n=-1), INVALID), (dict(cu=FAKE, n=(1 << 24) + 1), INVALID)])
def test_store_and_load_refused(lib, bad, want):  # noqa: F811
    a = dict(ROWS, g={}) | bad
    g = None if a["g"] is None else ctypes.byref(geom(**a["g"]))
    assert lib.qsa_store_kv_tokens_fp8(g, a["k"], a["ks"], a["v"], a["vs"], a["cu"], a["n"], a["table"], a["lens"],
                                       a["kp"], a["ke"], a["vp"], a["ve"], None) == want
    if "ks" in bad or "vs" in bad:
        return
    assert lib.qsa_load_kv_tokens_fp8(g, a["cu"], a["n"], a["table"], a["lens"], a["kp"], a["ke"], a["vp"], a["ve"],
                                      a["k"], a["v"], None) == want
