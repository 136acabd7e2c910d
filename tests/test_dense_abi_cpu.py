"""What the prologue and dense attention calls refuse before anything touches a
GPU, and their host-side parts (rotation plans, workspace sizes)."""
import ctypes
import math

import numpy as np
import pytest

import cache_reference as cr
from nvfp4_block_sparse_gb300 import binding
from test_abi_cpu import FAKE, geom, lib  # noqa: F401  (lib: a fixture)

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4


def at(address):
    return ctypes.c_void_p(address)


# ---------------------------------------------------------------------------
# rotation plans
# ---------------------------------------------------------------------------

def config(**kw):
    c = dict(rotary_dim=64, scaling=0, theta=1e6, factor=4.0, original_context=8192.0, low=1.0,
             high=32.0, attention_factor=0.0)
    c.update(kw)
    return binding.qsa_rope_config_t(**c)


def turns(lib, **kw):  # noqa: F811
    plan = binding.qsa_rope_t()
    assert lib.qsa_rope_init(ctypes.byref(config(**kw)), ctypes.byref(plan)) == 0
    return plan


@pytest.mark.parametrize("bad", [
    dict(rotary_dim=0), dict(rotary_dim=8), dict(rotary_dim=72), dict(rotary_dim=272),
    dict(rotary_dim=-16), dict(scaling=-1), dict(scaling=4), dict(theta=1.0), dict(theta=0.0),
    dict(theta=math.nan), dict(theta=math.inf), dict(attention_factor=-1.0),
    dict(attention_factor=math.nan), dict(scaling=1, factor=0.0), dict(scaling=1, factor=-2.0),
    dict(scaling=2, factor=math.inf), dict(scaling=2, original_context=0.0),
    dict(scaling=2, low=0.0), dict(scaling=3, low=4.0, high=4.0), dict(scaling=3, low=8.0, high=4.0),
    dict(scaling=3, high=math.inf), dict(scaling=3, original_context=math.nan),
])
def test_rope_plans_refused(lib, bad):  # noqa: F811
    plan = binding.qsa_rope_t()
    assert lib.qsa_rope_init(ctypes.byref(config(**bad)), ctypes.byref(plan)) == INVALID
    assert lib.qsa_rope_init(None, ctypes.byref(plan)) == INVALID
    assert lib.qsa_rope_init(ctypes.byref(config()), None) == INVALID


@pytest.mark.parametrize("scaling,name", [(0, "none"), (1, "linear"), (2, "yarn"), (3, "wavelength")])
@pytest.mark.parametrize("rot,theta", [(16, 1.5), (64, 1e4), (256, 1e8)])
def test_rope_plan_frequencies(lib, scaling, name, rot, theta):  # noqa: F811
    plan = turns(lib, rotary_dim=rot, scaling=scaling, theta=theta)
    f, amp = cr.freqs(rot, theta, name, 4.0, 8192.0, 1.0, 32.0)
    got = np.array([t / 2.0**64 for t in plan.turns[:rot // 2]])
    # a few 53-bit roundings of a frequency (power, interpolation, division by 2 pi)
    ref = f / (2 * math.pi)
    ref = ref - np.floor(ref)
    assert np.abs(got - ref).max() <= 16 * 2.0**-53 * max(1.0, f.max())
    assert plan.rotary_dim == rot and not any(plan.turns[rot // 2:])
    assert abs(plan.amplitude - amp) <= 2.0**-23 * amp


def test_rope_plan_attention_factor(lib):  # noqa: F811
    assert turns(lib, attention_factor=0.75).amplitude == 0.75
    assert turns(lib, scaling=2, factor=0.5).amplitude == 1.0      # (no ln of less than one)


def test_rope_rows_refused(lib):  # noqa: F811
    g, plan = geom(), turns(lib)
    call = lambda g=g, p=plan, s=FAKE, o=None, c=FAKE: lib.qsa_rope_rows(  # noqa: E731
        None if g is None else ctypes.byref(g), None if p is None else ctypes.byref(p), s, o, c, None)
    assert call(g=None) == INVALID
    assert call(p=None) == INVALID
    assert call(p=binding.qsa_rope_t()) == INVALID            # never filled
    assert call(s=None) == INVALID
    assert call(c=None) == INVALID
    assert call(c=at(260)) == INVALID
    assert call(g=geom(rows_per_req=4097)) == UNSUPPORTED


# ---------------------------------------------------------------------------
# norms, append, read-back
# ---------------------------------------------------------------------------

def norm(**kw):
    c = dict(rotary_dim=64, interleaved=0, weight_plus_one=0, eps=1e-6)
    c.update(kw)
    return binding.qsa_norm_rope_t(**c)


NORM = dict(q=FAKE, q_stride=8 * 128, k=FAKE, k_stride=2 * 128, qw=FAKE, kw=FAKE, cs=FAKE,
            q_out=at(1 << 20), k_out=at(1 << 21))
BAD_NORM = [
    dict(n=None), dict(n=norm(rotary_dim=-16)), dict(n=norm(rotary_dim=24)),
    dict(n=norm(rotary_dim=144)), dict(n=norm(eps=-1.0)), dict(n=norm(eps=math.inf)),
    dict(n=norm(eps=math.nan)), dict(q=None), dict(q_out=None), dict(k=None),
    dict(q_stride=8 * 128 - 8), dict(q_stride=8 * 128 + 4), dict(q_stride=-1024),
    dict(q_stride=1 << 41), dict(k_stride=128), dict(k_stride=0), dict(q=at(264)), dict(k=at(258)),
    dict(qw=at(264)), dict(kw=at(2)), dict(cs=None), dict(cs=at(264)), dict(q_out=at(264)),
    # in place with rows further apart than the output's
    dict(q_out=FAKE, q_stride=8 * 128 + 8),
]
BAD_K_OUT = [dict(k_out=None), dict(k_out=at(264)), dict(k_out=FAKE, k_stride=2 * 128 + 8)]


def test_geometry_helper_is_the_one_assumed():
    g = geom()
    assert (g.num_q_heads, g.num_kv_heads, g.head_dim, g.page_size) == (8, 2, 128, 64)


@pytest.mark.parametrize("bad", BAD_NORM + BAD_K_OUT)
def test_qk_norm_rope_refused(lib, bad):  # noqa: F811
    a = dict(NORM, n=norm()) | bad
    st = lib.qsa_qk_norm_rope(ctypes.byref(geom()), None if a["n"] is None else ctypes.byref(a["n"]),
                              a["q"], a["q_stride"], a["k"], a["k_stride"], a["qw"], a["kw"], a["cs"],
                              a["q_out"], a["k_out"], None)
    assert st == INVALID


STORE = dict(NORM, v=FAKE, v_stride=2 * 128, ik=FAKE, ks=1.0, vs=1.0, pt=FAKE, sl=FAKE, kp=FAKE,
             ksf=FAKE, vp=FAKE, vsf=FAKE, ikp=FAKE)


@pytest.mark.parametrize("bad", BAD_NORM + [
    dict(v=None), dict(v=at(264)), dict(v_stride=128), dict(v_stride=2 * 128 + 4), dict(ik=None),
    dict(ik=at(2)), dict(ks=0.0), dict(ks=math.inf), dict(vs=-1.0), dict(vs=math.nan), dict(pt=None),
    dict(sl=None), dict(kp=None), dict(kp=at(258)), dict(ksf=None), dict(vp=None), dict(vp=at(1)),
    dict(vsf=None), dict(ikp=None), dict(ikp=at(257)),
])
def test_store_rope_refused(lib, bad):  # noqa: F811
    a = dict(STORE, n=norm()) | bad
    st = lib.qsa_store_kv_tokens_rope(
        ctypes.byref(geom()), None if a["n"] is None else ctypes.byref(a["n"]), a["q"], a["q_stride"],
        a["k"], a["k_stride"], a["v"], a["v_stride"], a["ik"], a["qw"], a["kw"], a["cs"], a["ks"],
        a["vs"], a["pt"], a["sl"], a["q_out"], a["kp"], a["ksf"], a["vp"], a["vsf"], a["ikp"], None)
    assert st == INVALID


@pytest.mark.parametrize("i,value", [(1, None), (2, None), (3, None), (4, None), (5, None), (6, None),
                                     (7, math.inf), (8, math.nan), (9, None), (10, None), (3, at(2)),
                                     (5, at(2)), (9, at(264)), (10, at(8))])
def test_load_refused(lib, i, value):  # noqa: F811
    a = [ctypes.byref(geom())] + [FAKE] * 6 + [1.0, 1.0, FAKE, FAKE, None]
    a[i] = value
    assert lib.qsa_load_kv_tokens(*a) == INVALID
    a = [ctypes.byref(geom(rows_per_req=4097))] + [FAKE] * 6 + [1.0, 1.0, FAKE, FAKE, None]
    assert lib.qsa_load_kv_tokens(*a) == UNSUPPORTED


# ---------------------------------------------------------------------------
# dense attention
# ---------------------------------------------------------------------------

def dense(lib, g, **bad):  # noqa: F811
    need = lib.qsa_dense_attention_workspace_bytes(ctypes.byref(g)) if g is not None else 0
    a = dict(q=FAKE, kp=FAKE, ksf=FAKE, vp=FAKE, vsf=FAKE, ks=1.0, vs=1.0, sm=0.1, pt=FAKE, sl=FAKE,
             window=0, sinks=None, out=FAKE, lse=FAKE, ws=FAKE, ws_bytes=need) | bad
    return lib.qsa_dense_attention(
        None if g is None else ctypes.byref(g), a["q"], a["kp"], a["ksf"], a["vp"], a["vsf"], a["ks"],
        a["vs"], a["sm"], a["pt"], a["sl"], a["window"], a["sinks"], a["out"], a["lse"], a["ws"],
        a["ws_bytes"], None)


@pytest.mark.parametrize("bad", [dict([(n, None)]) for n in ("q", "kp", "ksf", "vp", "vsf", "pt", "sl",
                                                              "out", "lse")]
                         + [dict([(n, at(264))]) for n in ("q", "kp", "ksf", "vp", "vsf", "out")]
                         + [dict(window=-1), dict(ks=0.0), dict(ks=-1.0), dict(ks=math.nan),
                            dict(sm=0.0), dict(sm=math.inf), dict(vs=math.inf), dict(vs=math.nan)])
@pytest.mark.parametrize("rows", [1, 40])
def test_dense_refused(lib, bad, rows):  # noqa: F811
    assert dense(lib, geom(rows_per_req=rows), **bad) == INVALID


def test_dense_workspace_and_geometry(lib):  # noqa: F811
    for g in (geom(), geom(rows_per_req=5), geom(rows_per_req=4096),
              geom(head_dim=256, rows_per_req=77)):
        need = lib.qsa_dense_attention_workspace_bytes(ctypes.byref(g))
        assert need > 0 and need % 256 == 0
        assert dense(lib, g, ws_bytes=need - 1) == WORKSPACE
        assert dense(lib, g, ws=None) == WORKSPACE
        assert dense(lib, g, ws=at(256 + 128)) == WORKSPACE
    wide = geom(num_q_heads=129, num_kv_heads=1)
    assert lib.qsa_dense_attention_workspace_bytes(ctypes.byref(wide)) == 0
    assert dense(lib, wide, ws_bytes=1 << 30) == UNSUPPORTED
    assert dense(lib, None) == INVALID
    assert lib.qsa_dense_attention_workspace_bytes(None) == 0
    # a workspace does not grow with the batch or the contexts, but for descriptors
    a = lib.qsa_dense_attention_workspace_bytes(ctypes.byref(geom(batch=1, max_blocks=1)))
    b = lib.qsa_dense_attention_workspace_bytes(ctypes.byref(geom(batch=500, max_blocks=1000)))
    assert b - a <= 152 * 32
