"""Rotation plans against 70 digits: every frequency right to the last bit of
its 64-bit fraction of a turn, so that angles stay right at any position."""
import ctypes

import pytest

import rope_exact
from nvfp4_block_sparse_gb300 import binding
from test_abi_cpu import lib  # noqa: F401  (a fixture)
from test_dense_abi_cpu import INVALID, config

SCALINGS = {"none": {}, "linear": dict(factor=4.0), "linear 1/3": dict(factor=1 / 3),
            "yarn": dict(factor=32.0, original=4096.0, low=1.0, high=32.0),
            "yarn 1.7": dict(factor=1.7, original=8192.0, low=1.0, high=32.0),
            "wavelength": dict(factor=8.0, original=8192.0, low=1.0, high=4.0),
            "wavelength 3.3": dict(factor=3.3, original=10000.0, low=0.7, high=5.1)}


@pytest.mark.parametrize("name", sorted(SCALINGS))
@pytest.mark.parametrize("rot,theta", [(16, 1e4), (80, 5e5), (128, 1e6), (256, 1e7), (256, 1.0001),
                                       (64, 1e300)])
def test_frequencies_to_the_last_bit(lib, name, rot, theta):  # noqa: F811
    scaling, kw = name.split()[0], SCALINGS[name]
    plan = binding.qsa_rope_t()
    kind = binding.ROPE_SCALINGS[scaling]
    cfg = config(rotary_dim=rot, theta=theta, scaling=kind, factor=kw.get("factor", 1.0),
                 original_context=kw.get("original", 1.0), low=kw.get("low", 1.0), high=kw.get("high", 2.0))
    assert lib.qsa_rope_init(ctypes.byref(cfg), ctypes.byref(plan)) == 0
    for got, x in zip(plan.turns, rope_exact.turns(rot, theta, scaling, **kw)):
        want = int(((x - int(x)) * 2**64).to_integral_value()) % 2**64
        off = (got - want) % 2**64
        assert min(off, 2**64 - off) <= 1, (got, want)


def test_plans_outside_the_range_refused(lib):  # noqa: F811
    plan = binding.qsa_rope_t()
    plan.rotary_dim, plan.turns[3] = 5, 7
    for bad in (dict(scaling=1, factor=1e-320), dict(scaling=3, factor=1e-300, low=1e300, high=1e301),
                dict(scaling=1, factor=2.0**-32), dict(attention_factor=1e-60),
                dict(attention_factor=1e60)):
        assert lib.qsa_rope_init(ctypes.byref(config(**bad)), ctypes.byref(plan)) == INVALID
        assert (plan.rotary_dim, plan.turns[3]) == (5, 7)      # left as it was
