"""The bounds by which dense attention's outputs are compared see what can go
wrong there: mistakes planted in the reference's inputs exceed them, also in
contexts so long that one page is a thousandth of a row's weight."""
import numpy as np
import pytest

import cache_reference as cr
import dense_bounds
import qsa_workloads as qw


def workload(L, D, P, rows=1):
    c = qw.Case(name="bounds", seed=51, batch=1, rows_per_req=rows, num_q_heads=4, num_kv_heads=1,
                head_dim=D, page_size=P, ctx_lo=L, ctx_hi=L, k=1, window=1, max_blocks=-(-L // P))
    return cr.host(qw.make_workload(c))


def mistakes(w):
    P, L = w["page_size"], int(w["seqlens"][0])
    blocks = w["page_table"].shape[1]

    def page(i):
        return int(w["page_table"][0, i])

    def without(name, i, lo=0, hi=None):
        x = w[name].copy()
        x[page(i), :, lo:hi] = 0
        return {name: x}

    yield "values of a page", without("v_sf", blocks // 2)
    yield "values of 32 tokens", without("v_sf", blocks // 3, 0, 32)
    yield "keys of a page", without("k_sf", 5)
    pt = w["page_table"].copy()
    pt[0, 3] = -1
    yield "a missing page", {"page_table": pt}
    pt = w["page_table"].copy()
    pt[0, 3] = pt[0, 9]
    yield "another page", {"page_table": pt}
    pt = w["page_table"].copy()
    pt[0, blocks // 2:blocks // 2 + -(-L // (152 * P))] = -1
    yield "the part of one of 152", {"page_table": pt}


@pytest.mark.parametrize("L,D,P", [(20011, 128, 64), (45728, 128, 64), (45000, 256, 32)])
def test_planted_mistakes_exceed_the_bounds(L, D, P):
    w = workload(L, D, P)
    ref = dense_bounds.dense(w)
    bf16 = cr.bf16(ref[0].astype(np.float32))
    dense_bounds.compare(bf16, ref[1].astype(np.float32), ref)      # the definition itself is within
    for name, change in mistakes(w):
        out = dense_bounds.dense(dict(w, **change))[0]
        assert (np.abs(out - ref[0]) > ref[2]).any(), name


def test_lost_rows_and_windows_exceed_the_bounds():
    w = workload(9000, 128, 64, rows=3)
    ref = dense_bounds.dense(w, window=4000)
    for other in (dense_bounds.dense(w, window=4064), dense_bounds.dense(w, window=4000,
                                                                          sinks=np.full(4, 5.0)),
                  dense_bounds.dense(w, window=4000, q=np.roll(w["q"], 1, 0))):
        assert (np.abs(other[0] - ref[0]) > ref[2]).any()
        assert (np.abs(other[1] - ref[1]) > ref[3]).any()


def test_agrees_with_the_plain_reference():
    w = workload(777, 256, 32, rows=5)
    sinks = np.array([0.5, -np.inf, 2.0, -1.0])
    for window in (0, 100):
        out, lse, _ = cr.dense(w, window, sinks)
        mine = dense_bounds.dense(w, window, sinks)
        np.testing.assert_allclose(mine[0], out, rtol=1e-12, atol=1e-14)
        np.testing.assert_allclose(mine[1], lse, rtol=1e-12)
