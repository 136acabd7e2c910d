"""GPU tests of the prologue's numbers at their extremes: rotation rows at far
positions against 70 digits and the bound that the header states, and norms of
query and key heads of zeros, vanishing squares and magnitudes near fp32's end,
by the kernel for few rows and by the one for many."""
import numpy as np
import pytest
import torch

import cache_reference as cr
import rope_exact
from test_gpu_prologue import SCALINGS, draw, geom, plan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    import nvfp4_block_sparse_gb300 as m
    m.load(build_if_missing=True)
    return m


@pytest.mark.parametrize("sc", SCALINGS, ids=lambda s: s["scaling"])
@pytest.mark.parametrize("rot,theta", [(16, 1e4), (80, 5e5), (128, 1e6), (256, 1e7)])
def test_rope_rows_within_the_stated_bound(qsa, sc, rot, theta):
    gen = torch.Generator().manual_seed(rot)
    pos = torch.cat([torch.tensor([0, 1, -1, 2**31 - 1, -2**31, 2**30 + 1, 1380000000]),
                     torch.randint(-2**31, 2**31, (57,), generator=gen)]).to(torch.int32)
    g = geom(batch=16, rows_per_req=4)
    rope = plan(qsa, rot, theta, sc)
    cs = torch.full((64, rot // 2, 2), float("nan"), device="cuda")
    qsa.qsa_rope_rows(g, rope, None, cs, positions=pos.cuda())
    amp = cr.freqs(rot, theta, **sc)[1]
    kw = {k: v for k, v in sc.items() if k != "scaling"}
    ref = np.array(rope_exact.rows(pos.tolist(), rope_exact.turns(rot, theta, sc["scaling"], **kw))) * amp
    err = np.abs(cs.cpu().numpy().astype(np.float64) - ref)
    assert (err <= 2e-7 * amp).all(), err.max() / amp


@pytest.mark.parametrize("rows", [1, 700])        # by single steps, and by four
@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("D,inter", [(128, False), (256, True)])
@pytest.mark.parametrize("spread", [0.0, 1e-20, 1e-30, 1e15, 1e18])
def test_norms_at_the_extremes(qsa, rows, weights, D, inter, spread):
    # (at 1e18 some rows' sums of squares are infinite: their heads become zeros)
    g = geom(batch=2, rows_per_req=rows, head_dim=D)
    T = 2 * rows
    x = draw(T, 8, 2, D, 96, seed=11, spread=spread)
    x["q"][::3, 1] = 0.0
    x["k"][::3, 1] = 0.0
    nr = qsa.make_norm_rope(96, interleaved=inter, eps=1e-6)
    q = torch.full((T, 8, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    k = torch.full((T, 2, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    qw_, kw_ = (x["q_weight"], x["k_weight"]) if weights else (None, None)
    qsa.qsa_qk_norm_rope(g, nr, x["q"], x["k"], qw_, kw_, x["cs"], q, k)
    h = cr.host(x)
    with np.errstate(over="ignore", invalid="ignore"):
        for got, src in ((q, "q"), (k, "k")):
            ref = cr.norm_rope(h[src], h[src + "_weight"] if weights else None, h["cs"], 96, inter, 1e-6,
                               False)
            np.testing.assert_array_equal(got.cpu().float().numpy(), ref, err_msg=src)
