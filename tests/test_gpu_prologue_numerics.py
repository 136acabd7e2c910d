"""GPU tests of the prologue's numbers at their extremes: rotation rows at far
positions against 70 digits and the bound that the header states."""
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
