"""GPU tests of dense attention's numbers where they can go wrong: contexts so
long that a lost page hardly shows, and queries and values that are NaN or
infinite.  The bounds are derived in dense_bounds.py."""
import numpy as np
import pytest
import torch

import cache_reference as cr
import dense_bounds
import qsa_workloads as qw

pytestmark = pytest.mark.gpu

# rows, query heads, KV heads, head_dim, page size: every kernel of the two files
KERNELS = {
    "decode_8": (1, 8, 2, 128, 64), "decode_16": (2, 16, 2, 128, 64),
    "hd256_decode_8": (1, 8, 2, 256, 32), "hd256_decode_16": (1, 24, 2, 256, 32),
    "tile": (6, 8, 2, 128, 64), "tile_pair": (66, 4, 1, 128, 128),
    "hd256_tile": (6, 24, 2, 256, 32), "hd256_tile_pair": (33, 4, 1, 256, 64),
}


@pytest.fixture(scope="module")
def qsa():
    import nvfp4_block_sparse_gb300 as m
    m.load(build_if_missing=True)
    return m


def workload(name, L, batch=1, seed=71, **kw):
    R, Hq, Hkv, D, P = KERNELS[name]
    return qw.make_workload(qw.Case(name=name, seed=seed, batch=batch, rows_per_req=R, num_q_heads=Hq,
                                    num_kv_heads=Hkv, head_dim=D, page_size=P, ctx_lo=L, ctx_hi=L, k=1,
                                    window=1, max_blocks=-(-L // P), **kw), "cuda")


def run(qsa, w, window=0, sinks=None):
    step = qsa.DenseStep(qw.geometry(w), window=window, device="cuda")
    step.out.fill_(7.0)
    step.lse.fill_(7.0)
    step.run(w, sinks=sinks)
    torch.cuda.synchronize()
    assert step.status() == 0
    return step


def check(w, step, window=0, sinks=None, alike=False):
    ref = dense_bounds.dense(cr.host(w), window, None if sinks is None else sinks.cpu().numpy(),
                             alike=alike)
    dense_bounds.compare(step.out.float().cpu().numpy(), step.lse.cpu().numpy(), ref)


@pytest.mark.parametrize("name,L", [
    ("decode_8", 20011), ("decode_8", 45728), ("decode_16", 30001), ("hd256_decode_8", 45000),
    ("hd256_decode_16", 20000), ("tile", 45728), ("tile_pair", 18176), ("hd256_tile", 16385),
    ("hd256_tile_pair", 12000)])
def test_long_contexts(qsa, name, L):
    w = workload(name, L)
    check(w, run(qsa, w))
    sinks = torch.linspace(-1.0, 9.0, w["num_q_heads"], device="cuda")
    check(w, run(qsa, w, L // 2 + 5, sinks), L // 2 + 5, sinks)


def test_divided_and_whole_units_together(qsa):
    # lengths from one token to 45728 in one call: some units are divided, some are not
    for name in ("decode_8", "hd256_decode_16", "tile"):
        w = workload(name, 9000, batch=5)
        R = w["rows_per_req"]
        w["seqlens"] = torch.tensor([9000, R, 700, 4097, 8191], dtype=torch.int32, device="cuda")
        check(w, run(qsa, w))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("name", sorted(KERNELS))
def test_rows_that_are_not_finite(qsa, name, value):
    # a row whose queries are not finite has no finite lse and no finite output, and certainly
    # not the lse of a row that sees nothing; the other rows are what they are without it
    w = workload(name, 1500, batch=2)
    clean = run(qsa, w)
    Hq = w["num_q_heads"]
    rows = w["q"].view(-1, w["head_dim"])
    bad = torch.arange(0, rows.shape[0], 5, device="cuda")
    rows[bad, (bad * 7) % w["head_dim"]] = value
    got = run(qsa, w)
    lse, out = got.lse.view(-1), got.out.view(-1, w["head_dim"]).float()
    assert lse.numel() == w["batch"] * w["rows_per_req"] * Hq
    assert not torch.isfinite(lse[bad]).any() and not torch.isneginf(lse[bad]).any()
    assert not torch.isfinite(out[bad]).any()
    good = torch.ones(rows.shape[0], dtype=torch.bool, device="cuda")
    good[bad] = False
    assert torch.equal(lse[good], clean.lse.view(-1)[good])
    assert torch.equal(got.out.view(-1, w["head_dim"])[good], clean.out.view(-1, w["head_dim"])[good])


@pytest.mark.parametrize("name", sorted(KERNELS))
def test_values_that_are_not_finite(qsa, name):
    # a NaN scale of one visible block of values: NaN in its sixteen dims of the rows that see it
    w = workload(name, 1500)
    clean = run(qsa, w)
    P = w["page_size"]
    w["v_sf"][int(w["page_table"][0, 700 // P]), :, 700 % P, 3] = 0x7F
    got = run(qsa, w)
    assert torch.equal(got.lse, clean.lse)
    assert torch.isnan(got.out[..., 48:64]).all()
    keep = torch.ones(w["head_dim"], dtype=torch.bool, device="cuda")
    keep[48:64] = False
    assert torch.equal(got.out[..., keep], clean.out[..., keep])
