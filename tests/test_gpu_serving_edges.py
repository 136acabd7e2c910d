"""GPU tests of the prologue and dense attention where serving goes wrong: more
requests than a warp has lanes and more units than the GPU has SMs, padded
batches, shared pages, windows at page borders, streams, calls at once, and
quantisation far from the middle of its range.  References and tolerances as
in the files of the two operators."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import cache_reference as cr
import qsa_workloads as qw
from test_gpu_dense import case, check, run, sink_of
from test_gpu_prologue import POOLS, append, cache_case, draw

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def qsa():
    import nvfp4_block_sparse_gb300 as m
    m.load(build_if_missing=True)
    return m


# batch, rows, query heads, KV heads, head_dim, longest length
SHAPES = {
    "decode_wide_batch": (300, 1, 8, 2, 128, 200),     # 600 units, 300 groups
    "decode_g16_batch": (200, 1, 16, 1, 128, 500),
    "hd256_decode_batch": (90, 1, 24, 2, 256, 300),
    "verify_batch": (100, 4, 24, 2, 128, 260),         # tile kernel, 200 units
    "hd256_verify_batch": (80, 3, 16, 2, 256, 300),
    "context_batch": (40, 70, 8, 2, 128, 400),         # pairs, two tiles a CTA, 40 groups
    "hd256_context_batch": (40, 30, 12, 2, 256, 300),
    "one_request_of_many": (64, 2, 16, 1, 128, 60),
}


@pytest.mark.parametrize("window", [0, 130])
@pytest.mark.parametrize("name", sorted(SHAPES))
def test_batches_with_padding(qsa, name, window):
    # Requests of length zero, one, shorter than their rows, and one far longer than the rest;
    # unused rows of the page table hold -1 and their lengths are zero.
    B, R, Hq, Hkv, D, longest = SHAPES[name]
    P = 32 if D == 256 else 64
    w = qw.make_workload(case(batch=B, rows_per_req=R, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D,
                              page_size=P, ctx_lo=1, ctx_hi=longest, max_blocks=-(-3 * longest // P),
                              k=1, window=1), "cuda")
    L = w["seqlens"].clone()
    L[::7] = 0
    L[1::11] = 1
    L[B // 2] = 3 * longest
    w["page_table"] = torch.randint(0, w["num_pages"], w["page_table"].shape, dtype=torch.int32,
                                    device="cuda", generator=torch.Generator("cuda").manual_seed(B))
    w["page_table"][L == 0] = -1
    w["seqlens"] = L
    sinks = sink_of(w, window > 0)
    check(w, run(qsa, w, window, sinks), window, sinks)


@pytest.mark.parametrize("D,rows,Hq", [(128, 1, 8), (128, 9, 8), (128, 80, 8), (256, 1, 8), (256, 6, 8),
                                       (256, 70, 8)])
@pytest.mark.parametrize("window", [1, 63, 64, 65, 128, 1000])
def test_windows_at_page_borders(qsa, D, rows, Hq, window):
    w = qw.make_workload(case(batch=2, rows_per_req=rows, num_q_heads=Hq, head_dim=D, ctx_lo=rows,
                              ctx_hi=900), "cuda")
    w["seqlens"] = torch.tensor([640, 641], dtype=torch.int32, device="cuda")
    check(w, run(qsa, w, window), window)


@pytest.mark.parametrize("D,rows", [(128, 1), (128, 12), (128, 90), (256, 2), (256, 12), (256, 90)])
def test_one_page_everywhere(qsa, D, rows):
    # every block of every request is the same page, but for holes in the first and last
    w = qw.make_workload(case(batch=3, rows_per_req=rows, head_dim=D, ctx_lo=rows, ctx_hi=1200), "cuda")
    w["page_table"][:] = w["num_pages"] - 1
    w["page_table"][0, 0] = -1
    w["page_table"][1, int((w["seqlens"][1] - 1) // w["page_size"])] = w["num_pages"]
    check(w, run(qsa, w))


@pytest.mark.parametrize("rows", [1, 12, 90])
def test_tables_longer_than_a_warp(qsa, rows):
    # 90 blocks of which every third is missing, from a window that starts inside one
    w = qw.make_workload(case(batch=1, rows_per_req=rows, ctx_lo=5700, ctx_hi=5700, max_blocks=90),
                         "cuda")
    w["page_table"][0, ::3] = -1
    check(w, run(qsa, w))
    check(w, run(qsa, w, 4500), 4500)


@pytest.mark.parametrize("D,P", [(128, 64), (128, 128), (256, 32), (256, 64)])
@pytest.mark.parametrize("rows,window", [(1, 0), (3, 200), (9, 0), (9, 200), (40, 129), (70, 0), (150, 0),
                                         (150, 300)])
def test_page_sizes(qsa, D, P, rows, window):
    # a chunk of the kernels is a part of a page, one page or several; some are missing
    w = qw.make_workload(case(batch=3, rows_per_req=rows, head_dim=D, page_size=P, ctx_lo=rows,
                              ctx_hi=1300, max_blocks=-(-1300 // P), invalid_frac=0.3), "cuda")
    sinks = sink_of(w, window > 0)
    check(w, run(qsa, w, window, sinks), window, sinks)


@pytest.mark.parametrize("rows", [2, 12, 90])
def test_two_calls_at_once(qsa, rows):
    # two steps with workspaces of their own, in flight on two streams
    w = qw.make_workload(case(rows_per_req=rows, ctx_lo=900, ctx_hi=1300), "cuda")
    alone = run(qsa, w)
    steps = [qsa.DenseStep(qw.geometry(w), device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for step, s in zip(steps, streams):
            step.run(w, stream=s)
    torch.cuda.synchronize()
    for step in steps:
        assert step.status() == 0
        assert torch.equal(step.out, alone.out) and torch.equal(step.lse, alone.lse)


@pytest.mark.parametrize("rows", [1, 12, 90])
def test_calls_behind_one_another_with_other_lengths(qsa, rows):
    # a workspace serves calls of one geometry whatever the lengths: records and tickets of one
    # call mean nothing to the next
    w = qw.make_workload(case(rows_per_req=rows, ctx_lo=rows, ctx_hi=1300), "cuda")
    step = qsa.DenseStep(qw.geometry(w), device="cuda")
    lengths = [w["seqlens"].clone(), torch.tensor([0, 0, 0], dtype=torch.int32, device="cuda"),
               torch.tensor([1, 1344, 0], dtype=torch.int32, device="cuda"), w["seqlens"].clone()]
    first = None
    for L in lengths:
        check(dict(w, seqlens=L), run(qsa, dict(w, seqlens=L), step=step))
        first = step.out.clone() if first is None else first
    assert torch.equal(first, step.out)


def test_geometries_share_a_workspace(qsa):
    # context rows, verify rows and decode rows by turns on one workspace: what one leaves
    # there (descriptors that name its last CTA, records) means nothing to the next
    works = [qw.make_workload(case(batch=b, rows_per_req=r, num_q_heads=4 * hkv, num_kv_heads=hkv,
                                   head_dim=D, ctx_lo=L, ctx_hi=L, max_blocks=-(-L // 64)), "cuda")
             for b, r, hkv, D, L in ((3, 80, 1, 128, 18176), (1, 1, 2, 128, 45728), (40, 5, 2, 256, 900),
                                     (2, 2, 2, 128, 9000), (60, 30, 2, 128, 700), (1, 1, 2, 256, 45000))]
    steps = [qsa.DenseStep(qw.geometry(w), device="cuda") for w in works]
    shared = max((s.workspace for s in steps), key=lambda t: t.numel())
    for s in steps:
        s.workspace = shared
    for _ in range(2):
        for w, s in zip(works, steps):
            check(w, run(qsa, w, step=s))


@pytest.mark.parametrize("k_scale,v_scale,spread", [
    (1e-30, 1e30, 1.0), (1e-38, 3e38, 1.0), (2.0**-126, 2.0**-100, 1e-30), (1.0, 1.0, 0.0),
    (0.01, 448.0 * 6.0, 1e4), (1e20, 1e-20, 1e15), (3e-3, 1 / 3, 100.0),
])
@pytest.mark.parametrize("rows", [1, 40])
def test_append_far_from_the_middle(qsa, k_scale, v_scale, spread, rows):
    # scales that saturate every code, leave only zeros, or have no reciprocal in fp32
    w = qw.make_workload(cache_case(rows_per_req=rows, ctx_lo=rows, ctx_hi=400, max_blocks=7, k=2),
                         "cuda")
    w["k_scale"], w["v_scale"] = k_scale, v_scale
    T = w["batch"] * rows
    x = draw(T, 8, 2, 128, 64, seed=7, spread=spread)
    nr = qsa.make_norm_rope(64)
    x["k_weight"] = None if spread > 1e3 else x["k_weight"]
    pools = {n: w[n].clone() for n in POOLS}
    q_out = torch.empty(T, 8, 128, dtype=torch.bfloat16, device="cuda")
    append(qsa, w, x, nr, pools, q_out)
    two = {n: w[n].clone() for n in POOLS}
    k2 = torch.empty(T, 2, 128, dtype=torch.bfloat16, device="cuda")
    qsa.qsa_qk_norm_rope(qw.geometry(w), nr, None, x["k"], None, x["k_weight"], x["cs"], None, k2)
    qsa.qsa_store_kv_tokens(qw.geometry(w), k2, x["v"].contiguous(), x["ik_new"], k_scale, v_scale,
                            w["page_table"], w["seqlens"], *(two[n] for n in POOLS))
    for n in POOLS:
        assert torch.equal(two[n], pools[n]), n


@pytest.mark.parametrize("rows", [1, 40])
def test_append_of_infinities_and_nan(qsa, rows):
    # whatever the values, the fused call leaves the bytes of the two
    w = qw.make_workload(cache_case(rows_per_req=rows, ctx_lo=rows, ctx_hi=400, max_blocks=7, k=2),
                         "cuda")
    T = w["batch"] * rows
    x = draw(T, 8, 2, 128, 64, seed=8)
    for i, value in enumerate((float("inf"), float("-inf"), float("nan"), 3e38, 1e-40)):
        x["k"][:, :, i::37] = value
        x["v"][:, i % 2, i::41] = value
    x["v"][0] = float("nan")
    nr = qsa.make_norm_rope(64)
    for weight in (None, x["k_weight"]):
        new = dict(x, k_weight=weight)
        pools, two = ({n: w[n].clone() for n in POOLS} for _ in range(2))
        append(qsa, w, dict(new, q=None), nr, pools, None)
        k2 = torch.empty(T, 2, 128, dtype=torch.bfloat16, device="cuda")
        qsa.qsa_qk_norm_rope(qw.geometry(w), nr, None, x["k"], None, weight, x["cs"], None, k2)
        qsa.qsa_store_kv_tokens(qw.geometry(w), k2, x["v"].contiguous(), x["ik_new"], w["k_scale"],
                                w["v_scale"], w["page_table"], w["seqlens"], *(two[n] for n in POOLS))
        for n in POOLS:
            assert torch.equal(two[n], pools[n]), n


def test_append_of_a_padded_batch(qsa):
    # rows of requests without a length or a page: queries are written, the pools stay
    w = qw.make_workload(cache_case(batch=6, rows_per_req=4), "cuda")
    w["seqlens"][:3] = torch.tensor([0, 2, 21 * 64 + 2], dtype=torch.int32, device="cuda")
    w["page_table"][3] = -1
    w["page_table"][4] = 2**31 - 1
    x = draw(24, 8, 2, 128, 64, seed=2)
    nr = qsa.make_norm_rope(64)
    pools = {n: w[n].clone() for n in POOLS}
    q_out = torch.empty(24, 8, 128, dtype=torch.bfloat16, device="cuda")
    append(qsa, w, x, nr, pools, q_out)
    h, hx = cr.host(w), cr.host(x)
    q, _, ref = cr.store_rope(h, hx, hx["cs"], 64, False, 1e-6, False)
    np.testing.assert_array_equal(q_out.cpu().float().numpy(), q)
    for n in POOLS:
        np.testing.assert_array_equal(pools[n].cpu().numpy(), ref[n], err_msg=n)


def test_dense_step_refusals(qsa):
    w = qw.make_workload(case(rows_per_req=2), "cuda")
    step = qsa.DenseStep(qw.geometry(w), device="cuda")
    for name, value in (("q", w["q"].float()), ("k_sf", w["k_sf"].float()),
                        ("page_table", w["page_table"].long()), ("seqlens", w["seqlens"].long())):
        with pytest.raises(TypeError):
            step.run(dict(w, **{name: value}))
    for name, value in (("q", w["q"].cpu()), ("q", w["q"][:3]), ("page_table", w["page_table"][:, :5]),
                        ("seqlens", w["seqlens"][:2]), ("v_pool", w["v_pool"].transpose(1, 2))):
        with pytest.raises(ValueError):
            step.run(dict(w, **{name: value}))
    with pytest.raises(ValueError):
        step.run(w, sinks=torch.zeros(3, device="cuda"))
    with pytest.raises(TypeError):
        step.run(w, sinks=torch.zeros(8, device="cuda", dtype=torch.float64))
    step.run(w)
    assert step.status() == 0


def test_operators_hold_every_bounds_check():
    if os.environ.get("QSA_BOUNDS_CHECKED") == "1":
        pytest.skip("this is the checked run")
    r = subprocess.run(
        [sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p", "no:cacheprovider",
         "tests/test_gpu_dense.py", "tests/test_gpu_prologue.py", "tests/test_gpu_serving_edges.py"],
        cwd=ROOT, env=dict(os.environ, QSA_BOUNDS_CHECKED="1"), capture_output=True, text=True,
        timeout=1800)
    tail = (r.stdout + r.stderr)[-3000:]
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and " failed" not in r.stdout, tail
