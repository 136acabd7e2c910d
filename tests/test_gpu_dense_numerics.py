"""GPU tests of dense attention's numbers where they can go wrong: contexts so
long that a lost page hardly shows, rows whose weights span many powers of two,
scales whose product leaves fp32, and queries, keys and values that are NaN or
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
    # lengths from a row to 9000 tokens in one call: some units are divided, some are not
    for name in ("decode_8", "hd256_decode_16", "tile"):
        w = workload(name, 9000, batch=5)
        R = w["rows_per_req"]
        w["seqlens"] = torch.tensor([9000, R, 700, 4097, 8191], dtype=torch.int32, device="cuda")
        check(w, run(qsa, w))


def dominated(name, gap, period, L=8256):
    """Every period-th token, without values, is `gap` nats above the others, whose logits are
    zero and whose values are all positive: the output is what the others add up to."""
    w = workload(name, L)
    w["k_pool"].zero_()
    w["k_sf"].fill_(0x38)                 # 1
    w["k_scale"], w["sm_scale"] = 1.0, 1 / 16
    w["v_pool"].bitwise_and_(0x77)        # no sign
    P = w["page_size"]
    q = torch.zeros_like(w["q"])
    q[..., :16] = 1.0
    w["q"] = q
    sf = torch.tensor(float(gap)).to(torch.float8_e4m3fn)
    assert float(sf) == gap
    for t in range(0, L, period):
        page, slot = int(w["page_table"][0, t // P]), t % P
        w["k_pool"][page, :, slot, :8] = 0x22            # sixteen ones
        w["k_sf"][page, :, slot, 0] = int(sf.view(torch.uint8))
        w["v_sf"][page, :, slot] = 0
    return w


@pytest.mark.parametrize("period", [32, 64, 8256])
@pytest.mark.parametrize("gap", [8, 12, 14, 16])
@pytest.mark.parametrize("name", sorted(KERNELS))
def test_weights_far_below_the_largest(qsa, name, gap, period):
    w = dominated(name, gap, period)
    check(w, run(qsa, w), alike=True)


@pytest.mark.parametrize("name", sorted(KERNELS))
def test_weights_far_above_the_first(qsa, name):
    # the other way round: the largest logits come last, after many small ones, and each step is
    # one that a base with headroom does not follow at once
    L = 4096
    w = dominated(name, 1, 1, L)
    P = w["page_size"]
    w["v_sf"].copy_(workload(name, L)["v_sf"])
    steps = [1, 2, 4, 8, 10, 12, 14, 16, 18, 20, 22, 24, 26, 28, 30, 32]
    for t in range(L):
        sf = torch.tensor(float(steps[t * len(steps) // L])).to(torch.float8_e4m3fn)
        w["k_sf"][int(w["page_table"][0, t // P]), :, t % P, 0] = int(sf.view(torch.uint8))
    check(w, run(qsa, w), alike=True)


# (factor on k_scale, on sm_scale, on the queries): powers of two, so that nothing is rounded
@pytest.mark.parametrize("factors", [(2.0**-100, 2.0**-20, 2.0**120), (2.0**-120, 1.0, 2.0**120),
                                     (2.0**100, 2.0**10, 2.0**-110), (1.0, 2.0**-120, 2.0**120)])
@pytest.mark.parametrize("name", ["decode_8", "hd256_decode_16", "tile", "tile_pair", "hd256_tile_pair"])
def test_scales_far_apart_cancel(qsa, name, factors):
    w = workload(name, 1111, invalid_frac=0.2)
    q = w["q"].float()
    w["q"] = torch.where(q.abs() < 2.0**-10, 0.0, q).to(torch.bfloat16)   # (stays normal when scaled)
    a, b, c = factors
    far = dict(w, k_scale=w["k_scale"] * a, sm_scale=w["sm_scale"] * b, q=(w["q"].double() * c).to(torch.bfloat16))
    # The scales are fp32 arguments: k_scale 2^-120 lies below 2^-126, where fp32's steps are 2^-149,
    # so the call sees its multiple of 2^-149, and that one times 2^120 is what it has to agree with.
    w.update(k_scale=float(np.float32(far["k_scale"])) / a, sm_scale=float(np.float32(far["sm_scale"])) / b)
    plain = run(qsa, w, 700)
    assert torch.isfinite(far["q"]).all()
    got = run(qsa, far, 700)
    assert torch.equal(got.out, plain.out) and torch.equal(got.lse, plain.lse)


@pytest.mark.parametrize("factors", [(1e-30, 1e-20, 1.0), (1e-38, 1e-38, 1.0), (1e-20, 1e-3, 1e-37)])
@pytest.mark.parametrize("name", ["decode_8", "hd256_decode_16", "tile", "tile_pair", "hd256_tile_pair"])
def test_logits_that_vanish(qsa, name, factors):
    # every visible token counts alike; masked ones (ends, holes, the window) do not count
    w = workload(name, 1111, invalid_frac=0.2)
    a, b, c = factors
    w.update(k_scale=a, sm_scale=b, q=(w["q"].double() * c).to(torch.bfloat16))
    for window in (0, 700):
        check(w, run(qsa, w, window), window, alike=True)


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


@pytest.mark.parametrize("name", sorted(KERNELS))
def test_keys_that_are_not_finite(qsa, name):
    # a NaN scale of a block of keys: no finite result for rows that see it, nothing for the others
    w = workload(name, 1500, batch=2)
    clean = run(qsa, w, 1000)
    w["k_sf"][int(w["page_table"][1, 700 // w["page_size"]]), :, 700 % w["page_size"], 3] = 0x7F
    got = run(qsa, w, 1000)
    half = got.lse.shape[0] // 2
    assert torch.equal(got.lse[:half], clean.lse[:half]) and torch.equal(got.out[:half], clean.out[:half])
    assert torch.isnan(got.lse[half:]).all() and torch.isnan(got.out[half:]).all()
    late = run(qsa, w, 100)                  # a window behind it
    assert torch.isfinite(late.lse).all() and torch.isfinite(late.out).all()


@pytest.mark.parametrize("size", [2.0**17, 2.0**19, 2.0**21, 2.0**23])
@pytest.mark.parametrize("name", sorted(KERNELS))
def test_logits_large_in_magnitude(qsa, name, size):
    # all logits near `size`, whose fp32 steps the exponents' arguments inherit: weights near fp16's
    # end must not pass it.  Every token's logit is the row's offset plus 0 to 14.
    L = 8000
    w = workload(name, L)
    gen = torch.Generator(device="cuda").manual_seed(9)
    w["k_pool"].zero_()
    w["k_pool"][..., :16] = 0x22                                    # thirty-two ones
    w["k_sf"].fill_(0x38)                                           # 1
    level = torch.rand(w["k_sf"].shape[:3], generator=gen, device="cuda") * torch.rand(
        (w["num_pages"], 1, 1), generator=gen, device="cuda") * 448
    w["k_sf"][..., 1] = level.to(torch.float8_e4m3fn).view(torch.uint8)
    w["k_scale"], w["sm_scale"] = 1.0, 1 / 16
    q = torch.zeros_like(w["q"], dtype=torch.float32)
    rows = q.view(-1, w["head_dim"])
    rows[:, :16] = size * (1 + torch.arange(rows.shape[0], device="cuda")[:, None] / 128)
    rows[:, 16:32] = 2.0**-5
    w["q"] = q.to(torch.bfloat16)
    step = run(qsa, w)
    out, lse, _, _ = dense_bounds.dense(cr.host(w))
    # the products' sums in steps of 2^-23 of up to 4 size, D / 16 of them, two roundings more
    dz = (w["head_dim"] / 16 + 2) * 2.0**-23 * 4 * size
    got = step.lse.cpu().numpy()
    assert np.isfinite(got).all() and np.abs(got - lse).max() <= dz + 2.0**-18 * size
    values = cr.values(w["v_pool"].cpu().numpy(), w["v_sf"].cpu().numpy()) * w["v_scale"]
    got = step.out.float().cpu().numpy()
    assert np.isfinite(got).all() and np.abs(got).max() <= 1.01 * np.abs(values).max()
