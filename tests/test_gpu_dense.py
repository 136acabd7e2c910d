"""GPU tests of dense attention over the NVFP4 paged cache against a 64-bit
reference.

Tolerances.  The kernels multiply exact fp16 queries and keys (a query element
below 2^-24 of its row's largest vanishes), add in fp32, and round the weights
P to fp16 before the product with V.  With p the weights of a row:
  out  half a bf16 step of the result (2^-8 |out|, its relative bound), the
       weights' rounding 2^-11 sum p|V|, taken twice for the fp32 sums and the
       exponent's error, and half an fp16 subnormal step (2^-25) per token for
       weights far below the largest
  lse  D products in fp32, D 2^-24 sum |q K| sm <= 128..256 * 6e-8 * 10 < 2e-4
"""
import numpy as np
import pytest
import torch

import cache_reference as cr
import qsa_workloads as qw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    import nvfp4_block_sparse_gb300 as m
    m.load(build_if_missing=True)
    return m


def case(**kw):
    base = dict(name="dense", seed=51, batch=3, rows_per_req=1, num_q_heads=8, num_kv_heads=2,
                page_size=64, ctx_lo=300, ctx_hi=1300, k=6, window=2, max_blocks=21, pool="perm")
    base.update(kw)
    return qw.Case(**base)


def run(qsa, w, window=0, sinks=None, step=None):
    step = step or qsa.DenseStep(qw.geometry(w), window=window, device="cuda")
    step.out.fill_(float("nan"))
    step.lse.fill_(float("nan"))
    step.run(w, sinks=sinks)
    torch.cuda.synchronize()
    assert step.status() == 0
    return step


def check(w, step, window=0, sinks=None):
    h = cr.host(w)
    ref, lse, mag = cr.dense(h, window=window, sinks=None if sinks is None else sinks.cpu().numpy())
    out = step.out.float().cpu().numpy().astype(np.float64)
    got = step.lse.cpu().numpy().astype(np.float64)
    vmax = 6 * 448 * abs(w["v_scale"])
    tol = 2.0**-8 * np.abs(ref) + 2 * 2.0**-11 * mag + int(w["seqlens"].max()) * 2.0**-25 * vmax + 1e-7
    err = np.abs(out - ref)
    assert (err <= tol).all(), (err.max(), (err / tol).max())
    fin = np.isfinite(lse)
    np.testing.assert_array_equal(np.isneginf(got), ~fin)
    assert np.abs(got[fin] - lse[fin]).max(initial=0) <= 2e-4
    rows, heads = np.nonzero(np.isneginf(lse))
    assert not out[rows, heads].any()


CASES = {
    # rows of one token: heads per KV head 1, 4, 8, 16, 12 and odd ones
    "decode_g4": (case(), 0, False),
    "decode_g1": (case(num_q_heads=2), 0, False),
    "decode_g16": (case(num_q_heads=32, num_kv_heads=2), 0, True),
    "decode_g7": (case(num_q_heads=7, num_kv_heads=1), 0, True),
    "decode_one_token": (case(ctx_lo=1, ctx_hi=1, max_blocks=1, k=1, window=1), 0, False),
    "decode_page_borders": (case(batch=5, ctx_lo=63, ctx_hi=66, max_blocks=2, k=1, window=1), 0, False),
    "decode_p128": (case(page_size=128, ctx_lo=100, ctx_hi=2600), 0, False),
    "decode_long": (case(batch=1, ctx_lo=20011, ctx_hi=20011, max_blocks=400), 0, True),
    "decode_many": (case(batch=70, ctx_lo=1, ctx_hi=400, max_blocks=7), 0, False),
    "decode_window": (case(), 100, True),
    "decode_window_1": (case(), 1, False),
    "decode_window_wide": (case(), 5000, False),
    "decode_holes": (case(invalid_frac=0.4), 0, False),
    "decode_all_holes": (case(invalid_frac=1.0), 0, False),
    "decode_all_holes_sink": (case(invalid_frac=1.0), 0, True),
    # verify rows
    "verify_r2": (case(rows_per_req=2), 0, False),
    "verify_r8_window": (case(rows_per_req=8), 37, True),
    "verify_short": (case(rows_per_req=6, ctx_lo=1, ctx_hi=9, max_blocks=1, k=1, window=1), 0, False),
    "verify_wide": (case(rows_per_req=4, num_q_heads=64, num_kv_heads=4), 0, False),
    # head_dim 256
    "hd256_decode": (case(head_dim=256, page_size=32, max_blocks=41, num_q_heads=24), 0, True),
    "hd256_decode_g4": (case(head_dim=256), 0, False),
    "hd256_verify": (case(head_dim=256, page_size=32, max_blocks=41, num_q_heads=24,
                          rows_per_req=4), 200, True),
    "hd256_holes": (case(head_dim=256, page_size=32, max_blocks=41, invalid_frac=0.5), 0, False),
    # context row groups
    "rows_77": (case(rows_per_req=77, ctx_lo=70, ctx_hi=500), 0, True),
    "rows_130_window": (case(rows_per_req=130, ctx_lo=100, ctx_hi=700, num_q_heads=12), 65, False),
    "rows_holes": (case(rows_per_req=40, invalid_frac=0.5), 0, False),
    "rows_long": (case(batch=1, rows_per_req=33, ctx_lo=5001, ctx_hi=5001, max_blocks=80), 0, False),
    "rows_g128": (case(rows_per_req=5, num_q_heads=128, num_kv_heads=1), 0, True),
    "hd256_rows": (case(head_dim=256, page_size=32, max_blocks=41, rows_per_req=50,
                        num_q_heads=24), 0, True),
    "hd256_rows_p64": (case(head_dim=256, rows_per_req=200, ctx_lo=150, ctx_hi=900), 120, False),
}


def sink_of(w, on):
    if not on:
        return None
    s = torch.linspace(-2.0, 6.0, w["num_q_heads"], device="cuda")
    s[0] = float("-inf")          # a head without one
    return s


@pytest.mark.parametrize("name", sorted(CASES))
def test_dense_matches_reference(qsa, name):
    c, window, with_sinks = CASES[name]
    w = qw.make_workload(c, "cuda")
    sinks = sink_of(w, with_sinks)
    check(w, run(qsa, w, window, sinks), window, sinks)


@pytest.mark.parametrize("name", ["decode_g4", "verify_r8_window", "hd256_verify", "rows_77",
                                  "hd256_rows"])
def test_what_no_row_sees_may_be_anything(qsa, name):
    # Tokens behind the last and before every window: scales that are NaN, codes of
    # the largest value, page ids out of range.
    c, window, with_sinks = CASES[name]
    w = qw.make_workload(c, "cuda")
    sinks = sink_of(w, with_sinks)
    clean = run(qsa, w, window, sinks)
    P, R, MB = w["page_size"], w["rows_per_req"], w["max_blocks"]
    pt = w["page_table"].clone()
    for b, L in enumerate(w["seqlens"].tolist()):
        first = max(0, max(L - R + 1, 0) - window) if window else 0
        for beta in range(MB):
            page = int(pt[b, beta])
            for lo, hi in ((0, min(P, max(0, first - beta * P))), (max(0, min(P, L - beta * P)), P)):
                if page >= 0 and lo < hi:
                    for n in ("k", "v"):
                        w[n + "_sf"][page, :, lo:hi] = 0x7F
                        w[n + "_pool"][page, :, lo:hi] = 0x77
            if beta * P >= L or (beta + 1) * P <= first:
                w["page_table"][b, beta] = (-5, 2**31 - 1)[beta % 2]
    dirty = run(qsa, w, window, sinks)
    assert torch.equal(clean.out, dirty.out) and torch.equal(clean.lse, dirty.lse)


def test_lengths_of_zero_and_past_the_table(qsa):
    w = qw.make_workload(case(batch=4, rows_per_req=3), "cuda")
    w["seqlens"] = torch.tensor([0, 2, 21 * 64 + 500, 700], dtype=torch.int32, device="cuda")
    w["page_table"] = torch.randint(0, w["num_pages"], w["page_table"].shape, device="cuda",
                                    dtype=torch.int32)      # pages may be shared
    check(w, run(qsa, w), 0, None)


@pytest.mark.parametrize("scale", [1e-30, 30.0])
def test_flat_and_sharp_rows(qsa, scale):
    # all logits alike, and rows where one token takes everything (the base moves often)
    w = qw.make_workload(case(rows_per_req=2, ctx_lo=900, ctx_hi=900), "cuda")
    w["q"] = (w["q"].float() * scale).to(torch.bfloat16)
    h = cr.host(w)
    step = run(qsa, w)
    ref, lse, mag = cr.dense(h)
    out = step.out.float().cpu().numpy()
    # logits grow with the queries, and with them their fp32 rounding: 128 terms of
    # up to 30 * 4.5 * 4.5 / 11.3 each, times 2^-24
    dz = 128 * 2.0**-24 * max(scale, 1) * 2
    tol = 2.0**-8 * np.abs(ref) + (2.0**-10 + 2 * dz) * mag + 900 * 2.0**-25 * 6 * 448 * w["v_scale"]
    assert (np.abs(out - ref) <= tol).all()
    assert np.abs(step.lse.cpu().numpy() - lse).max() <= 2e-4 + dz


def test_offsets_past_32_bits(qsa):
    # a pool of 2^32 code bytes and more per plane: pages at its end
    NP, P, Hkv, D = 530000, 128, 1, 128
    w = qw.make_workload(case(batch=2, num_q_heads=4, num_kv_heads=1, page_size=P, ctx_lo=400,
                              ctx_hi=500, max_blocks=4, k=2), "cuda")
    big = {n: torch.empty((NP, Hkv, P, D // d), dtype=torch.uint8, device="cuda")
           for n, d in (("k_pool", 2), ("k_sf", 16), ("v_pool", 2), ("v_sf", 16))}
    clean = run(qsa, w)
    n = w["num_pages"]
    for name, t in big.items():
        t[NP - n:] = w[name]
    moved = dict(w, **big, num_pages=NP,
                 page_table=torch.where(w["page_table"] >= 0, w["page_table"] + (NP - n), -1).to(torch.int32))
    got = run(qsa, moved)
    assert torch.equal(clean.out, got.out) and torch.equal(clean.lse, got.lse)


@pytest.mark.parametrize("name", ["decode_long", "verify_r8_window", "rows_77", "hd256_rows"])
def test_same_bits_again_in_a_graph_and_on_a_stream(qsa, name):
    c, window, with_sinks = CASES[name]
    w = qw.make_workload(c, "cuda")
    sinks = sink_of(w, with_sinks)
    first = run(qsa, w, window, sinks)
    again = run(qsa, w, window, sinks, step=first) and (first.out.clone(), first.lse.clone())
    other = qsa.DenseStep(qw.geometry(w), window=window)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other.run(w, sinks=sinks, stream=s)
    s.synchronize()
    assert torch.equal(other.out, again[0]) and torch.equal(other.lse, again[1])
    # two captured graphs that share the workspace, replayed one after the other
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            other.run(w, sinks=sinks)
        graphs.append(gr)
    for gr in graphs * 2:
        other.out.zero_()
        gr.replay()
        assert torch.equal(other.out, again[0])
    # new inputs behind the same addresses
    w["seqlens"] -= (w["seqlens"] > 100).to(torch.int32) * 37
    graphs[0].replay()
    torch.cuda.synchronize()
    check(w, other, window, sinks)


def test_a_step_of_the_whole_run(qsa):
    # rotation rows -> norms, rotation and append -> dense attention and, on the same
    # cache, the sparse step with every block selected: the two agree
    w = qw.make_workload(case(rows_per_req=4, k=21, window=2), "cuda")
    T, Hq, Hkv, D = 12, 8, 2, 128
    gen = torch.Generator(device="cuda").manual_seed(3)
    wide = torch.randn(T, Hq + 2 * Hkv, D, generator=gen, device="cuda").to(torch.bfloat16)
    new = dict(q=wide[:, :Hq], k=wide[:, Hq:Hq + Hkv], v=wide[:, Hq + Hkv:],
               ik_new=torch.randint(-127, 128, (T, 64), generator=gen, device="cuda").to(torch.int8),
               q_weight=torch.ones(D, dtype=torch.bfloat16, device="cuda"),
               k_weight=torch.ones(D, dtype=torch.bfloat16, device="cuda"))
    rope = qsa.make_rope(rotary_dim=64, theta=1e6)
    nr = qsa.make_norm_rope(64)
    before = cr.host(w)
    step = qsa.DenseStep(qw.geometry(w))
    cs = torch.empty(T, 32, 2, device="cuda")
    qsa.qsa_rope_rows(step.cg, rope, w["seqlens"], cs)
    step.store(w, new, nr, cs)
    step.run(w, q=step.q)
    torch.cuda.synchronize()
    q, _, pools = cr.store_rope(before, cr.host(new), cs.cpu().numpy(), 64, False, 1e-6, False)
    np.testing.assert_array_equal(step.q.cpu().float().numpy(), q)
    w["q"] = step.q
    for n, ref in pools.items():
        np.testing.assert_array_equal(w[n].cpu().numpy(), ref)
    check(w, step)
    sparse = qsa.DecodeStep(qw.geometry(w), 21, 2)
    sparse.run(w)
    torch.cuda.synchronize()
    assert (sparse.out.float() - step.out.float()).abs().max() <= 2.0**-7 * step.out.float().abs().max()
    assert (sparse.lse - step.lse).abs().max() <= 2e-4


@pytest.mark.parametrize("R,G", [(1, 4), (3, 4), (4, 4), (9, 4), (30, 4), (70, 8), (200, 3)])
@pytest.mark.parametrize("D,P", [(128, 64), (128, 128), (256, 32), (256, 64)])
@pytest.mark.parametrize("B,window", [(3, 0), (3, 100), (200, 0), (200, 33)])
def test_values_that_a_row_does_not_see(qsa, B, window, D, P, R, G):
    """A NaN scale of V makes NaN of the rows that see it, in its 16 dims, and of nothing else: not of the rows ahead
    of it, and not of those that have left it behind.  (200 requests: whole units; 3: divided ones.)"""
    dev = "cuda"
    lo, hi = R + 300, R + (900 if B < 100 else 400)
    MB = -(-hi // P)
    NP = B * MB + 2
    gen, rng = torch.Generator(device=dev).manual_seed(R), np.random.default_rng(R)
    g = qsa.make_geom(batch=B, rows_per_req=R, num_q_heads=2 * G, num_kv_heads=2, head_dim=D, index_dim=64,
                      page_size=P, max_blocks=MB, num_pages=NP)
    table = rng.permutation(NP)[:B * MB].reshape(B, MB).astype(np.int32)
    lens = rng.integers(lo, hi + 1, B).astype(np.int32)
    pools = []
    for _ in "kv":
        pools += [torch.randint(0, 256, (NP, 2, P, D // 2), generator=gen, dtype=torch.uint8, device=dev),
                  torch.randint(0x28, 0x38, (NP, 2, P, D // 16), generator=gen, dtype=torch.uint8, device=dev)]
    q = torch.randn(B * R, 2 * G, D, generator=gen, device=dev).to(torch.bfloat16)
    ws = torch.empty(qsa.qsa_dense_attention_workspace_bytes(g), dtype=torch.uint8, device=dev)
    qsa.qsa_workspace_init(ws)

    def call():
        out, lse = torch.empty_like(q), torch.empty(B * R, 2 * G, device=dev)
        qsa.qsa_dense_attention(g, q, *pools, 1.0, 1.0, D**-0.5, torch.from_numpy(table).to(dev),
                                torch.from_numpy(lens).to(dev), out, lse, ws, window=window)
        assert qsa.qsa_workspace_status(ws) == 0
        return out, lse
    plain = call()
    nan = torch.zeros(B * R, 2 * G, D, dtype=torch.bool, device=dev)
    for b in sorted({0, 1, 2, B // 2, B - 1}):
        old = int(lens[b]) - R                             # row j sees tokens up to old + j
        for tok in [old + R - 1, old, 0, *rng.integers(max(0, old - 200), old + R, 9)]:
            h, group = int(rng.integers(2)), int(rng.integers(D // 16))
            pools[3][int(table[b, tok // P]), h, int(tok) % P, group] = 0x7F if rng.integers(2) else 0xFF
            first, end = max(0, int(tok) - old), R if not window else min(R, int(tok) + window - old)
            if end > first:
                nan[b * R + first:b * R + end, h * G:(h + 1) * G, 16 * group:16 * group + 16] = True
    out, lse = call()
    assert torch.equal(lse, plain[1])
    wrong = out.isnan() != nan
    assert not wrong.any(), (int(wrong.sum()), wrong.nonzero()[:3].tolist())
    assert torch.equal(out[~nan], plain[0][~nan])
