"""GPU tests of the step's prologue: rotation rows, head norms with the
rotation, the NVFP4 append with both, and cache rows read back.

The norms, the rotation and the quantiser are sequences of IEEE fp32 operations
by definition, so their results are compared bit for bit; cos and sin with the
bound that the header states (2e-7 times the amplitude)."""
import numpy as np
import pytest
import torch

import cache_reference as cr
import qsa_workloads as qw

pytestmark = pytest.mark.gpu

POOLS = ("k_pool", "k_sf", "v_pool", "v_sf", "ik_pool")


@pytest.fixture(scope="module")
def qsa():
    import nvfp4_block_sparse_gb300 as m
    m.load(build_if_missing=True)
    return m


def geom(**kw):
    base = dict(batch=2, rows_per_req=3, num_q_heads=8, num_kv_heads=2, head_dim=128, index_dim=64,
                page_size=64, max_blocks=8, num_pages=20)
    base.update(kw)
    return base


# ---------------------------------------------------------------------------
# rotation rows
# ---------------------------------------------------------------------------

SCALINGS = [dict(scaling="none"), dict(scaling="linear", factor=4.0),
            dict(scaling="yarn", factor=32.0, original=4096.0, low=1.0, high=32.0),
            dict(scaling="wavelength", factor=8.0, original=8192.0, low=1.0, high=4.0)]


def plan(qsa, rot, theta, sc):
    kw = dict(scaling=sc["scaling"], factor=sc.get("factor", 1.0),
              original_context=sc.get("original", 0.0))
    if sc["scaling"] == "yarn":
        kw.update(beta_slow=sc["low"], beta_fast=sc["high"])
    elif sc["scaling"] == "wavelength":
        kw.update(low_freq=sc["low"], high_freq=sc["high"])
    return qsa.make_rope(rotary_dim=rot, theta=theta, **kw)


@pytest.mark.parametrize("sc", SCALINGS, ids=lambda s: s["scaling"])
@pytest.mark.parametrize("rot,theta", [(16, 1e4), (80, 5e5), (128, 1e6), (256, 1e7)])
def test_rope_rows(qsa, sc, rot, theta):
    g = geom(batch=5, rows_per_req=7)
    lens = torch.tensor([7, 100, 4097, 131072, 2**31 - 1], dtype=torch.int32, device="cuda")
    rope = plan(qsa, rot, theta, sc)
    cs = torch.full((35, rot // 2, 2), float("nan"), device="cuda")
    qsa.qsa_rope_rows(g, rope, lens, cs)
    f, amp = cr.freqs(rot, theta, **sc)
    ref = cr.rope_rows(cr.positions(lens.cpu().numpy(), 7), f, amp)
    # The plan's frequencies and the reference's are within 2^-52 of each other
    # relatively (two roundings each), so at position 2^31 their angles are within
    # 2^31 * 2^-52 * f rad.
    pos = cr.positions(lens.cpu().numpy(), 7).astype(np.float64)
    tol = 2e-7 * amp + np.abs(pos)[:, None, None] * f[None, :, None] * 2.0**-50 * amp
    err = np.abs(cs.cpu().numpy().astype(np.float64) - ref)
    assert (err <= tol).all(), err.max()


def test_rope_rows_of_given_positions(qsa):
    g = geom(batch=3, rows_per_req=2)
    pos = torch.tensor([0, 5, 5, 123456, -3, 77], dtype=torch.int32, device="cuda")
    rope = qsa.make_rope(rotary_dim=64, theta=1e4, attention_factor=1.5)
    cs = torch.empty(6, 32, 2, device="cuda")
    qsa.qsa_rope_rows(g, rope, None, cs, positions=pos)
    f, _ = cr.freqs(64, 1e4)
    err = np.abs(cs.cpu().numpy() - cr.rope_rows(pos.cpu().numpy(), f, 1.5))
    assert err.max() <= 2e-7 * 1.5 + 1e-9
    assert torch.equal(cs[1], cs[2])


def test_rope_rows_of_many_rows(qsa):
    g = geom(batch=9, rows_per_req=4096)     # more rows than one wave of threads
    lens = torch.arange(9, dtype=torch.int32, device="cuda") * 10000 + 4096
    rope = qsa.make_rope(rotary_dim=32, theta=1e4)
    cs = torch.empty(9 * 4096, 16, 2, device="cuda")
    qsa.qsa_rope_rows(g, rope, lens, cs)
    f, amp = cr.freqs(32, 1e4)
    ref = cr.rope_rows(cr.positions(lens.cpu().numpy(), 4096), f, amp)
    assert np.abs(cs.cpu().numpy() - ref).max() <= 2e-7 + 1e-9


# ---------------------------------------------------------------------------
# norms and rotation
# ---------------------------------------------------------------------------

def draw(T, Hq, Hkv, D, rot, seed, spread=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    wide = (r(T, Hq + 2 * Hkv, D) * spread).to(torch.bfloat16)
    a = r(T, max(rot // 2, 1)) * 3
    return dict(q=wide[:, :Hq], k=wide[:, Hq:Hq + Hkv], v=wide[:, Hq + Hkv:],
                q_weight=(1 + 0.3 * r(D)).to(torch.bfloat16),
                k_weight=(0.3 * r(D)).to(torch.bfloat16),
                cs=torch.stack([a.cos(), a.sin()], -1).contiguous(),
                ik_new=torch.randint(-127, 128, (T, 64), generator=gen, device="cuda").to(torch.int8))


CASES = [  # B, R, Hq, Hkv, D, rot, interleaved, weight_plus_one
    (1, 1, 8, 1, 128, 128, False, False), (3, 5, 6, 2, 128, 48, True, True),
    (2, 7, 9, 3, 128, 16, False, True), (4, 1, 5, 5, 128, 0, False, False),
    (2, 3, 24, 2, 256, 64, True, False), (3, 4, 2, 1, 256, 256, False, False),
    (2, 9, 7, 7, 256, 240, True, True), (2, 700, 8, 4, 128, 112, False, False),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_qk_norm_rope_bitwise(qsa, case):
    B, R, Hq, Hkv, D, rot, inter, plus = case
    g = geom(batch=B, rows_per_req=R, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D)
    x = draw(B * R, Hq, Hkv, D, rot, seed=sum(case))
    nr = qsa.make_norm_rope(rot, interleaved=inter, eps=1e-5, weight_plus_one=plus)
    q_out = torch.full((B * R, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    k_out = torch.full((B * R, Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    cs = x["cs"] if rot else None
    qsa.qsa_qk_norm_rope(g, nr, x["q"], x["k"], x["q_weight"], x["k_weight"], cs, q_out, k_out)
    h = cr.host(x)
    for got, src, w in ((q_out, "q", "q_weight"), (k_out, "k", "k_weight")):
        ref = cr.norm_rope(h[src], h[w], h["cs"], rot, inter, 1e-5, plus)
        np.testing.assert_array_equal(got.cpu().view(torch.int16).numpy().view(np.uint16), cr.bits(ref))


def test_qk_norm_rope_in_place_and_without_weights(qsa):
    g = geom(batch=2, rows_per_req=3)
    x = draw(6, 8, 2, 128, 64, seed=5)
    nr = qsa.make_norm_rope(64)
    h = cr.host(x)
    q, k = x["q"].contiguous(), x["k"].contiguous()
    qsa.qsa_qk_norm_rope(g, nr, q, k, None, x["k_weight"], x["cs"], q, k)
    ref_q = cr.norm_rope(h["q"], None, h["cs"], 64, False, 1e-6, False)
    ref_k = cr.norm_rope(h["k"], h["k_weight"], h["cs"], 64, False, 1e-6, False)
    np.testing.assert_array_equal(q.cpu().float().numpy(), ref_q)
    np.testing.assert_array_equal(k.cpu().float().numpy(), ref_k)
    # keys alone
    k2 = torch.zeros_like(k)
    qsa.qsa_qk_norm_rope(g, nr, None, x["k"], None, x["k_weight"], x["cs"], None, k2)
    assert torch.equal(k2, k)


@pytest.mark.parametrize("spread", [0.0, 1e-20, 1e15])
def test_qk_norm_extremes(qsa, spread):
    # zeros, and magnitudes whose squares vanish or stay just inside fp32
    g = geom(batch=1, rows_per_req=2)
    x = draw(2, 8, 2, 128, 128, seed=3, spread=spread)
    nr = qsa.make_norm_rope(128, eps=1e-6)
    q, k = torch.empty(2, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(
        2, 2, 128, dtype=torch.bfloat16, device="cuda")
    qsa.qsa_qk_norm_rope(g, nr, x["q"], x["k"], x["q_weight"], x["k_weight"], x["cs"], q, k)
    h = cr.host(x)
    np.testing.assert_array_equal(q.cpu().float().numpy(), cr.norm_rope(
        h["q"], h["q_weight"], h["cs"], 128, False, 1e-6, False))


# ---------------------------------------------------------------------------
# append and read-back
# ---------------------------------------------------------------------------

def cache_case(**kw):
    base = dict(name="prologue", seed=41, batch=3, rows_per_req=1, num_q_heads=8, num_kv_heads=2,
                page_size=64, ctx_lo=300, ctx_hi=1300, k=6, window=2, max_blocks=21, pool="perm")
    base.update(kw)
    return qw.Case(**base)


APPEND = {
    "decode": cache_case(),
    "verify_p128": cache_case(rows_per_req=4, page_size=128, ctx_lo=129, ctx_hi=2600),
    "short_requests": cache_case(rows_per_req=6, ctx_lo=1, ctx_hi=8, max_blocks=2, k=2, window=1),
    "invalid_pages": cache_case(rows_per_req=5, invalid_frac=0.7),
    "hd256_p32": cache_case(head_dim=256, page_size=32, max_blocks=41, rows_per_req=4,
                            num_q_heads=24, num_kv_heads=2),
    "hd256_p64_rows": cache_case(head_dim=256, rows_per_req=131, ctx_lo=131, ctx_hi=800,
                                 num_q_heads=6, num_kv_heads=3),
    "one_head_rows": cache_case(rows_per_req=77, ctx_lo=60, ctx_hi=300, num_q_heads=1,
                                num_kv_heads=1),
}


def append(qsa, w, x, nr, pools, q_out):
    qsa.qsa_store_kv_tokens_rope(qw.geometry(w), nr, x["q"], x["k"], x["v"], x["ik_new"],
                                 x["q_weight"], x["k_weight"], x["cs"], w["k_scale"], w["v_scale"],
                                 w["page_table"], w["seqlens"], q_out, *(pools[n] for n in POOLS))


@pytest.mark.parametrize("name", sorted(APPEND))
@pytest.mark.parametrize("inter", [False, True])
def test_append_bitwise(qsa, name, inter):
    w = qw.make_workload(APPEND[name], "cuda")
    T, Hq, Hkv, D = w["batch"] * w["rows_per_req"], w["num_q_heads"], w["num_kv_heads"], w["head_dim"]
    x = draw(T, Hq, Hkv, D, 96, seed=T + D)
    nr = qsa.make_norm_rope(96, interleaved=inter, weight_plus_one=inter)
    pools = {n: w[n].clone() for n in POOLS}
    q_out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    append(qsa, w, x, nr, pools, q_out)
    torch.cuda.synchronize()
    h, hx = cr.host(w), cr.host(x)
    q, k, ref = cr.store_rope(h, hx, hx["cs"], 96, inter, 1e-6, inter)
    np.testing.assert_array_equal(q_out.cpu().float().numpy(), q)
    for n in POOLS:      # every byte, the untouched ones too
        np.testing.assert_array_equal(pools[n].cpu().numpy(), ref[n], err_msg=n)

    # the same bytes as the two calls one after the other
    two = {n: w[n].clone() for n in POOLS}
    k2 = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda")
    qsa.qsa_qk_norm_rope(qw.geometry(w), nr, None, x["k"], None, x["k_weight"], x["cs"], None, k2)
    qsa.qsa_store_kv_tokens(qw.geometry(w), k2, x["v"].contiguous(), x["ik_new"], w["k_scale"],
                            w["v_scale"], w["page_table"], w["seqlens"], *(two[n] for n in POOLS))
    for n in POOLS:
        assert torch.equal(two[n], pools[n]), n

    # read back; rows without a slot are left as they were
    ko = torch.full((T, Hkv, D), 5.0, dtype=torch.bfloat16, device="cuda")
    vo = torch.full((T, Hkv, D), 5.0, dtype=torch.bfloat16, device="cuda")
    qsa.qsa_load_kv_tokens(qw.geometry(w), w["page_table"], w["seqlens"], pools["k_pool"],
                           pools["k_sf"], pools["v_pool"], pools["v_sf"], w["k_scale"],
                           w["v_scale"], ko, vo)
    rk, rv = cr.load_rows({**h, **ref}, np.full((T, Hkv, D), 5.0, np.float32),
                          np.full((T, Hkv, D), 5.0, np.float32))
    np.testing.assert_array_equal(ko.cpu().float().numpy(), rk)
    np.testing.assert_array_equal(vo.cpu().float().numpy(), rv)


def test_append_without_queries_and_graph_replay(qsa):
    w = qw.make_workload(APPEND["verify_p128"], "cuda")
    T, Hq, Hkv, D = w["batch"] * w["rows_per_req"], w["num_q_heads"], w["num_kv_heads"], w["head_dim"]
    x = draw(T, Hq, Hkv, D, 64, seed=9)
    nr = qsa.make_norm_rope(64)
    pools = {n: w[n].clone() for n in POOLS}
    x0 = dict(x, q=None)
    append(qsa, w, x0, nr, pools, None)
    graph_pools = {n: w[n].clone() for n in POOLS}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        append(qsa, w, x0, nr, graph_pools, None)
    for n in POOLS:
        assert torch.equal(graph_pools[n], w[n]), "nothing runs at capture"
    graph.replay()
    graph.replay()
    for n in POOLS:
        assert torch.equal(graph_pools[n], pools[n]), n


# ---------------------------------------------------------------------------
# refusals that need tensors
# ---------------------------------------------------------------------------

def test_refusals(qsa):
    g = geom(batch=2, rows_per_req=3)
    x = draw(6, 8, 2, 128, 64, seed=1)
    nr = qsa.make_norm_rope(64)
    q, k = torch.empty(6, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(
        6, 2, 128, dtype=torch.bfloat16, device="cuda")
    cs = torch.zeros(6, 128, 2, device="cuda")    # more than any of the plans below reads
    ok = [g, nr, x["q"], x["k"], x["q_weight"], x["k_weight"], cs, q, k]

    def refused(i, value, kind):
        bad = list(ok)
        bad[i] = value
        with pytest.raises(kind):
            qsa.qsa_qk_norm_rope(*bad)

    refused(2, x["q"].float(), TypeError)
    refused(2, x["q"].cpu(), ValueError)
    refused(2, x["q"].transpose(0, 1), ValueError)
    refused(2, x["q"][:, :, ::2], ValueError)
    refused(2, x["q"][:5], ValueError)
    refused(6, cs[:1], ValueError)
    refused(6, None, qsa.QsaError)
    refused(8, x["k"], ValueError)                       # outputs are contiguous
    refused(1, qsa.make_norm_rope(24), qsa.QsaError)     # not a multiple of 16
    refused(1, qsa.make_norm_rope(144), qsa.QsaError)    # wider than the head
    refused(1, qsa.make_norm_rope(64, eps=float("nan")), qsa.QsaError)
    with pytest.raises(qsa.QsaError):                    # queries without a place to go
        qsa.qsa_qk_norm_rope(g, nr, x["q"], x["k"], None, None, x["cs"], None, k)
    rows = torch.empty(6, 2 * 128 + 4, dtype=torch.bfloat16, device="cuda")
    refused(3, rows[:, :256].view(6, 2, 128), qsa.QsaError)   # rows 520 bytes apart
