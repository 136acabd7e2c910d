"""GPU tests of calls directly behind the prologue on one stream: the sparse
decode attention reads the queries that the prologue's launch before it writes,
with nothing in between (layers that share a selection).  Both launches may
overlap, so the bits are compared with a run that synchronises between them."""
import pytest
import torch

import qsa_workloads as qw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    import nvfp4_block_sparse_gb300 as m
    m.load(build_if_missing=True)
    return m


GEOMS = {
    "hd128": dict(num_q_heads=32, num_kv_heads=4, page_size=64, max_blocks=12),
    "hd256": dict(num_q_heads=24, num_kv_heads=2, page_size=32, head_dim=256, max_blocks=24),
}


@pytest.mark.parametrize("attention", ["sparse_decode", "select_sparse_decode", "noalloc"])
@pytest.mark.parametrize("prologue", ["norm_rope", "store"])
@pytest.mark.parametrize("geometry", sorted(GEOMS))
def test_queries_of_the_launch_before(qsa, geometry, prologue, attention):
    case = qw.Case(name="order", seed=61, batch=64, rows_per_req=1, ctx_lo=300, ctx_hi=700, k=6,
                   window=2, **GEOMS[geometry])
    w = qw.make_workload(case, "cuda")
    g = qw.geometry(w)
    T, Hq, Hkv, D = 64, w["num_q_heads"], w["num_kv_heads"], w["head_dim"]
    gen = torch.Generator(device="cuda").manual_seed(4)
    new = [torch.randn(T, Hq + 2 * Hkv, D, generator=gen, device="cuda").to(torch.bfloat16)
           for _ in range(2)]
    for x in new:      # the same keys and values, so that only the queries differ
        x[:, Hq:] = new[0][:, Hq:]
    ik = torch.randint(-127, 128, (T, 64), generator=gen, device="cuda").to(torch.int8)
    weight = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    cs = torch.empty(T, 32, 2, device="cuda")
    qsa.qsa_rope_rows(g, qsa.make_rope(rotary_dim=64, theta=1e6), w["seqlens"], cs)
    nr = qsa.make_norm_rope(64)
    q = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    k_out = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda")
    pools = [w[n] for n in ("k_pool", "k_sf", "v_pool", "v_sf")]
    scales = (w["k_scale"], w["v_scale"])
    if prologue == "store":     # the rows are there before the selection is made
        qsa.qsa_store_kv_tokens_rope(g, nr, None, new[0][:, Hq:Hq + Hkv], new[0][:, Hq + Hkv:], ik,
                                     None, weight, cs, *scales, w["page_table"], w["seqlens"], None,
                                     *pools, w["ik_pool"])
    step = qsa.DecodeStep(g, 6, 2)
    step.run(w)
    torch.cuda.synchronize()
    sel = step.sel.clone()

    def write_queries(x):
        if prologue == "store":
            qsa.qsa_store_kv_tokens_rope(g, nr, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], ik,
                                         weight, weight, cs, *scales, w["page_table"], w["seqlens"],
                                         q, *pools, w["ik_pool"])
        else:
            qsa.qsa_qk_norm_rope(g, nr, x[:, :Hq], x[:, Hq:Hq + Hkv], weight, weight, cs, q, k_out)

    def attend(out, lse):
        tail = (*scales, w["sm_scale"], w["page_table"], w["seqlens"])
        if attention == "sparse_decode":
            qsa.qsa_sparse_decode(g, q, *pools, *tail, sel, 6, out, lse, step.workspace)
        elif attention == "noalloc":
            qsa.qsa_sparse_decode_noalloc(g, q, *pools, *tail, sel, 6, out, lse)
        else:
            qsa.qsa_select_sparse_decode(g, step.scores, 2, q, *pools, *tail, 6, step.sel, step.nsel,
                                         out, lse, step.workspace)

    out = torch.empty(2, T, Hq, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(2, T, Hq, device="cuda")
    for i in range(2):
        write_queries(new[i])
        torch.cuda.synchronize()
        attend(out[i], lse[i])
        torch.cuda.synchronize()
    assert not torch.equal(out[0], out[1])
    got = torch.empty(40, T, Hq, D, dtype=torch.bfloat16, device="cuda")
    got_lse = torch.empty(40, T, Hq, device="cuda")
    for i in range(40):
        write_queries(new[i % 2])
        attend(got[i], got_lse[i])
    torch.cuda.synchronize()
    for i in range(40):
        assert torch.equal(got[i], out[i % 2]) and torch.equal(got_lse[i], lse[i % 2]), i
