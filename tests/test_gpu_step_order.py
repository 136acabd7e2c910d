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


def alternate(write, read, results):
    """write(i) and read(out) by turns, i = 0, 1, 0, ..: 30 times without a synchronise, compared
    with what a synchronise between the two gives."""
    want = []
    for i in range(2):
        write(i)
        torch.cuda.synchronize()
        out = results()
        read(out)
        torch.cuda.synchronize()
        want.append(out)
    assert not torch.equal(want[0][0], want[1][0])
    got = [results() for _ in range(30)]
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        write(i % 2)
        read(out)
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        for a, b in zip(out, want[i % 2]):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("rows", [1, 3, 12, 70])
@pytest.mark.parametrize("geometry", sorted(GEOMS))
def test_a_dense_step_back_to_back(qsa, geometry, rows):
    # rotation rows -> norms, rotation and append -> dense attention, and the rows read back, each
    # directly behind the one that writes what it reads
    case = qw.Case(name="order", seed=62, batch=8, rows_per_req=rows, ctx_lo=300, ctx_hi=700, k=6,
                   window=2, **GEOMS[geometry])
    w = qw.make_workload(case, "cuda")
    step = qsa.DenseStep(qw.geometry(w))
    T, Hq, Hkv, D = 8 * rows, w["num_q_heads"], w["num_kv_heads"], w["head_dim"]
    gen = torch.Generator(device="cuda").manual_seed(5)
    news = []
    for _ in range(2):
        x = torch.randn(T, Hq + 2 * Hkv, D, generator=gen, device="cuda").to(torch.bfloat16)
        news.append(dict(q=x[:, :Hq], k=x[:, Hq:Hq + Hkv], v=x[:, Hq + Hkv:], q_weight=None, k_weight=None,
                         ik_new=torch.randint(-127, 128, (T, 64), generator=gen, device="cuda").to(torch.int8)))
    ropes = [qsa.make_rope(rotary_dim=64, theta=t) for t in (1e4, 1e6)]
    nr = qsa.make_norm_rope(64)
    cs = torch.empty(T, 32, 2, device="cuda")

    def write(i):
        qsa.qsa_rope_rows(step.cg, ropes[i], w["seqlens"], cs)
        step.store(w, news[i], nr, cs)

    def read(out):
        step.run(w, q=step.q, out=out[0], lse=out[1])
        qsa.qsa_load_kv_tokens(step.cg, w["page_table"], w["seqlens"], w["k_pool"], w["k_sf"], w["v_pool"],
                               w["v_sf"], w["k_scale"], w["v_scale"], out[2], out[3])

    def read_back_first(out):
        qsa.qsa_load_kv_tokens(step.cg, w["page_table"], w["seqlens"], w["k_pool"], w["k_sf"], w["v_pool"],
                               w["v_sf"], w["k_scale"], w["v_scale"], out[2], out[3])
        step.run(w, q=step.q, out=out[0], lse=out[1])

    def results():
        return [torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(T, Hq, device="cuda"),
                torch.zeros(T, Hkv, D, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(T, Hkv, D, dtype=torch.bfloat16, device="cuda")]

    alternate(write, read, results)
    alternate(write, read_back_first, results)
    assert step.status() == 0
