"""The prompt's layer and the decode steps behind it, as a server runs them: rotation rows of several
axes, norms, attention over packed prompts, their rows into the 8-bit cache, decode and verify rows over
it, another stream's work meanwhile; against 64 bits."""
import math

import numpy as np
import pytest
import torch

import cache8_reference as c8
import nvfp4_block_sparse_gb300 as qsa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def layer(seed, lens, Hkv, G, D, P, room):
    g = torch.Generator(device=DEV).manual_seed(seed)
    B, T = len(lens), sum(lens)
    w = c8.geometry(seed, B, 1, Hkv, D, P, max(lens) + room, max(lens) + room, G=G)
    for n in ("k_pool", "v_pool", "k_exp", "v_exp"):
        w[n][:] = 0x7F if n.endswith("pool") else 0          # what was there is nobody's business
    w["seqlens"] = np.array(lens, np.int32)
    x = torch.randn(T + 5, (G + 2) * Hkv, D, generator=g, device=DEV).to(torch.bfloat16)
    weight = (1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16)
    return w, x, weight


def rows_of(x, Hkv, G, weight):
    Hq = G * Hkv
    return dict(q=x[:, :Hq], k=x[:, Hq:Hq + Hkv], v=x[:, Hq + Hkv:], q_weight=weight, k_weight=weight)


@pytest.mark.parametrize("D,P,G", [(128, 64, 4), (256, 32, 6)])
def test_prompt_then_decode_then_verify(D, P, G):
    lens, Hkv, R = [130, 17, 300], 2, 3
    w, x, weight = layer(D, lens, Hkv, G, D, P, 40)
    d = c8.on_gpu(w)
    T, B = sum(lens), len(lens)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
    plan = qsa.make_rope_axes([D // 8, D // 8, D // 4], theta=1e6)
    pos = torch.stack([torch.cat([torch.arange(n, device=DEV) // k for n in lens]) for k in (1, 2, 3)]).to(torch.int32)
    cs = torch.empty(T, D // 2, 2, device=DEV)
    qsa.qsa_rope_axes_rows(plan, pos, cs)
    norm = qsa.make_norm_rope(D)
    step = qsa.PromptStep({n: w[n] for n in qsa.GEOM_FIELDS}, rows=T + 9)
    sm = 1 / math.sqrt(D)
    new = rows_of(x[:T], Hkv, G, weight)
    step.run(new, cu, norm, cs, sm, w=d)
    # the attention within the prompts, on the rows as they were normalised and rotated
    q, k = (torch.empty(T, n, D, dtype=torch.bfloat16, device=DEV) for n in (G * Hkv, Hkv))
    flat = qsa.make_geom(**dict({n: w[n] for n in qsa.GEOM_FIELDS}, batch=T, rows_per_req=1))
    qsa.qsa_qk_norm_rope(flat, norm, new["q"], new["k"], weight, weight, cs, q, k)
    torch.cuda.synchronize()
    assert step.status() == 0 and torch.equal(q, step.q[:T]) and torch.equal(k, step.k[:T])
    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    c8.compare(step.out[:T], step.lse[:T],
               c8.prompt(host(q), host(k), host(new["v"]), cu.tolist(), float(np.float32(sm))))
    # what the cache then holds
    pools = c8.store(w, k.float().cpu().numpy(), new["v"].float().cpu().numpy(), cu.tolist())
    names = ("k_pool", "k_exp", "v_pool", "v_exp")
    for n, ref in zip(names, pools):
        np.testing.assert_array_equal(d[n].cpu().numpy(), ref, err_msg=n)
    # decode rows, then verify rows, each appended and attended to
    for rows, seed in ((1, 1), (R, 2), (1, 3)):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        w = dict(w, rows_per_req=rows, seqlens=w["seqlens"] + rows, **dict(zip(names, pools)))
        d["seqlens"].add_(rows)
        y = torch.randn(B * rows, (G + 2) * Hkv, D, generator=gen, device=DEV).to(torch.bfloat16)
        cs2 = torch.empty(B * rows, D // 2, 2, device=DEV)
        at = (d["seqlens"].long()[:, None] - rows + torch.arange(rows, device=DEV)).flatten().to(torch.int32)
        qsa.qsa_rope_axes_rows(plan, at.repeat(3, 1), cs2)
        dense = qsa.DenseStep({n: w[n] for n in qsa.GEOM_FIELDS}, cache="fp8", window=200 if rows == R else 0)
        more = rows_of(y, Hkv, G, weight)
        dense.store(d, more, norm, cs2)
        dense.run(dict(d, sm_scale=sm), q=dense.q)
        torch.cuda.synchronize()
        assert dense.status() == 0
        pools = c8.store(w, dense.k.float().cpu().numpy(), more["v"].float().cpu().numpy())
        for n, ref in zip(names, pools):
            np.testing.assert_array_equal(d[n].cpu().numpy(), ref, err_msg=n)
        w = dict(w, **dict(zip(names, pools)))
        c8.compare(dense.out, dense.lse, c8.dense(w, dense.window, q=host(dense.q)))


def test_steps_behind_one_another_and_on_two_streams():
    """The same run without a wait between its calls, twice at once on two streams: the same bits."""
    lens, Hkv, G, D = [90, 260], 2, 4, 128
    w, x, weight = layer(3, lens, Hkv, G, D, 64, 20)
    T, sm = sum(lens), 128**-0.5
    cu = torch.tensor([0, 90, 350], dtype=torch.int32, device=DEV)
    norm, plan = qsa.make_norm_rope(D), qsa.make_rope_axes([32, 32], theta=1e4, layout="interleaved")
    pos = torch.stack([torch.cat([torch.arange(n, device=DEV) for n in lens])] * 2).to(torch.int32)
    geom = {n: w[n] for n in qsa.GEOM_FIELDS}

    def whole(stream, wait):
        d = c8.on_gpu(w)
        cs = torch.empty(T, D // 2, 2, device=DEV)
        prompt, dense = qsa.PromptStep(geom, T), qsa.DenseStep(geom, cache="fp8")
        cs2 = torch.empty(2, D // 2, 2, device=DEV)
        last = torch.tensor([[91, 261]] * 2, dtype=torch.int32, device=DEV)
        new = rows_of(x[T:T + 2], Hkv, G, weight)
        after = d["seqlens"] + 1
        torch.cuda.synchronize()
        pause = torch.cuda.synchronize if wait else (lambda: None)
        qsa.qsa_rope_axes_rows(plan, pos, cs, stream=stream)
        pause()
        prompt.run(rows_of(x[:T], Hkv, G, weight), cu, norm, cs, sm, w=d, stream=stream)
        pause()
        qsa.qsa_rope_axes_rows(plan, last, cs2, stream=stream)
        dense.store(dict(d, seqlens=after), new, norm, cs2, stream=stream)
        pause()
        dense.run(dict(d, seqlens=after, sm_scale=sm), q=dense.q, stream=stream)
        return prompt, dense, d

    want = whole(None, True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [whole(s, False) for s in streams]
        torch.cuda.synchronize()
        for prompt, dense, d in got:
            assert prompt.status() == 0 and dense.status() == 0
            assert torch.equal(prompt.out, want[0].out) and torch.equal(prompt.lse, want[0].lse)
            assert torch.equal(dense.out, want[1].out) and torch.equal(dense.lse, want[1].lse)
            assert all(torch.equal(d[n], want[2][n]) for n in ("k_pool", "k_exp", "v_pool", "v_exp"))


def test_many_rows_of_a_prompt_step():
    """More rows than a geometry has requests: the norms run in pieces."""
    T, D = 65535 + 12, 128
    geom = dict(batch=1, rows_per_req=1, num_q_heads=1, num_kv_heads=1, head_dim=D, index_dim=64, page_size=64,
                max_blocks=1, num_pages=1)
    x = torch.randn(T, 3, D, device=DEV).to(torch.bfloat16)
    new = dict(q=x[:, :1], k=x[:, 1:2], v=x[:, 2:], q_weight=None, k_weight=None)
    cs = torch.randn(T, 16, 2, device=DEV)
    step = qsa.PromptStep(geom, T, window=4)
    step.run(new, torch.tensor([0, 0], dtype=torch.int32, device=DEV), qsa.make_norm_rope(32), cs, 0.1)
    torch.cuda.synchronize()
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    a, b = new["k"][..., :16].float(), new["k"][..., 16:32].float()
    want = torch.cat([a * c - b * s, b * c + a * s, new["k"][..., 32:].float()], -1)
    assert step.status() == 0 and torch.equal(step.k, want.to(torch.bfloat16))
    with pytest.raises(ValueError):
        step.run(dict(new, k=torch.empty(T + 1, 1, D, dtype=torch.bfloat16, device=DEV)), None, None, None, 0.1)


def test_offsets_beyond_32_bits():
    """Pages at the far end of pools of more than 2^32 bytes."""
    Hkv, G, D, P = 8, 2, 256, 64
    per = Hkv * P * D
    NP = (1 << 32) // per + 40
    w, x, weight = layer(7, [70, 40], Hkv, G, D, P, 30)
    small = dict(w)
    w["num_pages"] = NP
    w["page_table"] = (NP - 1 - w["page_table"]).astype(np.int32)      # the last pages
    big = {n: torch.zeros(NP, Hkv, P, D, dtype=torch.uint8, device=DEV) for n in ("k_pool", "v_pool")}
    big.update({n: torch.zeros(NP, Hkv, P // 16, dtype=torch.uint8, device=DEV) for n in ("k_exp", "v_exp")})
    big.update(page_table=torch.from_numpy(w["page_table"]).to(DEV), seqlens=torch.from_numpy(w["seqlens"]).to(DEV))
    little = c8.on_gpu(small)
    res = []
    for geo, d in ((w, big), (small, little)):
        geom = {n: geo[n] for n in qsa.GEOM_FIELDS}
        cu = torch.tensor([0, 70, 110], dtype=torch.int32, device=DEV)
        prompt = qsa.PromptStep(geom, 110)
        prompt.run(rows_of(x[:110], Hkv, G, weight), cu, qsa.make_norm_rope(0), None, 0.05, w=d)
        out = []
        for rows in (1, 3, 20):
            g = dict(geom, rows_per_req=rows)
            dense = qsa.DenseStep(g, cache="fp8")
            q = torch.randn(2 * rows, G * Hkv, D, generator=torch.Generator(device=DEV).manual_seed(rows),
                            device=DEV).to(torch.bfloat16)
            dense.run(dict(d, sm_scale=0.05), q=q)
            kv = [torch.empty(2 * rows, Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
            qsa.qsa_load_kv_tokens_fp8(dense.cg, d["page_table"], d["seqlens"], d["k_pool"], d["k_exp"], d["v_pool"],
                                       d["v_exp"], *kv)
            out += [dense.out, dense.lse, *kv]
        torch.cuda.synchronize()
        res.append(out)
    assert all(torch.equal(a, b) for a, b in zip(*res))
