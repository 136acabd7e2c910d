"""The operators on prompts and the 8-bit cache at their largest: rows and tokens whose offsets pass 32 bits,
against the same rows in small calls, or against 64 bits."""
import math

import pytest
import torch

import nvfp4_block_sparse_gb300 as qsa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def geom(**kw):
    base = dict(batch=1, rows_per_req=1, num_q_heads=1, num_kv_heads=1, head_dim=128, index_dim=64, page_size=64,
                max_blocks=1, num_pages=1)
    return qsa.make_geom(**dict(base, **kw))


def test_axes_rows_past_32_bits():
    T = 1 << 24                                        # as many as are allowed: 2^32 floats
    plan = qsa.make_rope_axes([40, 44, 44], theta=1e6)
    pos = torch.arange(T, dtype=torch.int32, device=DEV).repeat(3, 1)
    pos[1] //= 2
    pos[2] //= 3
    cs = torch.empty(T, 128, 2, device=DEV)
    qsa.qsa_rope_axes_rows(plan, pos, cs)
    for a in (0, (1 << 23) - 50, T - 999):
        part = torch.empty(999, 128, 2, device=DEV)
        qsa.qsa_rope_axes_rows(plan, pos[:, a:a + 999].contiguous(), part)
        torch.cuda.synchronize()
        assert torch.equal(cs[a:a + 999], part)


def test_rows_of_the_cache_past_32_bits():
    """Four requests of 2^22 new rows of two heads: 2^32 elements in and codes out."""
    T, Hkv, D, P, B = 1 << 24, 2, 128, 128, 4
    MB = T // P
    pools = {n: torch.full((MB, Hkv, P, D), 0x7F, dtype=torch.uint8, device=DEV) for n in ("k_pool", "v_pool")}
    pools.update({n: torch.zeros(MB, Hkv, P // 16, dtype=torch.uint8, device=DEV) for n in ("k_exp", "v_exp")})
    order = ("k_pool", "k_exp", "v_pool", "v_exp")
    table = torch.arange(MB - 1, -1, -1, dtype=torch.int32, device=DEV).view(B, MB // B)
    lens = torch.full((B,), T // B, dtype=torch.int32, device=DEV)
    kv = torch.empty(T, 2 * Hkv, D, dtype=torch.bfloat16, device=DEV)
    for a in range(0, T, 1 << 20):
        kv[a:a + (1 << 20)] = torch.randn(1 << 20, 2 * Hkv, D, device=DEV).to(torch.bfloat16)
    cu = torch.arange(0, T + 1, T // B, dtype=torch.int32, device=DEV)
    g = geom(batch=B, num_q_heads=Hkv, num_kv_heads=Hkv, page_size=P, max_blocks=MB // B, num_pages=MB)
    qsa.qsa_store_kv_tokens_fp8(g, kv[:, :Hkv], kv[:, Hkv:], table, lens, *(pools[n] for n in order), cu_rows=cu)
    back = torch.empty(2, T, Hkv, D, dtype=torch.bfloat16, device=DEV)
    qsa.qsa_load_kv_tokens_fp8(g, table, lens, *(pools[n] for n in order), back[0], back[1], cu_rows=cu)
    torch.cuda.synchronize()
    for a in range(0, T, 1 << 20):                     # within half a step of the block's codes everywhere
        for x, y in ((kv[a:a + (1 << 20), :Hkv], back[0, a:a + (1 << 20)]),
                     (kv[a:a + (1 << 20), Hkv:], back[1, a:a + (1 << 20)])):
            x, y = x.float(), y.float()
            # (steps of 2^-3 of a code's binade; below 2^-6 of the block's scale, at most its largest / 224, of 2^-9)
            top = x.reshape(-1, 16, Hkv, D).abs().amax((1, 3), keepdim=True).expand(-1, 16, Hkv, D).reshape(x.shape)
            assert ((x - y).abs() <= torch.maximum(x.abs() / 16, top / 224 / 1024)).all()
    n, last = 1000 * 16, T - 1000 * 16                 # the last rows alone: the same bytes
    small = {k: torch.zeros_like(v[:n // P]) for k, v in pools.items()}
    g2 = geom(num_q_heads=Hkv, num_kv_heads=Hkv, page_size=P, max_blocks=n // P, num_pages=n // P)
    qsa.qsa_store_kv_tokens_fp8(g2, kv[last:, :Hkv], kv[last:, Hkv:],
                                torch.arange(n // P - 1, -1, -1, dtype=torch.int32, device=DEV)[None].contiguous(),
                                torch.tensor([n], dtype=torch.int32, device=DEV), *(small[k] for k in order),
                                cu_rows=torch.tensor([0, n], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert all(torch.equal(small[k], pools[k][:n // P]) for k in order)


@pytest.mark.parametrize("R", [1, 6])
def test_a_context_of_millions(R):
    """4 194 304 tokens (less a few) of one request, few vectors and tiles; a window at the far end."""
    P, D, MB, G = 128, 128, 1 << 15, 4
    L = MB * P - 5
    gen = torch.Generator(device=DEV).manual_seed(R)
    pools = []
    for _ in "kv":
        code = torch.randint(0, 256, (MB, 1, P, D), generator=gen, dtype=torch.uint8, device=DEV)
        code[(code & 0x7F) > 0x50] &= 0xBF                               # finite and of moderate size
        pools += [code, torch.randint(120, 124, (MB, 1, P // 16), generator=gen, dtype=torch.uint8, device=DEV)]
    table = torch.randperm(MB, generator=gen, device=DEV).to(torch.int32)[None].contiguous()
    lens = torch.tensor([L], dtype=torch.int32, device=DEV)
    q = torch.randn(R, G, D, generator=gen, device=DEV).to(torch.bfloat16)
    g = geom(num_q_heads=G, rows_per_req=R, page_size=P, max_blocks=MB, num_pages=MB)
    ws = torch.empty(qsa.qsa_dense_attention_fp8_workspace_bytes(g), dtype=torch.uint8, device=DEV)
    qsa.qsa_workspace_init(ws)

    def values(code, exps):
        x = code[table[0].long()].reshape(-1, 16, D).view(torch.float8_e4m3fn).float()
        return (x * torch.exp2(exps[table[0].long()].reshape(-1, 1, 1).float() - 127)).reshape(-1, D)[:L]
    k, v = values(pools[0], pools[1]), values(pools[2], pools[3])
    for window in (0, 5000):
        out, lse = torch.empty(R, G, D, dtype=torch.bfloat16, device=DEV), torch.empty(R, G, device=DEV)
        qsa.qsa_dense_attention_fp8(g, q, *pools, 0.1, table, lens, out, lse, ws, window=window)
        torch.cuda.synchronize()
        assert qsa.qsa_workspace_status(ws) == 0
        for r in range(R):
            n = L - R + r + 1
            lo = max(0, n - window) if window else 0
            z = 0.1 * (q[r].double() @ k[lo:n].double().T)
            want = torch.logsumexp(z, -1)
            wt = torch.exp(z - want[:, None])
            o = wt @ v[lo:n].double()
            # logits and sums in fp32 (2^-24 of |z| <= 64 or so, and of a sum of 2^22 in a tree of chunks), the
            # weights' 2^-11 and the output's 2^-8, of what each is of
            size = wt @ v[lo:n].double().abs()
            tol = size * (2.0**-11 + 2.0**-13) + o.abs() * 2.0**-8 + 1e-30
            assert (lse[r].double() - want).abs().max() <= 2.0**-24 * 64 * 8 + 2.0**-13
            assert ((out[r].double() - o).abs() <= tol).all()


def test_prompts_past_32_bits():
    """2^31 elements of queries and more: the last sequences as in a small call, bit for bit."""
    n, B, Hq, Hkv, D = 100, 661, 128, 8, 256
    T = n * B
    assert T * Hq * D > 1 << 31
    gen = torch.Generator(device=DEV).manual_seed(0)
    q = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
    for a in range(0, T, 6610):
        q[a:a + 6610] = torch.randn(6610, Hq, D, generator=gen, device=DEV).to(torch.bfloat16)
    kv = torch.randn(T, 2 * Hkv, D, generator=gen, device=DEV).to(torch.bfloat16)

    def run(a):
        rows = T - a
        g = geom(batch=rows // n, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D)
        ws = torch.empty(qsa.qsa_prompt_attention_workspace_bytes(g, rows), dtype=torch.uint8, device=DEV)
        qsa.qsa_workspace_init(ws)
        out = torch.zeros(rows, Hq, D, dtype=torch.bfloat16, device=DEV)
        lse = torch.zeros(rows, Hq, device=DEV)
        cu = torch.arange(0, rows + 1, n, dtype=torch.int32, device=DEV)
        qsa.qsa_prompt_attention(g, q[a:], kv[a:, :Hkv], kv[a:, Hkv:], cu, 1 / math.sqrt(D), out, lse, ws)
        torch.cuda.synchronize()
        assert qsa.qsa_workspace_status(ws) == 0
        return out, lse
    out, lse = run(0)
    part, part_lse = run(T - 3 * n)
    assert torch.equal(out[-3 * n:], part) and torch.equal(lse[-3 * n:], part_lse)
    z = torch.einsum("hd,sd->hs", q[-1, :16].double(), kv[-n:, 0].double()) / math.sqrt(D)
    assert (lse[-1, :16].double() - torch.logsumexp(z, -1)).abs().max() < 1e-5
