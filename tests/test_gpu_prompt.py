"""Attention over packed prompts on the GPU against 64 bits: lengths from one token on, every way that
heads fill tiles, windows and sinks, what lies outside the sequences, and the call's refusals."""
import math

import numpy as np
import pytest
import torch

import cache8_reference as c8
import nvfp4_block_sparse_gb300 as qsa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def geom(B, Hq, Hkv, D):
    return qsa.make_geom(batch=B, rows_per_req=1, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, index_dim=64,
                         page_size=64, max_blocks=1, num_pages=1)


def inputs(T, Hq, Hkv, D, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=DEV)
    x[:, :Hq] *= torch.linspace(0.5, 2.0, Hq, device=DEV)[:, None]
    x = x.to(torch.bfloat16)
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def run(q, k, v, cu, sm=None, window=0, sinks=None, out=None, lse=None, ws=None, stream=None, fill=9.0):
    T, Hq, D = q.shape
    g = geom(len(cu) - 1, Hq, k.shape[1], D)
    if ws is None:
        ws = torch.empty(qsa.qsa_prompt_attention_workspace_bytes(g, T), dtype=torch.uint8, device=DEV)
        qsa.qsa_workspace_init(ws)
    out = torch.full((T, Hq, D), fill, dtype=torch.bfloat16, device=DEV) if out is None else out
    lse = torch.full((T, Hq), fill, device=DEV) if lse is None else lse
    cu = cu if isinstance(cu, torch.Tensor) else torch.tensor(cu, dtype=torch.int32, device=DEV)
    qsa.qsa_prompt_attention(g, q, k, v, cu, 1 / math.sqrt(D) if sm is None else sm, out, lse, ws, window=window,
                             sinks=sinks, stream=stream)
    torch.cuda.synchronize()
    assert qsa.qsa_workspace_status(ws) == 0
    return out, lse


def host(*x):
    return [t.double().cpu().numpy() for t in x]


def check(q, k, v, cu, sm=None, window=0, sinks=None, alike=False):
    out, lse = run(q, k, v, cu, sm, window, sinks)
    sm = float(np.float32(1 / math.sqrt(q.shape[2]) if sm is None else sm))
    ref = c8.prompt(*host(q, k, v), cu, sm, window, None if sinks is None else sinks.double().cpu().numpy(), alike)
    rows = np.zeros(len(q), bool)
    for a, b in zip(cu[:-1], cu[1:]):
        rows[a:b] = True
    assert (out[torch.from_numpy(~rows)] == 9.0).all() and (lse[torch.from_numpy(~rows)] == 9.0).all()
    c8.compare(out[torch.from_numpy(rows)], lse[torch.from_numpy(rows)], [r[rows] for r in ref])
    return out, lse


def packed(lens, ahead=0):
    return [int(x) for x in np.concatenate([[0], np.cumsum(lens)]) + ahead]


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("Hkv,G", [(1, 1), (2, 2), (1, 3), (2, 4), (1, 7), (2, 8), (1, 12), (1, 16)])
@pytest.mark.parametrize("lens", [[1], [2, 1, 130], [127, 128, 129], [300, 0, 17, 64, 0, 1]])
def test_lengths(D, Hkv, G, lens):
    cu = packed(lens)
    check(*inputs(cu[-1], G * Hkv, Hkv, D, sum(lens)), cu)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("G,n", [(1, 700), (3, 1100), (8, 900), (100, 150), (128, 70)])
def test_long(D, G, n):
    cu = packed([n, n // 3])
    check(*inputs(cu[-1], G, 1, D, n), cu)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("window,sinks", [(1, False), (1, True), (37, False), (128, True), (300, False), (5000, True)])
def test_windows_and_sinks(D, window, sinks):
    cu = packed([500, 31, 257])
    s = torch.linspace(-3, 8, 8, device=DEV) if sinks else None
    check(*inputs(cu[-1], 8, 2, D, window), cu, window=window, sinks=s)


def test_sinks_alone():
    cu = packed([5, 600])
    check(*inputs(cu[-1], 4, 2, 128), cu, sinks=torch.tensor([-math.inf, 0.0, 30.0, -5.0], device=DEV))


@pytest.mark.parametrize("D", [128, 256])
def test_many_sequences(D):
    """More than a warp has lanes, empty ones among them, more units than pairs of CTAs."""
    rng = np.random.default_rng(D)
    lens = rng.integers(0, 90, 150)
    lens[[3, 77]] = 700
    cu = packed(lens)
    check(*inputs(cu[-1], 8, 4, D), cu)
    lens = [400, 1, 260] + [33] * 29                     # and exactly as many as it has lanes
    cu = packed(lens)
    check(*inputs(cu[-1], 12, 4, D), cu)


@pytest.mark.parametrize("D", [128, 256])
def test_outside_the_sequences(D):
    """Rows ahead of the first sequence and behind the last, NaN and infinities: nobody looks; neither does
    a sequence at its neighbours."""
    lens = [130, 77, 260]
    cu = packed(lens, ahead=11)
    q, k, v = inputs(cu[-1] + 40, 8, 2, D)
    plain, plain_lse = check(q, k, v, cu)
    for x in (q, k, v):
        x[:11], x[cu[-1]:] = math.nan, math.inf
    out, lse = run(q, k, v, cu)
    assert torch.equal(out, plain) and torch.equal(lse, plain_lse)
    k[cu[1]:cu[2]], v[cu[1]:cu[2]] = math.nan, math.inf
    out, lse = run(q, k, v, cu)
    for a, b in ((cu[0], cu[1]), (cu[2], cu[3])):
        assert torch.equal(out[a:b], plain[a:b]) and torch.equal(lse[a:b], plain_lse[a:b])
    assert not torch.isfinite(lse[cu[1]:cu[2]]).any()


@pytest.mark.parametrize("D", [128, 256])
def test_tokens_ahead_of_a_window(D):
    """Keys and values that no row sees any more, or not yet, hold what they like."""
    cu = packed([1400])
    q, k, v = inputs(1400, 4, 1, D)
    plain, plain_lse = run(q, k, v, cu, window=50)
    k[:20], v[:20] = math.nan, math.nan
    out, lse = run(q, k, v, cu, window=50)
    assert torch.equal(out[600:], plain[600:]) and torch.equal(lse[600:], plain_lse[600:])
    q, k, v = inputs(1400, 4, 1, D)
    plain, plain_lse = run(q, k, v, cu)
    k[1399], v[1399] = math.inf, math.nan
    out, lse = run(q, k, v, cu)
    assert torch.equal(out[:1399 - 512], plain[:1399 - 512]) and torch.equal(lse[:1399], plain_lse[:1399])


def test_not_finite_queries():
    cu = packed([300])
    q, k, v = inputs(300, 4, 1, 128)
    plain, plain_lse = run(q, k, v, cu)
    q[100, 2, 7], q[200, 0, 0] = math.nan, math.inf
    out, lse = run(q, k, v, cu)
    hit = torch.zeros(300, 4, dtype=torch.bool, device=DEV)
    hit[100, 2] = hit[200, 0] = True
    assert torch.isnan(out[hit]).all() and not torch.isfinite(lse[hit]).any()
    assert torch.equal(out[~hit], plain[~hit]) and torch.equal(lse[~hit], plain_lse[~hit])


@pytest.mark.parametrize("D", [128, 256])
def test_logits_that_rise_and_large_values(D):
    """Later tokens with logits far above the first ones' (the base moves), and values of any size."""
    cu = packed([700])
    q, k, v = inputs(700, 4, 1, D)
    k *= torch.linspace(0.1, 8.0, 700, device=DEV)[:, None, None].to(torch.bfloat16)
    check(q, k, v, cu, alike=True)
    check(q, k.flip(0).contiguous(), v, cu, alike=True)
    for size in (2.0**100, 2.0**-100):
        check(q, k, (v.float() * size).to(torch.bfloat16), cu, alike=True)


def test_strides_streams_graphs():
    lens = [260, 31, 500]
    cu = packed(lens)
    q, k, v = inputs(cu[-1], 8, 2, 128)
    plain = run(q, k, v, cu)
    own = run(q.contiguous(), k.contiguous(), v.contiguous(), cu)
    assert all(torch.equal(a, b) for a, b in zip(plain, own))
    side = torch.cuda.Stream()
    for _ in range(3):
        got = run(q, k, v, cu, stream=side)
        assert all(torch.equal(a, b) for a, b in zip(plain, got))
    g = geom(3, 8, 2, 128)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    qsa.qsa_workspace_init(ws)
    out, lse = torch.full_like(plain[0], 9.0), torch.full_like(plain[1], 9.0)
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qsa.qsa_prompt_attention(g, q, k, v, cud, 128**-0.5, out, lse, ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, plain[0]) and torch.equal(lse, plain[1])
    cud.copy_(torch.tensor([0, 100, 100, 400]))          # the captured call follows the lengths
    out.fill_(9.0)
    lse.fill_(9.0)
    graph.replay()
    torch.cuda.synchronize()
    want = run(q, k, v, [0, 100, 100, 400])
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_lengths_that_are_not():
    """Lengths out of range or falling are held at the rows there are: no fault, other rows as they were."""
    q, k, v = inputs(300, 4, 1, 128)
    plain = run(q, k, v, [0, 300])
    for cu in ([0, 1 << 30], [-5, 300], [-2**31, 2**31 - 1]):
        assert torch.equal(run(q, k, v, cu)[0], plain[0])
    run(q, k, v, [200, 100, 300])
    run(q, k, v, [0] * 20 + [500, 3] * 20 + [-7] * 20)


def test_refused():
    q, k, v = inputs(50, 8, 2, 128)
    cu = torch.tensor([0, 20, 50], dtype=torch.int32, device=DEV)
    g = geom(2, 8, 2, 128)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    qsa.qsa_workspace_init(ws)
    out, lse = torch.empty(50, 8, 128, dtype=torch.bfloat16, device=DEV), torch.empty(50, 8, device=DEV)
    def call(q=q, k=k, v=v, cu=cu, sm=0.1, out=out, lse=lse, ws=ws, window=0, sinks=None):
        qsa.qsa_prompt_attention(g, q, k, v, cu, sm, out, lse, ws, window=window, sinks=sinks)
    call()
    for kw in (dict(k=k[:49]), dict(q=q[:, :4]), dict(v=v[..., :64]), dict(cu=cu[:2]), dict(out=out[1:]),
               dict(lse=lse[:49]), dict(cu=cu.cpu()), dict(sinks=torch.zeros(7, device=DEV)), dict(q=q.transpose(0, 1))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(q=q.float()), dict(cu=cu.long()), dict(out=out.half())):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(sm=0.0), dict(sm=math.inf), dict(window=-1), dict(ws=ws[:255]), dict(ws=ws[16:])):
        with pytest.raises(qsa.QsaError):
            call(**kw)
    call(q=q[:0], k=k[:0], v=v[:0], cu=torch.zeros(3, dtype=torch.int32, device=DEV))      # no rows


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("gap", [17.625, 0.357])
def test_sums_of_long_rows(D, gap):
    """131072 tokens: a first one whose weight the others', 2^-25.4 of it each, would vanish next to; and others
    of 0.7 of the first's, which are alike to the last bit."""
    n, cu = 131072, packed([131072])
    q, k, v = inputs(n, 1, 1, D)
    q[:], k[:] = 0, 0
    q[..., 0], k[0, 0, 0] = 1, gap
    out, lse = run(q, k, v, cu, sm=1.0)
    kh, vh = host(k[:, 0], v[:, 0])
    for r in (60000, 100000, n - 2, n - 1):
        want = c8.attend(host(q[r])[0], kh[:r + 1], vh[:r + 1], 1.0, weight=2.0**-8, alike=True)
        # lse as of attend().  out: the tensor cores add 16 products at a time to what is there, each cut off at 2^-25
        # of the largest, and round: 16 2^-25 + 2^-23 < 16 2^-24 for 16 tokens
        mag = np.exp(kh[None, :r + 1, 0] - want[1][:, None]) @ np.abs(vh[:r + 1])
        c8.compare(out[r], lse[r], [want[0], want[1], want[2] + (r + 1) * 2.0**-24 * mag, want[3]])


def spoiled(v, G, cu, window, at):
    """v with elements that are not finite put at `at` (row, KV head, dim, value), and what the outputs have of them:
    the rows that see them, in that dim, their sum."""
    x, add = v.clone(), torch.zeros(v.shape[0], v.shape[1] * G, v.shape[2], device=DEV)
    for row, h, d, value in at:
        x[row, h, d] = value
        end = min(b for b in cu if b > row)
        end = min(end, row + window) if window else end
        add[row:end, h * G:(h + 1) * G, d] += value
    return x, add


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("G", [1, 4, 8])
@pytest.mark.parametrize("window", [0, 1, 50, 128, 700])
def test_values_that_a_row_does_not_see(D, G, window):
    """Values that are not finite make so the rows that see them, in their dims, and nothing else: not the rows
    ahead of them, and not those that have left them behind."""
    cu = packed([1400, 3, 700])
    q, k, v = inputs(cu[-1], 2 * G, 2, D)
    rng = np.random.default_rng(G)
    kinds = [math.nan, math.inf, -math.inf]
    at = [(int(r), int(rng.integers(2)), int(rng.integers(D)), kinds[int(rng.integers(3))])
          for r in rng.integers(0, cu[-1], 12)]
    at += [(0, 0, 0, math.nan), (1399, 1, D - 1, math.inf), (1401, 0, 5, math.inf), (1402, 0, 5, -math.inf),
           (cu[-1] - 1, 1, 64, math.nan)]
    plain, plain_lse = run(q, k, v, cu, window=window)
    x, add = spoiled(v, G, cu, window, at)
    out, lse = run(q, k, x, cu, window=window)
    assert torch.equal(lse, plain_lse)
    want = (plain.float() + add).to(torch.bfloat16)
    bad = ~((out == want) | (out.isnan() & want.isnan()))
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist())


def test_values_that_a_row_does_not_see_many_sequences():
    """The same where each CTA has many units, some with such values and some without."""
    rng = np.random.default_rng(3)
    cu = packed(rng.integers(1, 300, 400))
    for D in (128, 256):
        q, k, v = inputs(cu[-1], 8, 2, D)
        at = [(int(r), int(rng.integers(2)), int(rng.integers(D)), math.nan) for r in rng.integers(0, cu[-1], 60)]
        plain, plain_lse = run(q, k, v, cu)
        x, add = spoiled(v, 4, cu, 0, at)
        out, lse = run(q, k, x, cu)
        want = (plain.float() + add).to(torch.bfloat16)
        assert torch.equal(lse, plain_lse) and torch.equal(out.nan_to_num(7.0), want.nan_to_num(7.0))
