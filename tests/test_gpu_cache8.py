"""Rotation rows of several axes and the 8-bit cache's append and read-back on
the GPU, against plain forms in 64 bits: codes and exponents bit for bit."""
import math

import numpy as np
import pytest
import torch

import cache8_reference as c8
import nvfp4_block_sparse_gb300 as qsa

pytestmark = pytest.mark.gpu
DEV = "cuda"
POOLS = ("k_pool", "k_exp", "v_pool", "v_exp")


def geom(w, **kw):
    return qsa.make_geom(**{n: dict(w, **kw)[n] for n in qsa.GEOM_FIELDS})


# ---------------------------------------------------------------------------
# rotation rows
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("layout,pairs", [
    ("sections", [64]), ("sections", [16, 24, 24]), ("sections", [1, 2, 4, 1]), ("interleaved", [24, 20, 20]),
    ("interleaved", [5, 3]), ("spectra", [11, 21, 32]), ("spectra", [100, 20, 5, 3])])
@pytest.mark.parametrize("T", [1, 77, 5000])
def test_axes_rows(layout, pairs, T):
    scaling = dict(scaling="yarn", factor=4.0, original_context=8192) if layout != "sections" else {}
    plan = qsa.make_rope_axes(pairs, theta=1e6, layout=layout, **scaling)
    axis = c8.axis_of(pairs, layout)
    assert list(plan.axis[:sum(pairs)]) == axis
    rng = np.random.default_rng(T)
    pos = rng.integers(-2**31, 2**31, (len(pairs), T)) if T == 77 else rng.integers(0, 200000, (len(pairs), T))
    cs = torch.full((T + 3, sum(pairs), 2), 7.0, device=DEV)
    qsa.qsa_rope_axes_rows(plan, torch.from_numpy(pos.astype(np.int32)).to(DEV), cs)
    got = cs.cpu().double().numpy()
    assert (got[T:] == 7.0).all()
    turns = np.array([plan.rope.turns[i] for i in range(sum(pairs))], dtype=np.uint64)
    phase = pos[axis].T.astype(np.int64).view(np.uint64) * turns       # modulo one turn
    a = phase.astype(np.float64) * (2 * math.pi / 2.0**64)
    ref = np.stack([np.cos(a), np.sin(a)], -1) * plan.rope.amplitude
    # 2e-7 is stated; of the reference's own, 2 pi (2^-53 + 2^-53)
    assert np.abs(got[:T] - ref).max() <= (2e-7 + 2e-15) * plan.rope.amplitude


def test_one_axis_is_the_plain_rows():
    T, pos = 300, torch.randint(0, 1 << 20, (300,), dtype=torch.int32, device=DEV)
    for scaling in ("none", "wavelength"):
        kw = dict(theta=5e5, scaling=scaling, factor=8.0, original_context=8192)
        a, b = (torch.empty(T, 48, 2, device=DEV) for _ in range(2))
        g = qsa.make_geom(batch=T, rows_per_req=1, num_q_heads=1, num_kv_heads=1, head_dim=128, index_dim=64,
                          page_size=64, max_blocks=1, num_pages=1)
        qsa.qsa_rope_rows(g, qsa.make_rope(rotary_dim=96, **kw), None, a, positions=pos)
        qsa.qsa_rope_axes_rows(qsa.make_rope_axes([48], **kw), pos[None], b)
        assert torch.equal(a, b)
        # three axes at the same positions, too
        qsa.qsa_rope_axes_rows(qsa.make_rope_axes([16, 16, 16], **kw), pos.repeat(3, 1), b)
        assert torch.equal(a, b)


def test_axes_rows_refused():
    plan = qsa.make_rope_axes([4, 4], theta=1e4)
    pos, cs = torch.zeros(2, 5, dtype=torch.int32, device=DEV), torch.empty(5, 8, 2, device=DEV)
    for bad in (lambda: qsa.qsa_rope_axes_rows(plan, pos[:1], cs), lambda: qsa.qsa_rope_axes_rows(plan, pos.T, cs),
                lambda: qsa.qsa_rope_axes_rows(plan, pos, cs[:4]), lambda: qsa.qsa_rope_axes_rows(plan, pos.cpu(), cs),
                lambda: qsa.qsa_rope_axes_rows(plan, pos[:, ::2], cs)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(TypeError):
        qsa.qsa_rope_axes_rows(plan, pos.long(), cs)
    qsa.qsa_rope_axes_rows(plan, pos[:, :0].contiguous(), cs)      # no rows: nothing to do


# ---------------------------------------------------------------------------
# append and read-back
# ---------------------------------------------------------------------------

def rows(T, Hkv, D, seed, spread=0.4):
    """Keys and values as parts of wider rows."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, 2 * Hkv + 1, D, generator=g, device=DEV)
    x *= torch.exp(spread * torch.randn(T, 2 * Hkv + 1, 1, generator=g, device=DEV))
    return x.to(torch.bfloat16)


def check(w, k, v, cu=None, back=None):
    """Appends and reads back on the GPU, against the reference."""
    d = c8.on_gpu(w)
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)
    qsa.qsa_store_kv_tokens_fp8(geom(w), k, v, d["page_table"], d["seqlens"], *(d[n] for n in POOLS), cu_rows=cud)
    ref = c8.store(w, k.float().cpu().numpy(), v.float().cpu().numpy(), cu)
    for n, x in zip(POOLS, ref):
        np.testing.assert_array_equal(d[n].cpu().numpy(), x, err_msg=n)
    back = w["rows_per_req"] if back is None else back
    T = len(k) if cu is not None else w["batch"] * back
    out = [torch.full((T, w["num_kv_heads"], w["head_dim"]), 3.5, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    w2 = dict(w, rows_per_req=back)
    qsa.qsa_load_kv_tokens_fp8(geom(w2), d["page_table"], d["seqlens"], *(d[n] for n in POOLS), *out, cu_rows=cud)
    want = c8.load(w2, ref, T, *(np.full(tuple(o.shape), 3.5) for o in out), cu)
    for got, x in zip(out, want):
        np.testing.assert_array_equal(got.double().cpu().numpy(), x)
    return d


@pytest.mark.parametrize("D,P", [(128, 64), (128, 128), (256, 32), (256, 64)])
@pytest.mark.parametrize("B,R,Hkv,lo,hi", [(1, 1, 1, 1, 1), (5, 1, 2, 1, 300), (9, 4, 2, 4, 200), (3, 37, 1, 40, 90),
                                           (2, 64, 3, 64, 64), (40, 3, 5, 3, 70)])
def test_append(D, P, B, R, Hkv, lo, hi):
    w = c8.geometry(B * R + D, B, R, Hkv, D, P, lo, hi, holes=0.1 if B > 5 else 0.0)
    x = rows(B * R, Hkv, D, R)
    check(w, x[:, :Hkv], x[:, Hkv:2 * Hkv], back=R + 15)


@pytest.mark.parametrize("D,P", [(128, 64), (256, 32)])
def test_append_packed(D, P):
    lens = [17, 0, 1, 200, 3, 0, 33, 64]
    w = c8.geometry(3, len(lens), 1, 2, D, P, 200, 330)
    w["seqlens"][:3] = [20, 0, 1]
    w["seqlens"][4] = 2             # fewer tokens than rows: the first of these has no place
    cu = np.concatenate([[0], np.cumsum(lens)])
    x = rows(cu[-1] + 9, 2, D, 1)   # rows behind the last request
    check(w, x[:, :2], x[:, 2:4], cu)
    check(w, x[4:, :2], x[4:, 2:4], cu + 5)          # and ahead of the first


def test_append_many_rows():
    """More rows than CTAs at a time, blocks that cross the rows of a CTA."""
    lens = [1700, 3, 2111, 1]
    w = c8.geometry(4, 4, 1, 2, 128, 64, 2111, 2200)
    cu = np.concatenate([[0], np.cumsum(lens)])
    x = rows(cu[-1], 2, 128, 5)
    check(w, x[:, :2], x[:, 2:4], cu)


def test_exponents_grow_and_hold():
    """A token after another with magnitudes that rise and fall: the block's codes at every step,
    and what rescaled values are worth."""
    w = c8.geometry(7, 1, 1, 1, 128, 64, 1, 1, spare=0)
    w["page_table"] = np.zeros((1, 1), np.int32)
    pools = [w[n] for n in POOLS]
    x = rows(16, 1, 128, 3, 0.0)
    for t, size in enumerate([1.0, 0.01, 40.0, 3.0, 1e4, 2.0**70, 1e-30, 0.0, 1.0, 5.0, 1e9, 1.0, 1.0, 2.0**80, 1.0, 1.0]):
        w.update(zip(POOLS, pools))
        w["seqlens"] = np.array([t + 1], np.int32)
        y = (x[t:t + 1].float() * size).to(torch.bfloat16)
        d = check(w, y[:, :1], y[:, 1:2])
        pools = [d[n].cpu().numpy() for n in POOLS]
    assert pools[1][0, 0, 0] == 127 + 64      # held at the largest


def test_a_block_begins_anew():
    """The first slot of a block forgets what the page's former tenant left."""
    w = c8.geometry(8, 1, 1, 2, 256, 32, 17, 17)
    w["k_exp"][:], w["v_exp"][:] = 200, 255
    x = rows(1, 2, 256, 3)
    d = check(w, x[:, :2], x[:, 2:4])
    page = w["page_table"][0, 0]
    assert (d["k_exp"][page, :, 1] < 140).all() and (d["k_exp"][page, :, 0] == 200).all()


@pytest.mark.parametrize("D", [128, 256])
def test_extremes(D):
    """Zeros, values next to every rounding border, not finite ones, largest and smallest bf16."""
    P = 64
    w = c8.geometry(9, 4, 16, 1, D, P, 16, 16)
    x = rows(64, 1, D, 2)[:, :2].clone()
    x[:16] = 0
    grid = torch.tensor([m * 2.0**-9 for m in range(16)] + [(8 + m) * 2.0**e for e in range(-6, 5) for m in range(8)])
    mids = ((grid[1:] + grid[:-1]) / 2).to(torch.bfloat16)
    x[16:32] = mids[torch.arange(16 * 2 * D) % len(mids)].view(16, 2, D).to(DEV)
    x[16, :, 0] = 448.0
    x[32, 0, 3], x[33, 1, 5], x[34, 0, 7] = math.inf, -math.inf, math.nan
    x[48:] = torch.finfo(torch.bfloat16).max
    x[49] = torch.finfo(torch.bfloat16).tiny
    x[50] = 1e-40
    check(w, x[:, :1], x[:, 1:2])


def test_strides_streams_and_graphs():
    """Rows of one projection, another stream, a captured call that follows the lengths."""
    w = c8.geometry(10, 6, 2, 2, 128, 64, 30, 120)
    d = c8.on_gpu(w)
    x = rows(12, 2, 128, 3)
    ref = c8.store(w, x[:, :2].float().cpu().numpy(), x[:, 2:4].float().cpu().numpy())
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    call = lambda **kw: qsa.qsa_store_kv_tokens_fp8(geom(w), x[:, :2], x[:, 2:4], d["page_table"],  # noqa: E731
                                                    d["seqlens"], *(d[n] for n in POOLS), **kw)
    before = [d[n].clone() for n in POOLS]
    call()
    for n, b in zip(POOLS, before):
        d[n].copy_(b)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        call()
    torch.cuda.synchronize()
    assert all(torch.equal(d[n], b) for n, b in zip(POOLS, before))
    call(stream=side)
    side.synchronize()
    for n, r in zip(POOLS, ref):
        np.testing.assert_array_equal(d[n].cpu().numpy(), r)
    for n, b in zip(POOLS, before):
        d[n].copy_(b)
    d["seqlens"].sub_(1)
    g.replay()
    torch.cuda.synchronize()
    w["seqlens"] = w["seqlens"] - 1
    ref = c8.store(w, x[:, :2].float().cpu().numpy(), x[:, 2:4].float().cpu().numpy())
    for n, r in zip(POOLS, ref):
        np.testing.assert_array_equal(d[n].cpu().numpy(), r)


def test_refused():
    w = c8.geometry(11, 2, 3, 2, 128, 64, 30, 60)
    d, x = c8.on_gpu(w), rows(6, 2, 128, 3)
    def call(k=x[:, :2], v=x[:, 2:4], cu=None, **kw):
        a = dict(d, **kw)
        qsa.qsa_store_kv_tokens_fp8(geom(w), k, v, a["page_table"], a["seqlens"], *(a[n] for n in POOLS), cu_rows=cu)
    call()
    for kw in (dict(k=x[:5, :2]), dict(k=x[:, :1]), dict(k=x[:, :2, :64]), dict(k=x[:, 0:4:2]),
               dict(v=x[:, 2:4].cpu()), dict(cu=torch.zeros(2, dtype=torch.int32, device=DEV)),
               dict(k_exp=d["k_exp"].flatten()[:-1]), dict(v_pool=d["v_pool"][1:])):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(k=x[:, :2].float()), dict(k_exp=d["k_exp"].int()), dict(seqlens=d["seqlens"].long())):
        with pytest.raises(TypeError):
            call(**kw)
    with pytest.raises(qsa.QsaError):
        call(k=torch.empty(6 * 300 + 4, dtype=torch.bfloat16, device=DEV)[4:].as_strided((6, 2, 128), (300, 128, 1)))
    call(k=x[:0, :2], v=x[:0, 2:4], cu=torch.zeros(3, dtype=torch.int32, device=DEV))     # no rows


def test_exponents_of_any_bits_are_read_back():
    """Exponent bytes outside the append's range count as the nearest of it, as they do in attention."""
    for D, P in ((128, 64), (256, 32)):
        w = c8.geometry(12, 3, 40, 2, D, P, 100, 130)
        rng = np.random.default_rng(D)
        for n in ("k_exp", "v_exp"):
            w[n][:] = rng.choice(np.array([0, 1, 94, 95, 127, 191, 192, 254, 255], np.uint8), w[n].shape)
        d = c8.on_gpu(w)
        out = [torch.full((120, 2, D), 3.5, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
        qsa.qsa_load_kv_tokens_fp8(geom(w), d["page_table"], d["seqlens"], *(d[n] for n in POOLS), *out)
        pools = [w["k_pool"], np.clip(w["k_exp"], 95, 191), w["v_pool"], np.clip(w["v_exp"], 95, 191)]
        want = c8.load(w, pools, 120, *(np.full((120, 2, D), 3.5) for _ in "kv"))
        for got, x in zip(out, want):
            np.testing.assert_array_equal(got.double().cpu().numpy(), x)


def test_rejected_rows_taken_back():
    """A step's rows raise the scales of the blocks they go to; the bytes of these blocks, kept before the step
    and written back behind it, leave the cache as if the step had been of the accepted rows alone."""
    w = c8.geometry(13, 4, 6, 2, 128, 64, 30, 200)
    d, x = c8.on_gpu(w), rows(24, 2, 128, 4)
    x[2::6] *= 1000                                     # a draft with large values, later rejected
    k, v = x[:, :2], x[:, 2:4]
    args = lambda lens: (d["page_table"], lens, *(d[n] for n in POOLS))  # noqa: E731
    first, last = d["seqlens"].long() - 6, d["seqlens"].long() - 1
    blocks = torch.stack([first // 16, last // 16], 1)                             # [B, 2], of six rows at most two
    page, at = d["page_table"].long().gather(1, blocks // 4), blocks % 4
    view = lambda n: d[n].view(d[n].shape[0], 2, 4, -1)  # noqa: E731
    kept = [view(n)[page, :, at].clone() for n in POOLS]
    qsa.qsa_store_kv_tokens_fp8(geom(w), k, v, *args(d["seqlens"]))
    for n, x0 in zip(POOLS, kept):
        view(n)[page, :, at] = x0
    two = [t.view(4, 6, 2, 128)[:, :2].reshape(8, 2, 128) for t in (k, v)]         # two of the six accepted
    qsa.qsa_store_kv_tokens_fp8(geom(w, rows_per_req=2), *two, *args(d["seqlens"] - 4))
    w2 = dict(w, rows_per_req=2, seqlens=w["seqlens"] - 4)
    ref = c8.store(w2, *(t.float().cpu().numpy() for t in two))
    for n, r in zip(POOLS, ref):
        np.testing.assert_array_equal(d[n].cpu().numpy(), r, err_msg=n)
