"""Plain references of the 8-bit cache and of packed prompts, on the host in 64 bits."""
import math

import numpy as np
import torch

BLOCK = 16
LEAST, MOST = -32, 64


def codes_of(x):
    """Values (at most 448 in magnitude, or NaN) to e4m3 codes, round to nearest even."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    return torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def values_of(codes):
    return torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn).double().numpy()


def cached(codes, exps):
    """[..., P, D] codes and [..., P / 16] exponents to values."""
    return values_of(codes) * np.repeat(np.exp2(exps.astype(np.float64) - 127), BLOCK, -1)[..., None]


def exponent(x):
    """The exponent of a block's new elements."""
    x = np.abs(x[np.isfinite(x)])
    e = LEAST
    while x.size and x.max() > 448.0 * 2.0**e and e < MOST:
        e += 1
    return e


def rows_of(w, cu, r):
    """(request, position) of row r, or None where it has no slot."""
    if cu is None:
        b, j, n = r // w["rows_per_req"], r % w["rows_per_req"], w["rows_per_req"]
    else:
        owner = [b for b in range(w["batch"]) if cu[b] <= r < cu[b + 1]]
        if not owner:
            return None
        b = owner[0]
        j, n = r - cu[b], cu[b + 1] - cu[b]
    pos = int(w["seqlens"][b]) - n + j
    if pos < 0 or pos >= w["max_blocks"] * w["page_size"]:
        return None
    if not 0 <= w["page_table"][b, pos // w["page_size"]] < w["num_pages"]:
        return None
    return b, pos


def store(w, k, v, cu=None):
    """The pools after the append of k and v (fp32 values of bf16) to those of w."""
    P = w["page_size"]
    pools = [w[n].copy() for n in ("k_pool", "k_exp", "v_pool", "v_exp")]
    blocks = {}
    for r in range(len(k)):
        at = rows_of(w, cu, r)
        if at is not None:
            b, pos = at
            blocks.setdefault((int(w["page_table"][b, pos // P]), pos % P // BLOCK), []).append((r, pos % P))
    for (page, i), rows in blocks.items():
        first = rows[0][1] % BLOCK
        for x, codes, exps in ((k, pools[0], pools[1]), (v, pools[2], pools[3])):
            for h in range(w["num_kv_heads"]):
                new = x[[r for r, _ in rows], h].astype(np.float64)
                e = exponent(new)
                if first:
                    was = min(max(int(exps[page, h, i]) - 127, LEAST), MOST)
                    e = max(e, was)
                    old = slice(i * BLOCK, i * BLOCK + first)
                    codes[page, h, old] = codes_of(values_of(codes[page, h, old]) * 2.0**(was - e))
                with np.errstate(invalid="ignore"):
                    y = np.where(np.isfinite(new), np.clip(new * 2.0**-e, -448, 448), np.nan)
                codes[page, h, [s for _, s in rows]] = codes_of(y)
                exps[page, h, i] = e + 127
    return pools


def load(w, pools, rows, k_out, v_out, cu=None):
    """k_out and v_out with the rows that have a slot replaced by what the cache holds."""
    P = w["page_size"]
    out = [k_out.copy(), v_out.copy()]
    for r in range(rows):
        at = rows_of(w, cu, r)
        if at is None:
            continue
        b, pos = at
        page, slot = w["page_table"][b, pos // P], pos % P
        for o, codes, exps in ((out[0], *pools[:2]), (out[1], *pools[2:])):
            two = 2.0**(exps[page, :, slot // BLOCK].astype(np.float64) - 127)
            o[r] = values_of(codes[page, :, slot]) * two[:, None]
    return out


def axis_of(pairs, layout):
    n, A = sum(pairs), len(pairs)
    if layout == "interleaved":
        return [i % A if i % A and i < A * pairs[i % A] else 0 for i in range(n)]
    return [a for a in range(A) for _ in range(pairs[a])]


def geometry(seed, B, R, Hkv, D, P, lo, hi, G=4, holes=0.0, spare=2):
    """A workload's geometry and an 8-bit cache full of values, on the host."""
    rng = np.random.default_rng(seed)
    MB = -(-max(hi, 1) // P)
    NP = B * MB + spare
    table = rng.permutation(NP)[:B * MB].reshape(B, MB).astype(np.int32)
    table[rng.random(table.shape) < holes] = -1
    w = dict(batch=B, rows_per_req=R, num_q_heads=G * Hkv, num_kv_heads=Hkv, head_dim=D, index_dim=64,
             page_size=P, max_blocks=MB, num_pages=NP, page_table=table,
             seqlens=rng.integers(lo, hi + 1, B).astype(np.int32), sm_scale=1 / math.sqrt(D))
    for n in ("k", "v"):
        x = rng.standard_normal((NP, Hkv, P // BLOCK, BLOCK, D)) * np.exp(0.4 * rng.standard_normal(
            (NP, Hkv, P // BLOCK, BLOCK, 1)))
        top = np.abs(x).max((-1, -2))
        e = np.ceil(np.log2(top / 448))
        w[n + "_pool"] = codes_of(x / np.exp2(e)[..., None, None]).reshape(NP, Hkv, P, D)
        w[n + "_exp"] = (e + 127).astype(np.uint8)
    return w


def on_gpu(w, device="cuda"):
    return {n: torch.from_numpy(np.ascontiguousarray(x)).to(device) if isinstance(x, np.ndarray) else x
            for n, x in w.items()}


# ---------------------------------------------------------------------------
# attention in 64 bits, with a bound of the kernels' error for every output
# ---------------------------------------------------------------------------

def attend(q, k, v, sm, extra=None, exps=None, weight=2.0**-11, alike=False):
    """One KV head's vectors q [G, D] over the tokens k, v [n, D] they see: out, lse and their bounds.

    With p the normalised weights, M the largest logit, A the largest sum_d |q_d K_d| of a token:
      2^-8 |out|                    the output's bf16 (half a step)
      8 weight sqrt(sum p^2 V^2)    the weights' roundings to nearest of up to `weight` each
                                    (Hoeffding: beyond 8 with probability 2 e^-32); rows whose weights
                                    are alike round alike, `alike`: weight sum p |V|
      (2 dz + 2^-17) sum p |V|      logits: D / 16 steps of the matrix instruction and two more
                                    roundings, dz = (D / 16 + 2) 2^-23 A; the exponent's fp32
                                    argument (below 2^7: half a step of 2^-17, twice) and its approximation
      2^-33 max(e^(z - lse) 2^e) sum |V| 2^-e     with fp16 weights (exps: the tokens' exponents of V, 0
                                    without): those below 2^-14 of the base's are subnormal, half a step
                                    of 2^-24; the base lies 2^8 below the largest or lower
    and of lse  2 dz + 2^-16 + 2^-21 |lse|."""
    G, D = q.shape
    if not len(k):
        # (a sink alone: its fp32 products with log2(e) and ln(2), two roundings and two rounded
        # constants of 2^-24 each)
        lse = np.full(G, -np.inf) if extra is None else np.asarray(extra, dtype=np.float64)
        return np.zeros((G, D)), lse, np.zeros((G, D)), 4 * 2.0**-24 * np.abs(lse)
    z = q @ k.T * sm
    top = z.max(-1) if extra is None else np.maximum(z.max(-1), extra)
    total = np.exp(z - top[:, None]).sum(-1)
    if extra is not None:
        total = total + np.exp(extra - top)
    lse = top + np.log(total)
    p, a = np.exp(z - lse[:, None]), np.abs(v)
    out, mag = p @ v, p @ a
    dz = (D / 16 + 2) * 2.0**-23 * (np.abs(q) @ np.abs(k).T).max(-1) * sm
    spread = weight * mag if alike else 8 * weight * np.sqrt(p**2 @ a**2)
    tol = 2.0**-8 * np.abs(out) + spread + (2 * dz + 2.0**-17)[:, None] * mag
    if weight == 2.0**-11:
        two = np.ones(len(k)) if exps is None else np.exp2(exps.astype(np.float64) - 127)
        tol = tol + 2.0**-33 * (p * two).max(-1)[:, None] * (a / two[:, None]).sum(0)
    return out, lse, tol, 2 * dz + 2.0**-16 + 2.0**-21 * np.abs(lse)


def dense(w, window=0, sinks=None, q=None, alike=False):
    """Dense attention over the 8-bit cache of w (on the host): out, lse and their bounds."""
    B, R, Hq, Hkv, D, P, MB, NP = (w[n] for n in ("batch", "rows_per_req", "num_q_heads", "num_kv_heads",
                                                  "head_dim", "page_size", "max_blocks", "num_pages"))
    G, q = Hq // Hkv, np.asarray(w["q"] if q is None else q, dtype=np.float64)
    res = [np.zeros((B * R, Hq, D)), np.zeros((B * R, Hq)), np.zeros((B * R, Hq, D)), np.zeros((B * R, Hq))]
    for b in range(B):
        n = [min(max(int(w["seqlens"][b]) - R + 1 + j, 0), MB * P) for j in range(R)]
        blocks = np.array([i for i in range(-(-n[-1] // P)) if 0 <= w["page_table"][b, i] < NP], dtype=np.int64)
        pages = w["page_table"][b, blocks]
        at = (blocks.reshape(-1, 1) * P + np.arange(P)).reshape(-1)
        for h in range(Hkv):
            ex = [np.clip(w[x][pages, h], 95, 191) for x in ("k_exp", "v_exp")]
            k = cached(w["k_pool"][pages, h], ex[0]).reshape(len(at), D)
            v = cached(w["v_pool"][pages, h], ex[1]).reshape(len(at), D)
            ve = np.repeat(ex[1], BLOCK, -1).reshape(-1)
            hs = slice(h * G, (h + 1) * G)
            for j in range(R):
                see = (at < n[j]) & (at >= (n[j] - window if window else 0))
                extra = None if sinks is None else np.asarray(sinks, dtype=np.float64)[hs]
                got = attend(q[b * R + j, hs], k[see], v[see], float(np.float32(w["sm_scale"])), extra, ve[see],
                             alike=alike)
                for r, x in zip(res, got):
                    r[b * R + j, hs] = x
    return res


def prompt(q, k, v, cu, sm, window=0, sinks=None, alike=False):
    """Packed causal attention q [T, Hq, D], k, v [T, Hkv, D]: out, lse (NaN in rows of no sequence)
    and their bounds: as of attend(), with bf16 weights."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    res = [np.full((T, Hq, D), np.nan), np.full((T, Hq), np.nan), np.zeros((T, Hq, D)), np.zeros((T, Hq))]
    for a, b in zip(cu[:-1], cu[1:]):
        n = b - a
        if n == 0:
            continue
        back = np.arange(n)[:, None] - np.arange(n)
        see = (back >= 0) & ((back < window) if window else True)
        for h in range(Hq):
            kk, vv, qq = k[a:b, h // G], v[a:b, h // G], q[a:b, h]
            z = np.where(see, qq @ kk.T * sm, -np.inf)
            top = z.max(-1) if sinks is None else np.maximum(z.max(-1), sinks[h])
            total = np.exp(z - top[:, None]).sum(-1) + (0 if sinks is None else np.exp(sinks[h] - top))
            lse = top + np.log(total)
            p, mag_v = np.exp(z - lse[:, None]), np.abs(vv)
            out, mag = p @ vv, p @ mag_v
            dz = (D / 16 + 2) * 2.0**-23 * np.where(see, np.abs(qq) @ np.abs(kk).T, 0).max(-1) * sm
            spread = 2.0**-9 * mag * (2 if alike else 1)
            if not alike:     # (Hoeffding where there are many, the sum of all roundings where there are few)
                spread = np.minimum(spread * 2, 8 * 2.0**-9 * np.sqrt(p**2 @ mag_v**2))
            res[0][a:b, h], res[1][a:b, h] = out, lse
            res[2][a:b, h] = 2.0**-8 * np.abs(out) + spread + (2 * dz + 2.0**-17)[:, None] * mag
            res[3][a:b, h] = 2 * dz + 2.0**-16 + 2.0**-21 * np.abs(lse)
    return res


def compare(got, got_lse, ref):
    """Asserts that results (tensors) are within the bounds of a reference's."""
    out, lse, tol, lse_tol = ref
    got, got_lse = got.detach().double().cpu().numpy(), got_lse.detach().double().cpu().numpy()
    err = np.abs(got - out)
    assert (err <= tol).all(), (np.nanmax(err), np.nanmax(err / np.maximum(tol, 1e-300)), np.isnan(err).sum())
    fin = np.isfinite(lse)
    np.testing.assert_array_equal(np.isneginf(got_lse), ~fin)
    e = np.abs(got_lse[fin] - lse[fin])
    assert (e <= lse_tol[fin]).all(), (e.max(), (e / lse_tol[fin]).max())
