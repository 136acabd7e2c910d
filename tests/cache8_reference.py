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
