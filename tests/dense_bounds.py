"""Dense attention in 64 bits with a bound of the kernels' error for every output.

The bound per output element, with p the row's normalised weights, M its largest
logit, A the largest sum_d |q_d K_d| of a token (scales included):
  2^-8 |out|                 the output's bf16 (half a step)
  8 2^-11 sqrt(sum p^2 V^2)  the weights' fp16: roundings to nearest of up to 2^-11 each
                             (Hoeffding: beyond 8 with probability 2 e^-32); rows whose
                             weights are alike round alike, `alike`: 2^-11 sum p |V|
  (2 dz + 2^-18) sum p |V|   logits: D / 16 steps of the matrix instruction and two more
                             roundings, dz = (D / 16 + 2) 2^-23 A; the exponent's fp32 argument
                             (up to 2^6: 2^-19) and its approximation
  2^-33 e^(M - lse) sum |V|  weights below 2^-14 of the base's are subnormal, half a step of
                             2^-24; the base lies 2^8 below the largest logit or lower
and of lse  2 dz + 2^-17 + 2^-21 |lse|.
"""
import numpy as np

import cache_reference as cr


def dense(w, window=0, sinks=None, q=None, alike=False):
    """out, lse and their bounds, in 64 bits; w on the host."""
    B, R, Hq, Hkv, D, P, MB, NP = (w[n] for n in ("batch", "rows_per_req", "num_q_heads",
                                                  "num_kv_heads", "head_dim", "page_size",
                                                  "max_blocks", "num_pages"))
    G, cap = Hq // Hkv, MB * P
    q = np.asarray(w["q"] if q is None else q, dtype=np.float64)
    out, tol = np.zeros((B * R, Hq, D)), np.zeros((B * R, Hq, D))
    lse, lse_tol = np.full((B * R, Hq), -np.inf), np.zeros((B * R, Hq))
    ks, vs, sm = (float(np.float32(w[n])) for n in ("k_scale", "v_scale", "sm_scale"))
    for b in range(B):
        n = [min(max(int(w["seqlens"][b]) - R + 1 + j, 0), cap) for j in range(R)]
        blocks = np.array([i for i in range(-(-n[-1] // P)) if 0 <= w["page_table"][b, i] < NP],
                          dtype=np.int64)
        pages = w["page_table"][b, blocks]
        at = (blocks.reshape(-1, 1) * P + np.arange(P)).reshape(-1)
        for h in range(Hkv):
            k = cr.values(w["k_pool"][pages, h], w["k_sf"][pages, h]).reshape(len(at), D) * ks
            v = cr.values(w["v_pool"][pages, h], w["v_sf"][pages, h]).reshape(len(at), D) * vs
            for j in range(R):
                hs, r = slice(h * G, (h + 1) * G), b * R + j
                see = (at < n[j]) & (at >= (n[j] - window if window else 0))
                extra = None if sinks is None else np.asarray(sinks, dtype=np.float64)[hs]
                if not see.any():
                    if extra is not None:
                        lse[r, hs] = extra
                    continue
                kk, vv = k[see], np.abs(v[see])
                z = q[r, hs] @ kk.T * sm
                top = z.max(-1)
                both = top if extra is None else np.maximum(top, extra)
                total = np.exp(z - both[:, None]).sum(-1)
                if extra is not None:
                    total = total + np.exp(extra - both)
                lse[r, hs] = both + np.log(total)
                p = np.exp(z - lse[r, hs][:, None])
                out[r, hs] = p @ v[see]
                mag = p @ vv
                dz = (D / 16 + 2) * 2.0**-23 * (np.abs(q[r, hs]) @ np.abs(kk).T).max(-1) * sm
                weights = 2.0**-11 * mag if alike else 8 * 2.0**-11 * np.sqrt(p**2 @ vv**2)
                tol[r, hs] = (2.0**-8 * np.abs(out[r, hs]) + weights
                              + (2 * dz + 2.0**-18)[:, None] * mag
                              + 2.0**-33 * np.exp(top - lse[r, hs])[:, None] * vv.sum(0))
                lse_tol[r, hs] = 2 * dz + 2.0**-17 + 2.0**-21 * np.abs(lse[r, hs])
    return out, lse, tol, lse_tol


def compare(got, got_lse, ref):
    """Asserts that results (numpy) are within the bounds of `ref`, what dense() gave."""
    out, lse, tol, lse_tol = ref
    err = np.abs(np.asarray(got, dtype=np.float64) - out)
    assert (err <= tol).all(), (np.nanmax(err), np.nanmax(err / np.maximum(tol, 1e-300)), np.isnan(err).sum())
    fin = np.isfinite(lse)
    np.testing.assert_array_equal(np.isneginf(got_lse), ~fin)
    e = np.abs(np.asarray(got_lse, dtype=np.float64)[fin] - lse[fin])
    assert (e <= lse_tol[fin]).all(), (e.max(), (e / lse_tol[fin]).max())
