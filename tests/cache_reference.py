"""Plain references of the prologue and of dense attention, on the host: numpy
in 64 bits, except where the operator's definition is a sequence of IEEE fp32
operations (then numpy's fp32, one rounding per operation)."""
import math

import numpy as np
import torch

import oracle

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def host(d):
    """Host copies of a dict's tensors: bf16 as fp32, the rest as they are."""
    return {k: (v.detach().cpu().float() if v.dtype == torch.bfloat16 else v.detach().cpu()).numpy()
            if isinstance(v, torch.Tensor) else v for k, v in d.items()}


def bits(x):
    """bf16 values in fp32 -> their bits."""
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).view(torch.int16).numpy().view(
        np.uint16)


def e4m3(b):
    return torch.from_numpy(np.ascontiguousarray(b)).view(torch.float8_e4m3fn).double().numpy()


def bf16(x):
    """fp32 -> nearest bf16, as fp32."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).float().numpy()


def freqs(rot, theta, scaling="none", factor=1.0, original=0.0, low=1.0, high=4.0):
    """Radians per position of each pair, and the factor on cos and sin."""
    f = [theta ** (-2 * i / rot) for i in range(rot // 2)]
    amp = 1.0
    if scaling == "linear":
        f = [x / factor for x in f]
    elif scaling == "yarn":
        at = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        a, b = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)
        m = [min(max((i - a) / max(b - a, 1e-3), 0), 1) for i in range(rot // 2)]
        f = [x * (1 - t) + x / factor * t for x, t in zip(f, m)]
        amp = 0.1 * math.log(factor) + 1 if factor > 1 else 1.0
    elif scaling == "wavelength":
        m = [min(max((original * x / (2 * math.pi) - low) / (high - low), 0), 1) for x in f]
        f = [x * t + x / factor * (1 - t) for x, t in zip(f, m)]
    return np.array(f), amp


def rope_rows(positions, f, amp):
    a = np.asarray(positions, dtype=np.float64)[:, None] * f
    return np.stack([np.cos(a), np.sin(a)], -1) * amp


def norm_rope(x, weight, cs, rot, interleaved, eps, plus_one):
    """x fp32 [T, H, D] (bf16 values), weight fp32 [D] or None, cs fp32: the bf16
    results as fp32, every operation rounded to fp32 in the header's order."""
    f = np.float32
    y = x.astype(f)
    D = y.shape[-1]
    if weight is not None:
        s = y * y
        while s.shape[-1] > 1:
            s = s[..., 0::2] + s[..., 1::2]
        r = f(1) / np.sqrt(s / f(D) + f(eps))
        w = weight.astype(f)
        if plus_one:
            w = f(1) + w
        y = (y * r) * w
    y = y.copy()
    if rot:
        h = rot // 2
        ia = np.arange(h) * 2 if interleaved else np.arange(h)
        ib = ia + 1 if interleaved else ia + h
        c, s = cs[:, None, :, 0].astype(f), cs[:, None, :, 1].astype(f)
        a, b = y[..., ia], y[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return bf16(y)


def positions(seqlens, R):
    return (seqlens.astype(np.int64)[:, None] - R + np.arange(R)).reshape(-1)


def slots(w):
    """(row, page, slot) of every row of the step that has a slot."""
    P, MB, NP, R = w["page_size"], w["max_blocks"], w["num_pages"], w["rows_per_req"]
    out = []
    for r, pos in enumerate(positions(w["seqlens"], R)):
        if 0 <= pos < MB * P:
            page = w["page_table"][r // R, pos // P]
            if 0 <= page < NP:
                out.append((r, int(page), int(pos % P)))
    return out


def unpack(codes):
    return np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])


def values(codes, sf):
    """e2m1 * e4m3, exact."""
    v = E2M1[unpack(codes)]
    return (v.reshape(*sf.shape, 16) * e4m3(sf)[..., None]).reshape(v.shape)


def load_rows(w, k_out, v_out):
    """k_out, v_out (fp32 [T, Hkv, D]) with the rows that have a slot replaced."""
    for r, page, slot in slots(w):
        for out, codes, sf, scale in ((k_out, w["k_pool"], w["k_sf"], w["k_scale"]),
                                      (v_out, w["v_pool"], w["v_sf"], w["v_scale"])):
            x = values(codes[page, :, slot], sf[page, :, slot]).astype(np.float32)
            out[r] = bf16(x * np.float32(scale))
    return k_out, v_out


def dense(w, window=0, sinks=None, q=None):
    """out, lse and the mean of |V| by the same weights, in 64 bits; w on the host."""
    B, R, Hq, Hkv, D, P, MB, NP = (w[n] for n in ("batch", "rows_per_req", "num_q_heads",
                                                  "num_kv_heads", "head_dim", "page_size",
                                                  "max_blocks", "num_pages"))
    G, cap = Hq // Hkv, MB * P
    q = np.asarray(w["q"] if q is None else q, dtype=np.float64)
    out = np.zeros((B * R, Hq, D))
    lse = np.full((B * R, Hq), -np.inf)
    mag = np.zeros((B * R, Hq, D))
    ks, vs = float(np.float32(w["k_scale"])), float(np.float32(w["v_scale"]))
    sm = float(np.float32(w["sm_scale"]))
    for b in range(B):
        n = [min(max(int(w["seqlens"][b]) - R + 1 + j, 0), cap) for j in range(R)]
        blocks = [i for i in range(-(-n[-1] // P)) if 0 <= w["page_table"][b, i] < NP]
        pages = w["page_table"][b, np.array(blocks, dtype=np.int64)]
        at = (np.array(blocks, dtype=np.int64).reshape(-1, 1) * P + np.arange(P)).reshape(-1)
        for h in range(Hkv):
            k = values(w["k_pool"][pages, h], w["k_sf"][pages, h]).reshape(len(blocks) * P, D) * ks
            v = values(w["v_pool"][pages, h], w["v_sf"][pages, h]).reshape(len(blocks) * P, D) * vs
            for j in range(R):
                see = (at < n[j]) & (at >= (n[j] - window if window else 0))
                hs = slice(h * G, (h + 1) * G)
                z = q[b * R + j, hs] @ k[see].T * sm
                extra = None if sinks is None else np.asarray(sinks, dtype=np.float64)[hs, None]
                every = z if extra is None else np.concatenate([z, extra], -1)
                if every.shape[-1] == 0:
                    continue
                m = every.max(-1, keepdims=True)
                m = np.where(np.isfinite(m), m, 0.0)
                total = np.exp(every - m).sum(-1, keepdims=True)
                with np.errstate(divide="ignore"):
                    lse[b * R + j, hs] = (m + np.log(total))[:, 0]
                if see.any():
                    out[b * R + j, hs] = np.exp(z - m) @ v[see] / total
                    mag[b * R + j, hs] = np.exp(z - m) @ np.abs(v[see]) / total
    return out, lse, mag


def store_rope(w, new, cs, rot, interleaved, eps, plus_one):
    """(rotated queries, pools) after the fused prologue."""
    q = norm_rope(new["q"], new["q_weight"], cs, rot, interleaved, eps, plus_one)
    k = norm_rope(new["k"], new["k_weight"], cs, rot, interleaved, eps, plus_one)
    as_new = {"k_new": bits(k), "v_new": bits(new["v"]), "ik_new": new["ik_new"]}
    return q, k, oracle.store_kv(w, as_new)
