"""Measured cases of the cache prologue (rotation rows, head norms with the
rotation, the paged NVFP4 append and its read-back) and of dense attention over
the NVFP4 paged cache, in their plain form (elementary torch operations) and
through the library's entry points.

Every case has the geometry fields of ``qsa_geom_t``: B requests of R new rows,
Hq query and Hkv KV heads of D dims, pages of P tokens.  Row j of request b is
the token at position L_b - R + j and sees L_b - R + 1 + j tokens.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _rope(name, B, R, rot, L, scaling, **kw):
    return dict(name=name, op="rope", B=B, R=R, rot=rot, L=L, scaling=scaling, **kw)


def _qk(name, B, R, Hq, Hkv, D, rot, inter, **kw):
    return dict(name=name, op="qk", B=B, R=R, Hq=Hq, Hkv=Hkv, D=D, rot=rot, inter=inter, **kw)


def _append(name, B, R, Hq, Hkv, D, P, rot, inter, L, **kw):
    return dict(name=name, op="append", B=B, R=R, Hq=Hq, Hkv=Hkv, D=D, P=P, rot=rot, inter=inter,
                L=L, **kw)


def _dense(name, B, R, Hq, Hkv, D, P, lo, hi, window=0, sinks=False, holes=False, **kw):
    return dict(name=name, op="dense", B=B, R=R, Hq=Hq, Hkv=Hkv, D=D, P=P, lo=lo, hi=hi,
                window=window, sinks=sinks, holes=holes, **kw)


def listed():
    return [
        # the angles of one speculative step of a serving batch, far into long contexts
        _rope("rope rows, verify step", 48, 4, 128, 131072, "yarn"),
        # the angles of four context chunks, rotating a quarter of a wide head
        _rope("rope rows, context", 4, 4096, 64, 1 << 20, "wavelength"),
        # one decode step's queries and keys: latency
        _qk("head norms, decode", 8, 1, 32, 4, 128, 128, False),
        # two context chunks at head_dim 256, a quarter of the head rotated, interleaved pairs
        _qk("head norms, context", 2, 4096, 24, 2, 256, 64, True),
        # the prologue of a speculative step, and its rows read back
        _append("append, verify step", 48, 4, 32, 4, 128, 64, 128, False, 32768),
        # the prologue of ragged context chunks at head_dim 256, and their rows read back
        _append("append, context", 4, 2047, 24, 2, 256, 32, 64, True, 16384),
        # a single request's decode row: latency
        _dense("dense, tiny decode", 1, 1, 8, 1, 128, 64, 4096, 4096),
        # a decode batch of mixed lengths, some pages missing
        _dense("dense, batched decode", 8, 1, 32, 4, 128, 64, 9000, 32768, holes=True),
        # few requests with long contexts
        _dense("dense, long decode", 4, 1, 32, 4, 128, 64, 131072, 131072),
        # a speculative step at head_dim 256 on a sliding-window layer with sinks
        _dense("dense, windowed verify", 32, 4, 24, 2, 256, 32, 8192, 16384, window=4096, sinks=True),
        # a short odd context chunk at head_dim 256 behind a cached prefix
        _dense("dense, odd context", 1, 77, 24, 2, 256, 64, 8101, 8101),
        # the large one: context chunks of two requests behind long prefixes
        _dense("dense, context", 2, 1024, 32, 4, 128, 64, 30000, 32768),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "qk", "append", "dense", "dense", "dense"])
    D = rng.choice([128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 3, 4, 7, 8, 12, 16])
    Hq = Hkv * G
    P = rng.choice([64, 128] if D == 128 else [32, 64])
    rot = 16 * rng.randint(1, D // 16)
    inter = rng.random() < 0.5
    if op == "rope":
        B = _log(rng, 1, 64)
        R = _log(rng, 1, max(1, min(4096, 16384 // B)))
        return {"op": "rope", "B": B, "R": R, "rot": rot, "L": _log(rng, max(R, 64), 1 << 20),
                "scaling": rng.choice(["none", "linear", "yarn", "wavelength"])}
    if op == "qk":
        B = _log(rng, 1, 64)
        R = _log(rng, 1, max(1, min(4096, 200000 // (B * (Hq + Hkv)))))
        return {"op": "qk", "B": B, "R": R, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot, "inter": inter}
    if op == "append":
        B = _log(rng, 1, 64)
        R = _log(rng, 1, max(1, min(4096, 150000 // (B * (Hq + 2 * Hkv)))))
        return {"op": "append", "B": B, "R": R, "Hq": Hq, "Hkv": Hkv, "D": D, "P": P, "rot": rot,
                "inter": inter, "L": _log(rng, max(R, 64), max(R + 64, 1 << 15))}
    R = rng.choice([1, 1, 2, 4, 5, 8, _log(rng, 9, 1024)])
    # at most the large case's products and the long case's cached values
    B = _log(rng, 1, max(1, min(48, (1 << 38) // (R * Hq * D * (2 * R + 64)))))
    top = max(2 * R + 64, min(131072, (1 << 38) // (B * R * Hq * D), (1 << 28) // (B * Hkv * D)))
    hi = _log(rng, R, top)
    lo = max(R, int(hi * rng.uniform(0.3, 1.0)))
    window = rng.choice([0, 0, _log(rng, 1, max(2, hi))])
    return {"op": "dense", "B": B, "R": R, "Hq": Hq, "Hkv": Hkv, "D": D, "P": P, "lo": lo, "hi": hi,
            "window": window, "sinks": rng.random() < 0.4, "holes": rng.random() < 0.3}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

THETA = 1.0e6
FACTOR = 8.0
ORIGINAL = 16384
LOW, HIGH = 1.0, 4.0            # wavelength bands, in rotations over the original context
FAST, SLOW = 32.0, 1.0          # yarn ramp, in rotations over the original context
EPS = 1e-6


def _freqs(rot, scaling):
    """Scaled frequencies (radians per position) and the factor on cos and sin, in 64 bits."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    f = THETA ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / FACTOR, 1.0
    if scaling == "yarn":
        dim = lambda turns: rot * math.log(ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(THETA))  # noqa: E731
        lo, hi = max(math.floor(dim(FAST)), 0), min(math.ceil(dim(SLOW)), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f * (1 - ramp) + f / FACTOR * ramp, 0.1 * math.log(FACTOR) + 1.0
    if scaling == "wavelength":
        turns = ORIGINAL * f / (2 * math.pi)
        mix = ((turns - LOW) / (HIGH - LOW)).clamp(0, 1)
        return f * mix + f / FACTOR * (1 - mix), 1.0
    return f, 1.0


def _lengths(case, gen, lo, hi):
    """Lengths in [lo, hi] that the case's numbers and the seed give."""
    return torch.randint(lo, hi + 1, (case["B"],), generator=gen, device=DEV).to(torch.int32)


def _encode(x):
    """Blocks of 16 values to e2m1 codes (packed) and e4m3 scales, for a tensor scale of one."""
    b = x.reshape(*x.shape[:-1], -1, 16)
    sf = (b.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = sf.float().unsqueeze(-1)
    y = torch.where(s > 0, b / torch.where(s > 0, s, 1.0), 0.0)
    code = torch.bucketize(y.abs(), torch.tensor(MIDS, device=DEV)).to(torch.uint8)
    code = (code | ((y < 0) & (code > 0)).to(torch.uint8) << 3).reshape(x.shape)
    return code[..., 0::2] | code[..., 1::2] << 4, sf.view(torch.uint8)


def _pages(case, gen, L_max):
    """A page table over a pool with spare pages, in no order."""
    B, P = case["B"], case["P"]
    mb = -(-L_max // P)
    n = B * mb + 3
    perm = torch.randperm(n, generator=gen, device=DEV)[: B * mb]
    return perm.to(torch.int32).reshape(B, mb).contiguous(), mb, n


def _pool(n, Hkv, P, D, gen):
    code = torch.empty(n, Hkv, P, D // 2, dtype=torch.uint8, device=DEV)
    sf = torch.empty(n, Hkv, P, D // 16, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (Hkv * P * D))
    for i in range(0, n, step):
        x = torch.randn(min(step, n - i), Hkv, P, D, generator=gen, device=DEV)
        code[i:i + step], sf[i:i + step] = _encode(x * 16.0)
    return code, sf


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)
    B, R, op = case["B"], case["R"], case["op"]
    T = B * R
    s["mids"] = torch.tensor(MIDS, device=DEV)
    s["mags"] = torch.tensor(E2M1 + tuple(-m for m in E2M1), device=DEV)
    s["six"] = torch.tensor(6.0, device=DEV)
    if op == "rope":
        s["seqlens"] = _lengths(case, gen, max(R, case["L"] // 2), case["L"])
        s["freqs"], s["amp"] = _freqs(case["rot"], case["scaling"])
        s["cs"] = torch.empty(T, case["rot"] // 2, 2, device=DEV)
    else:
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if op in ("qk", "append"):
        # the rows of one projection: queries, keys and values behind one another
        wide = torch.randn(T, (Hq + 2 * Hkv) * D, generator=gen, device=DEV) * 1.5
        s["qkv"] = wide.to(torch.bfloat16)
        s["wq"] = (1 + 0.2 * torch.randn(D, generator=gen, device=DEV)).to(torch.bfloat16)
        s["wk"] = (1 + 0.2 * torch.randn(D, generator=gen, device=DEV)).to(torch.bfloat16)
        s["seqlens"] = _lengths(case, gen, max(R, case.get("L", 4096) // 2), max(R, case.get("L", 4096)))
        f, _ = _freqs(case["rot"], "none")
        at = s["seqlens"].double()[:, None] - R + torch.arange(R, device=DEV)
        a = at.reshape(T, 1) * f
        s["cs"] = torch.stack([a.cos(), a.sin()], -1).float().contiguous()
        s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
        s["k_out"] = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=DEV)
    if op == "append":
        s["page_table"], s["MB"], s["NP"] = _pages(case, gen, max(R, case["L"]))
        s["ik"] = torch.randint(-127, 128, (T, 64), generator=gen, device=DEV).to(torch.int8)
        s["pools"] = [torch.zeros(s["NP"], Hkv, case["P"], D // d, dtype=torch.uint8, device=DEV)
                      for d in (2, 16, 2, 16)]
        s["ik_pool"] = torch.zeros(s["NP"], case["P"], 64, dtype=torch.int8, device=DEV)
        s["v_out"] = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=DEV)
        # as a calibration gives them: about a tensor's largest magnitude / (6 * 448), in 32 bits
        s["scales"] = torch.tensor([0.00213, 0.00277], device=DEV)
        s["k_scale"], s["v_scale"] = s["scales"].tolist()
    if op == "dense":
        s["seqlens"] = _lengths(case, gen, case["lo"], case["hi"])
        s["page_table"], s["MB"], s["NP"] = _pages(case, gen, case["hi"])
        if case["holes"]:
            gone = torch.rand(s["page_table"].shape, generator=gen, device=DEV) < 0.05
            s["page_table"] = torch.where(gone, -1, s["page_table"]).contiguous()
        k, ks = _pool(s["NP"], Hkv, case["P"], D, gen)
        v, vs = _pool(s["NP"], Hkv, case["P"], D, gen)
        s["pools"] = [k, ks, v, vs]
        s["k_scale"], s["v_scale"], s["sm_scale"] = 1 / 16.0, 1 / 16.0, 1 / math.sqrt(D)
        s["scales"] = torch.tensor([s["k_scale"], s["v_scale"]], device=DEV)
        # heads look about them or at few tokens: logits of standard deviation 0.5 to 2
        sharp = torch.linspace(0.5, 2.0, Hq, device=DEV)[:, None]
        s["q"] = (torch.randn(T, Hq, D, generator=gen, device=DEV) * sharp).to(torch.bfloat16)
        s["sink"] = torch.randn(Hq, generator=gen, device=DEV) + 2.0 if case["sinks"] else None
        s["out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(T, Hq, device=DEV)
    if op in ("rope", "qk"):
        s["MB"] = s["NP"] = 1
    if own:
        s["keeps"] = _own_keeps(s)     # the geometry, plan and workspace that a program keeps
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plain_rope(s):
    at = s["seqlens"].double()[:, None] - s["R"] + torch.arange(s["R"], device=DEV)
    a = at.reshape(-1, 1) * s["freqs"]
    return (torch.stack([a.cos(), a.sin()], -1) * s["amp"]).float()


def _plain_norm_rope(x, w, cs, rot, inter):
    """Norm of each head by its weight, then the rotation of its first `rot` dims, in 32 bits."""
    x = x.float()
    sq = x * x
    while sq.shape[-1] > 1:          # neighbours first
        sq = sq[..., 0::2] + sq[..., 1::2]
    y = (x * (1.0 / torch.sqrt(sq / x.shape[-1] + EPS))) * w.float()
    c, n = cs[:, None, :, 0], cs[:, None, :, 1]
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if inter else (y[..., : rot // 2], y[..., rot // 2: rot])
    a, b = a * c - b * n, b * c + a * n
    turned = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([turned, y[..., rot:]], -1).to(torch.bfloat16)


def _heads(s):
    T, Hq, Hkv, D = s["B"] * s["R"], s["Hq"], s["Hkv"], s["D"]
    x = s["qkv"].view(T, Hq + 2 * Hkv, D)
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def _plain_quantise(x, scale, s):
    """Codes (one to a byte) and e4m3 scales of blocks of 16, in 32 bits, each operation rounded."""
    b = x.float().reshape(*x.shape[:-1], -1, 16)
    sf = (b.abs().amax(-1) / s["six"] / scale).clamp(max=448.0).to(torch.float8_e4m3fn)
    den = (sf.float() * scale).unsqueeze(-1)
    y = torch.where(den > 0, b / torch.where(den > 0, den, 1.0), 0.0)
    mag, mids = y.abs(), s["mids"]
    # nearest, ties to the even code: up at the borders below an even code
    code = torch.bucketize(mag, mids) + ((mag == mids[1]) | (mag == mids[3]) | (mag == mids[5])).long()
    code = code | ((y < 0) & (code > 0)).long() << 3
    return code.reshape(x.shape), sf


def _values(codes, sf, scale, s):
    """What codes (one to a byte) and e4m3 scales stand for, in 32 bits."""
    v = s["mags"][codes.long()].reshape(*sf.shape, 16) * sf.float().unsqueeze(-1)
    return (v * scale).reshape(codes.shape)


def _unpack(packed):
    return torch.stack([packed & 15, packed >> 4], -1).flatten(-2)


def _plain_append(s):
    q, k, v = _heads(s)
    q = _plain_norm_rope(q, s["wq"], s["cs"], s["rot"], s["inter"])
    k = _plain_norm_rope(k, s["wk"], s["cs"], s["rot"], s["inter"])
    R, P = s["R"], s["P"]
    at = (s["seqlens"].long()[:, None] - R + torch.arange(R, device=DEV)).reshape(-1)
    of = torch.arange(s["B"], device=DEV).repeat_interleave(R)
    page, slot = s["page_table"][of, at // P].long(), at % P
    back = []
    for x, scale, codes, scales in ((k, s["scales"][0], *s["pools"][:2]), (v, s["scales"][1], *s["pools"][2:])):
        c, sf = _plain_quantise(x, scale, s)
        codes[page, :, slot] = (c[..., 0::2] | c[..., 1::2] << 4).to(torch.uint8)
        scales[page, :, slot] = sf.view(torch.uint8)
        back.append(_values(_unpack(codes[page, :, slot]), scales[page, :, slot].view(torch.float8_e4m3fn),
                            scale, s).to(torch.bfloat16))
    s["ik_pool"][page, slot] = s["ik"]
    return {"q": q, "k": back[0], "v": back[1], "ik": s["ik_pool"]}


def _plain_dense(s):
    B, R, Hq, Hkv, D, P = (s[n] for n in ("B", "R", "Hq", "Hkv", "D", "P"))
    G, cap = Hq // Hkv, s["MB"] * P
    page = s["page_table"].long()
    live = (page >= 0) & (page < s["NP"])
    page = torch.where(live, page, 0)

    def tokens(codes, sf, scale):     # [B, Hkv, cap, D]
        x = _values(_unpack(codes[page]), sf[page].view(torch.float8_e4m3fn), scale, s)
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, cap, D)

    at = torch.arange(cap, device=DEV)
    n = s["seqlens"].long()[:, None] - R + 1 + torch.arange(R, device=DEV)               # [B, R]
    see = (at < n[..., None]) & live.repeat_interleave(P, 1)[:, None]
    if s["window"]:
        see &= at >= n[..., None] - s["window"]
    q = s["q"].float().view(B, R, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, R * G, D)
    z = torch.matmul(q, tokens(s["pools"][0], s["pools"][1], s["scales"][0]).transpose(-1, -2)) * s["sm_scale"]
    z = z.view(B, Hkv, R, G, cap).masked_fill_(~see[:, None, :, None], -math.inf)
    top = z.amax(-1)
    sink = None if s["sink"] is None else s["sink"].view(1, Hkv, 1, G)
    top = top if sink is None else torch.maximum(top, sink)
    base = torch.where(top == -math.inf, 0.0, top)
    p = z.sub_(base[..., None]).exp_()
    total = p.sum(-1)
    total = total if sink is None else total + (sink - base).exp()
    o = torch.matmul(p.view(B, Hkv, R * G, cap), tokens(s["pools"][2], s["pools"][3], s["scales"][1]))
    o = o.view(B, Hkv, R, G, D) / torch.where(total > 0, total, 1.0)[..., None]
    lse = base + total.log()
    return {"out": o.permute(0, 2, 1, 3, 4).reshape(B * R, Hq, D).to(torch.bfloat16),
            "lse": lse.permute(0, 2, 1, 3).reshape(B * R, Hq)}


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _own_keeps(s):
    """What a program keeps from call to call: the geometry, the rotation's plan and the workspace."""
    import nvfp4_block_sparse_gb300 as qsa
    k = {"qsa": qsa, "geom": qsa.make_geom(
        batch=s["B"], rows_per_req=s["R"], num_q_heads=s.get("Hq", 1), num_kv_heads=s.get("Hkv", 1),
        head_dim=s.get("D", 256), index_dim=64, page_size=s.get("P", 64), max_blocks=s["MB"],
        num_pages=s["NP"])}
    if s["op"] == "rope":
        more = {"linear": dict(factor=FACTOR),
                "yarn": dict(factor=FACTOR, original_context=ORIGINAL, beta_fast=FAST, beta_slow=SLOW),
                "wavelength": dict(factor=FACTOR, original_context=ORIGINAL, low_freq=LOW, high_freq=HIGH)}
        k["rope"] = qsa.make_rope(rotary_dim=s["rot"], theta=THETA, scaling=s["scaling"],
                                  **more.get(s["scaling"], {}))
    elif s["op"] in ("qk", "append"):
        k["norm"] = qsa.make_norm_rope(rotary_dim=s["rot"], interleaved=s["inter"], eps=EPS)
    else:
        n = qsa.qsa_dense_attention_workspace_bytes(k["geom"])
        k["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        qsa.qsa_workspace_init(k["workspace"])
    return k


def _own_run(s):
    k, op = s["keeps"], s["op"]
    qsa, g = k["qsa"], k["geom"]
    if op == "rope":
        qsa.qsa_rope_rows(g, k["rope"], s["seqlens"], s["cs"])
        return {"cs": s["cs"]}
    if op == "dense":
        qsa.qsa_dense_attention(g, s["q"], *s["pools"], s["k_scale"], s["v_scale"], s["sm_scale"],
                                s["page_table"], s["seqlens"], s["out"], s["lse"], k["workspace"],
                                window=s["window"], sinks=s["sink"])
        return {"out": s["out"], "lse": s["lse"]}
    q, kn, v = _heads(s)
    if op == "qk":
        qsa.qsa_qk_norm_rope(g, k["norm"], q, kn, s["wq"], s["wk"], s["cs"], s["q_out"], s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    qsa.qsa_store_kv_tokens_rope(g, k["norm"], q, kn, v, s["ik"], s["wq"], s["wk"], s["cs"],
                                 s["k_scale"], s["v_scale"], s["page_table"], s["seqlens"],
                                 s["q_out"], *s["pools"], s["ik_pool"])
    qsa.qsa_load_kv_tokens(g, s["page_table"], s["seqlens"], *s["pools"], s["k_scale"], s["v_scale"],
                           s["k_out"], s["v_out"])
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"], "ik": s["ik_pool"]}


def run(state):
    if own:
        return _own_run(state)
    op = state["op"]
    if op == "rope":
        return {"cs": _plain_rope(state)}
    if op == "qk":
        q, k, _ = _heads(state)
        return {"q": _plain_norm_rope(q, state["wq"], state["cs"], state["rot"], state["inter"]),
                "k": _plain_norm_rope(k, state["wk"], state["cs"], state["rot"], state["inter"])}
    return _plain_append(state) if op == "append" else _plain_dense(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    B, R, op = case["B"], case["R"], case["op"]
    T = B * R
    if op == "rope":
        return {"bytes": 4 * B + T * case["rot"] * 4, "flops": T * case["rot"] * 10}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    turn = T * case["rot"] * 4 if op != "dense" else 0
    if op == "qk":
        n = T * (Hq + Hkv) * D
        return {"bytes": 4 * n + turn, "flops": 8 * n}
    if op == "append":
        # queries in and out; keys and values in, packed, unpacked and out; the index keys
        n = T * Hkv * D
        return {"bytes": 4 * T * Hq * D + turn + 2 * n * (2 + 2 * 9 / 16 + 2) + 2 * T * 64,
                "flops": 8 * T * (Hq + 2 * Hkv) * D}
    L = (case["lo"] + case["hi"]) / 2
    w = case["window"]
    each = min(L, w) if w else L - (R - 1) / 2            # tokens that a row sees
    read = min(L, w + R - 1) if w else L                  # tokens that a request's rows see together
    if case["holes"]:
        each, read = 0.95 * each, 0.95 * read
    return {"bytes": B * Hkv * read * D * 2 * 9 / 16 + T * Hq * (4 * D + 4), "flops": 4 * D * T * Hq * each}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_turned(x, weight, s):
    x = x.double()
    T, H, D = x.shape
    y = x / ((x ** 2).mean(-1, keepdim=True) + EPS).sqrt() * weight.double()
    h = s["rot"] // 2
    first = torch.arange(h, device=DEV) * (2 if s["inter"] else 1)
    second = first + (1 if s["inter"] else h)
    z = torch.view_as_complex(torch.stack([y[..., first], y[..., second]], -1)) * torch.view_as_complex(
        s["cs"].double())[:, None]
    y = y.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_cached(x, scale):
    """The value that each element of a block of 16 has in the cache."""
    b = x.unflatten(-1, (-1, 16))
    sf = (b.abs().amax(-1, keepdim=True) / 6 / scale).float().clamp(max=448).to(torch.float8_e4m3fn).double()
    grid = torch.tensor([-m for m in E2M1[:0:-1]] + list(E2M1), dtype=torch.float64, device=DEV)
    pos = torch.where(sf > 0, b / (sf * scale).clamp(min=1e-300), 0.0).clamp(-6, 6)
    up = torch.searchsorted(grid, pos.contiguous()).clamp(1, grid.numel() - 1)
    lower, upper = grid[up - 1], grid[up]
    return (torch.where(pos - lower <= upper - pos, lower, upper) * sf * scale).flatten(-2)


def _exact_dense(s):
    B, R, Hq, Hkv, D, P = (s[n] for n in ("B", "R", "Hq", "Hkv", "D", "P"))
    G = Hq // Hkv
    out = torch.zeros(B * R, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B * R, Hq), -math.inf, dtype=torch.float64, device=DEV)
    grid = torch.tensor(E2M1 + tuple(-m for m in E2M1), dtype=torch.float64, device=DEV)
    for b in range(B):
        L = int(s["seqlens"][b])
        blocks = torch.arange(-(-L // P), device=DEV)
        pages = s["page_table"][b, blocks].long()
        keep = pages >= 0
        blocks, pages = blocks[keep], pages[keep]
        where = (blocks[:, None] * P + torch.arange(P, device=DEV)).reshape(-1)
        for h in range(Hkv):
            kv = []
            for i, scale in ((0, s["k_scale"]), (2, s["v_scale"])):
                c = s["pools"][i][pages, h]
                e = torch.empty(*c.shape[:-1], D, dtype=torch.float64, device=DEV)
                e[..., 0::2], e[..., 1::2] = grid[(c % 16).long()], grid[(c // 16).long()]
                f = s["pools"][i + 1][pages, h].view(torch.float8_e4m3fn).double() * scale
                kv.append((e * f.repeat_interleave(16, -1)).reshape(-1, D))
            for j in range(R):
                n = L - R + 1 + j
                m = (where < n) & ((where >= n - s["window"]) if s["window"] else (where >= 0))
                heads = slice(h * G, (h + 1) * G)
                z = s["q"][b * R + j, heads].double() @ kv[0].T * s["sm_scale"]
                z[:, ~m] = -math.inf
                if s["sink"] is not None:
                    z = torch.cat([z, s["sink"][heads].double()[:, None]], -1)
                l = torch.logsumexp(z, -1)
                p = torch.exp(z - l[:, None]).nan_to_num(0.0)[:, : where.numel()]
                out[b * R + j, heads], lse[b * R + j, heads] = p @ kv[1], l
    return {"out": out, "lse": lse}


def exact(case, seed):
    op = case["op"]
    if op == "dense":
        # a row at a time in 64 bits: within 20 seconds up to this many products and rows
        if case["B"] * case["R"] * case["Hq"] * case["D"] * case["hi"] > 1e12:
            return None
        if case["B"] * case["R"] * case["Hkv"] > 20000:
            return None
        return _exact_dense(prepare(case, seed))
    s = prepare(case, seed)
    if op == "rope":
        pos = (s["seqlens"].double()[:, None] - s["R"] + torch.arange(s["R"], device=DEV)).flatten()
        turn = torch.polar(torch.full_like(pos, s["amp"])[:, None], torch.outer(pos, s["freqs"]))
        return {"cs": torch.view_as_real(turn)}
    q, k, v = _heads(s)
    q, k = _exact_turned(q, s["wq"], s), _exact_turned(k, s["wk"], s)
    if op == "qk":
        return {"q": q, "k": k}
    return {"q": q, "k": _exact_cached(k.to(torch.bfloat16).double(), s["k_scale"]),
            "v": _exact_cached(v.double(), s["v_scale"]), "ik": None}
