"""Measured cases of rotation rows with several position axes, the 8-bit paged
cache (append and read-back), dense attention over that cache, and attention
over whole packed prompts, in their plain form (elementary torch operations)
and through the library's entry points.

A block of the 8-bit cache is 16 tokens of one KV head: e4m3 codes and one
power of two, stored as its exponent plus 127.
"""
import math

import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16
F8 = torch.float8_e4m3fn
BLOCK = 16                   # tokens per scale
TOP = 448.0                  # largest e4m3 value
E_MIN, E_MAX = -32, 64       # exponents of the scales


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _axes(name, T, pairs, layout, at, scaling="none"):
    return dict(name=name, op="axes", T=T, pairs=pairs, layout=layout, at=at, scaling=scaling)


def _cache(name, B, lo, hi, Hkv, D, P, before, packed):
    return dict(name=name, op="cache", B=B, lo=lo, hi=hi, Hkv=Hkv, D=D, P=P, before=before, packed=packed)


def _dense(name, B, R, Hq, Hkv, D, P, lo, hi, window=0, sinks=False, holes=False):
    return dict(name=name, op="dense", B=B, R=R, Hq=Hq, Hkv=Hkv, D=D, P=P, lo=lo, hi=hi, window=window,
                sinks=sinks, holes=holes)


def _prompt(name, B, lo, hi, Hq, Hkv, D, window=0, sinks=False, spare=0):
    return dict(name=name, op="prompt", B=B, lo=lo, hi=hi, Hq=Hq, Hkv=Hkv, D=D, window=window, sinks=sinks,
                spare=spare)


def listed():
    return [
        # the angles of a decode batch of image conversations, axes interleaved: latency
        _axes("axes rows: decode", 64, "24,20,20", "interleaved", 131072),
        # the angles of packed prompts with images, a section of the head per axis
        _axes("axes rows: prompts", 16384, "16,24,24", "sections", 32768),
        # a speculative step's rows appended behind partly filled blocks, and read back
        _cache("cache: verify step", 48, 4, 4, 4, 128, 64, 32768, False),
        # packed prompts of different lengths written behind short prefixes, and read back
        _cache("cache: prompts", 6, 700, 2047, 2, 256, 32, 300, True),
        # a single request's decode row: latency
        _dense("dense: tiny decode", 1, 1, 8, 1, 128, 64, 4096, 4096),
        # a decode batch of mixed lengths, some pages missing
        _dense("dense: batched decode", 8, 1, 32, 4, 128, 64, 9000, 32768, holes=True),
        # a speculative step at head_dim 256 on a sliding-window layer with sinks
        _dense("dense: windowed verify", 32, 4, 24, 2, 256, 32, 8192, 16384, window=4096, sinks=True),
        # context chunks of two requests behind long prefixes
        _dense("dense: context", 2, 512, 32, 4, 128, 64, 14000, 16384),
        # one short prompt: latency
        _prompt("prompt: short", 1, 77, 77, 8, 1, 128),
        # packed prompts of odd lengths at head_dim 256, rows to spare behind the last
        _prompt("prompt: ragged", 6, 100, 2047, 24, 2, 256, spare=50),
        # packed prompts on a sliding-window layer with sinks
        _prompt("prompt: windowed", 4, 3000, 4096, 32, 4, 128, window=1024, sinks=True),
        # the large one: a long prompt
        _prompt("prompt: long", 1, 8192, 8192, 32, 4, 128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["axes", "cache", "dense", "dense", "prompt", "prompt"])
    if op == "axes":
        A, half = rng.choice([2, 3, 4]), 8 * rng.randint(2, 16)
        layout = rng.choice(["sections", "interleaved", "spectra"])
        share = half // A
        if layout == "interleaved":     # the first axis has what the others leave
            rest = [rng.randint(max(1, share // 2), share) for _ in range(A - 1)]
        else:
            rest = [rng.randint(1, share) for _ in range(A - 1)]
        pairs = ",".join(str(n) for n in [half - sum(rest)] + rest)
        return {"op": "axes", "T": _log(rng, 1, 16384), "pairs": pairs, "layout": layout,
                "at": _log(rng, 64, 1 << 20), "scaling": rng.choice(["none", "linear", "yarn", "wavelength"])}
    D = rng.choice([128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 3, 4, 7, 8, 12, 16])
    P = rng.choice([64, 128] if D == 128 else [32, 64])
    if op == "cache":
        packed = rng.random() < 0.5
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, min(4096, 60000 // (B * Hkv))))
        return {"op": "cache", "B": B, "lo": max(1, hi // 3) if packed else hi, "hi": hi, "Hkv": Hkv, "D": D,
                "P": P, "before": rng.choice([0, _log(rng, 1, 20000)]), "packed": packed}
    if op == "prompt":
        B = _log(rng, 1, 24)
        # at most the long case's products
        hi = _log(rng, 1, max(8, min(8192, int(math.sqrt((1 << 38) / (B * Hq * D))))))
        return {"op": "prompt", "B": B, "lo": max(1, int(hi * rng.uniform(0.2, 1.0))), "hi": hi, "Hq": Hq,
                "Hkv": Hkv, "D": D, "window": rng.choice([0, 0, _log(rng, 1, max(2, hi))]),
                "sinks": rng.random() < 0.4, "spare": rng.choice([0, rng.randint(1, 200)])}
    R = rng.choice([1, 1, 2, 4, 5, 8, _log(rng, 9, 1024)])
    B = _log(rng, 1, max(1, min(48, (1 << 37) // (R * Hq * D * (2 * R + 64)))))
    top = max(2 * R + 64, min(131072, (1 << 37) // (B * R * Hq * D), (1 << 27) // (B * Hkv * D)))
    hi = _log(rng, R, top)
    return {"op": "dense", "B": B, "R": R, "Hq": Hq, "Hkv": Hkv, "D": D, "P": P,
            "lo": max(R, int(hi * rng.uniform(0.3, 1.0))), "hi": hi,
            "window": rng.choice([0, 0, _log(rng, 1, max(2, hi))]), "sinks": rng.random() < 0.4,
            "holes": rng.random() < 0.3}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

THETA = 1.0e6
FACTOR = 8.0
ORIGINAL = 16384
LOW, HIGH = 1.0, 4.0            # wavelength bands, in turns over the original context
FAST, SLOW = 32.0, 1.0          # yarn ramp, in turns over the original context


def _spectrum(n, scaling):
    """Scaled frequencies (radians per position) of n pairs, in 64 bits."""
    i = torch.arange(n, dtype=torch.float64, device=DEV)
    f = THETA ** (-i / n)
    if scaling == "linear":
        return f / FACTOR
    if scaling == "yarn":
        dim = lambda turns: n * math.log(ORIGINAL / (turns * 2 * math.pi)) / math.log(THETA)  # noqa: E731
        lo, hi = max(math.floor(dim(FAST)), 0), min(math.ceil(dim(SLOW)), 2 * n - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f * (1 - ramp) + f / FACTOR * ramp
    if scaling == "wavelength":
        mix = ((ORIGINAL * f / (2 * math.pi) - LOW) / (HIGH - LOW)).clamp(0, 1)
        return f * mix + f / FACTOR * (1 - mix)
    return f


def _axis_of(pairs, layout):
    """The axis of each pair."""
    n, A = sum(pairs), len(pairs)
    if layout == "interleaved":
        return [i % A if i % A and i < A * pairs[i % A] else 0 for i in range(n)]
    return [a for a in range(A) for _ in range(pairs[a])]


def _positions(T, A, top, gen):
    """Positions of text (all axes alike) and images (a moment, rows and columns of patches)."""
    at = torch.arange(T, device=DEV) + int(torch.randint(max(1, top - T), (1,), generator=gen, device=DEV))
    pos = at.repeat(A, 1)
    side = 24
    for start in range(side, T, 4 * side * side):      # an image at every start
        n = min(side * side, T - start)
        p = torch.arange(n, device=DEV)
        base = pos[0, start].clone()
        pos[:, start:start + n] = base
        if A > 1:
            pos[1, start:start + n] = base + p // side
        if A > 2:
            pos[2, start:start + n] = base + p % side
    return pos.to(torch.int32).contiguous()


def _spread(case):
    """Lengths of packed rows, between lo and hi in no order: the case's own, as the outputs' shapes are."""
    return [case["lo"] + int((case["hi"] - case["lo"] + 1) * (0.5 + 0.618034 * i) % (case["hi"] - case["lo"] + 1))
            for i in range(case["B"])]


def _lengths(case, gen):
    return torch.randint(case["lo"], case["hi"] + 1, (case["B"],), generator=gen, device=DEV).to(torch.int32)


def _pages(B, L_max, P, gen):
    """A page table over a pool with spare pages, in no order."""
    mb = -(-L_max // P)
    n = B * mb + 3
    perm = torch.randperm(n, generator=gen, device=DEV)[: B * mb]
    return perm.to(torch.int32).reshape(B, mb).contiguous(), mb, n


def _exponent(m):
    """Least e in the range with m <= 448 2^e (whole numbers), of magnitudes m."""
    f, x = torch.frexp(m)                     # 448 = 0.875 2^9
    return torch.where(m > 0, x - 9 + (f > 0.875).int(), E_MIN).clamp(E_MIN, E_MAX)


def _pool(n, Hkv, P, D, gen):
    """Pages of keys or values: tokens and blocks of different magnitudes, as codes and exponents."""
    code = torch.empty(n, Hkv, P, D, dtype=torch.uint8, device=DEV)
    exps = torch.empty(n, Hkv, P // BLOCK, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (Hkv * P * D))
    for i in range(0, n, step):
        m = min(step, n - i)
        x = torch.randn(m, Hkv, P // BLOCK, BLOCK, D, generator=gen, device=DEV)
        x *= torch.exp(0.3 * torch.randn(m, Hkv, P // BLOCK, BLOCK, 1, generator=gen, device=DEV))
        e = _exponent(x.abs().amax((-1, -2)))
        code[i:i + m] = torch.ldexp(x, -e[..., None, None]).to(F8).view(torch.uint8).view(m, Hkv, P, D)
        exps[i:i + m] = (e + 127).to(torch.uint8)
    return code, exps


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s, op = dict(case), case["op"]
    randn = lambda *shape: torch.randn(*shape, generator=gen, device=DEV)  # noqa: E731
    if op == "axes":
        s["split"] = [int(n) for n in case["pairs"].split(",")]
        A, half, T = len(s["split"]), sum(s["split"]), case["T"]
        s["positions"] = _positions(T, A, case["at"], gen)
        s["axis"] = torch.tensor(_axis_of(s["split"], case["layout"]), device=DEV)
        s["freqs"] = (torch.cat([_spectrum(n, case["scaling"]) for n in s["split"]])
                      if case["layout"] == "spectra" else _spectrum(half, case["scaling"]))
        s["amp"] = 0.1 * math.log(FACTOR) + 1.0 if case["scaling"] == "yarn" else 1.0
        s["cs"] = torch.empty(T, half, 2, device=DEV)
    elif op == "cache":
        B, Hkv, D, P = (case[n] for n in ("B", "Hkv", "D", "P"))
        s["rows"] = _spread(case)
        rows = torch.tensor(s["rows"], device=DEV)
        before = torch.randint(case["before"] // 2, case["before"] + 1, (B,), generator=gen, device=DEV)
        s["seqlens"] = (before + rows).to(torch.int32)
        s["T"] = T = sum(s["rows"])
        s["cu"] = torch.cat([rows.new_zeros(1), rows.cumsum(0)]).to(torch.int32) if case["packed"] else None
        # keys and values are parts of a projection's rows
        s["kv"] = (randn(T, 2 * Hkv, D) * torch.exp(0.3 * randn(T, 2 * Hkv, 1))).to(BF16)
        s["page_table"], s["MB"], s["NP"] = _pages(B, case["before"] + case["hi"], P, gen)
        s["pools"] = [*_pool(s["NP"], Hkv, P, D, gen), *_pool(s["NP"], Hkv, P, D, gen)]
        # read back with the rows before them that share a block
        s["back"] = [n + BLOCK - 1 for n in s["rows"]]
        s["cu_back"] = torch.tensor([0, *s["back"]], device=DEV).cumsum(0).to(torch.int32) if case["packed"] else None
        s["out"] = [torch.zeros(sum(s["back"]), Hkv, D, dtype=BF16, device=DEV) for _ in range(2)]
    elif op == "dense":
        B, R, Hq, Hkv, D, P = (case[n] for n in ("B", "R", "Hq", "Hkv", "D", "P"))
        s["seqlens"] = _lengths(case, gen)
        s["page_table"], s["MB"], s["NP"] = _pages(B, case["hi"], P, gen)
        if case["holes"]:
            gone = torch.rand(s["page_table"].shape, generator=gen, device=DEV) < 0.05
            s["page_table"] = torch.where(gone, -1, s["page_table"]).contiguous()
        s["pools"] = [*_pool(s["NP"], Hkv, P, D, gen), *_pool(s["NP"], Hkv, P, D, gen)]
        s["T"] = B * R
    elif op == "prompt":
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        s["rows"] = _spread(case)
        lens = torch.tensor(s["rows"], device=DEV)
        s["T"] = T = sum(s["rows"]) + case["spare"]
        s["cu"] = torch.cat([lens.new_zeros(1), lens.cumsum(0)]).to(torch.int32)
        s["kv"] = randn(T, 2 * Hkv, D).to(BF16)
    if op in ("dense", "prompt"):
        # heads look about them or at few tokens: logits of standard deviation 0.5 to 2
        s["sm_scale"] = 1 / math.sqrt(D)
        s["q"] = (randn(s["T"], Hq, D) * torch.linspace(0.5, 2.0, Hq, device=DEV)[:, None]).to(BF16)
        s["sink"] = randn(Hq) + 2.0 if case["sinks"] else None
        s["o"] = torch.zeros(s["T"], Hq, D, dtype=BF16, device=DEV)
        s["lse"] = torch.zeros(s["T"], Hq, device=DEV)
    if own:
        s["keeps"] = _own_keeps(s)     # the geometry, plan and workspace that a program keeps
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plain_axes(s):
    a = s["positions"].double()[s["axis"]].T * s["freqs"]
    return {"cs": (torch.stack([a.cos(), a.sin()], -1) * s["amp"]).float()}


def _places(s, rows):
    """Request and position of each of the newest `rows` of the requests."""
    n = torch.tensor(rows, device=DEV)
    of = torch.arange(s["B"], device=DEV).repeat_interleave(n)
    nth = torch.arange(sum(rows), device=DEV) - (n.cumsum(0) - n)[of]
    return of, s["seqlens"].long()[of] - n[of] + nth


def _plain_cache(s):
    Hkv, P, per = s["Hkv"], s["P"], s["P"] // BLOCK
    of, pos = _places(s, s["rows"])
    page, slot = s["page_table"][of, pos // P].long(), pos % P
    block, nth = torch.unique(page * per + slot // BLOCK, return_inverse=True)
    first = torch.full_like(block, BLOCK).scatter_reduce(0, nth, slot % BLOCK, "amin")   # first new slot of it
    kept = torch.arange(BLOCK, device=DEV) < first[:, None]                              # [blocks, 16]
    k, v = s["kv"][:, :Hkv], s["kv"][:, Hkv:]
    heads = torch.arange(Hkv, device=DEV)
    for x, codes, exps in ((k, *s["pools"][:2]), (v, *s["pools"][2:])):
        x = x.float()
        size = torch.zeros(len(block), Hkv, device=DEV).scatter_reduce(
            0, nth[:, None].expand(-1, Hkv), x.abs().amax(-1), "amax")
        e = _exponent(size)
        at_page, at_block = block // per, block % per
        before = exps[at_page, :, at_block].int() - 127
        e = torch.where((first > 0)[:, None], torch.maximum(e, before), e)
        where = (at_block * BLOCK)[:, None] + torch.arange(BLOCK, device=DEV)            # slots of a block
        index = at_page[:, None, None], heads[None, :, None], where[:, None, :]
        old = codes[index].view(F8).float()                                              # [blocks, Hkv, 16, D]
        moved = torch.ldexp(old, (before - e)[..., None, None]).to(F8).view(torch.uint8)
        codes[index] = torch.where(kept[:, None, :, None], moved, codes[index])
        exps[at_page, :, at_block] = (e + 127).to(torch.uint8)
        codes[page, :, slot] = torch.ldexp(x, -e[nth][..., None]).to(F8).view(torch.uint8)
    of, pos = _places(s, s["back"])
    there = pos >= 0
    page, slot = s["page_table"][of, pos.clamp(min=0) // P].long(), pos % P
    for out, codes, exps in ((s["out"][0], *s["pools"][:2]), (s["out"][1], *s["pools"][2:])):
        val = torch.ldexp(codes[page, :, slot].view(F8).float(), (exps[page, :, slot // BLOCK].int() - 127)[..., None])
        out.copy_(torch.where(there[:, None, None], val.to(BF16), out))
    return {"k": s["out"][0], "v": s["out"][1]}


def _softmax_product(z, v, sink):
    """exp(z - lse) v and lse, z [..., tokens] masked by -inf, sink a logit more."""
    top = z.amax(-1)
    top = top if sink is None else torch.maximum(top, sink)
    base = torch.where(top == -math.inf, 0.0, top)
    p = z.sub_(base[..., None]).exp_()
    total = p.sum(-1)
    total = total if sink is None else total + (sink - base).exp()
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)[..., None]
    return o, base + total.log()


def _plain_dense(s):
    B, R, Hq, Hkv, D, P = (s[n] for n in ("B", "R", "Hq", "Hkv", "D", "P"))
    G, cap = Hq // Hkv, s["MB"] * P
    page = s["page_table"].long()
    live = (page >= 0) & (page < s["NP"])
    page = torch.where(live, page, 0)
    at = torch.arange(cap, device=DEV)
    n = s["seqlens"].long()[:, None] - R + 1 + torch.arange(R, device=DEV)               # [B, R]
    see = (at < n[..., None]) & live.repeat_interleave(P, 1)[:, None]
    if s["window"]:
        see &= at >= n[..., None] - s["window"]

    def tokens(codes, exps):     # [B, Hkv, cap, D]
        x = torch.ldexp(codes[page].view(F8).float(), (exps[page].int() - 127).repeat_interleave(BLOCK, -1)[..., None])
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, cap, D)

    q = s["q"].float().view(B, R, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, R * G, D)
    z = torch.matmul(q, tokens(*s["pools"][:2]).transpose(-1, -2)) * s["sm_scale"]
    z = z.view(B, Hkv, R, G, cap).masked_fill_(~see[:, None, :, None], -math.inf).view(B, Hkv, R * G, cap)
    sink = None if s["sink"] is None else s["sink"].view(1, Hkv, 1, G).expand(B, Hkv, R, G).reshape(B, Hkv, R * G)
    o, lse = _softmax_product(z, tokens(*s["pools"][2:]), sink)
    return {"out": o.view(B, Hkv, R, G, D).permute(0, 2, 1, 3, 4).reshape(B * R, Hq, D).to(BF16),
            "lse": lse.view(B, Hkv, R, G).permute(0, 2, 1, 3).reshape(B * R, Hq)}


def _plain_prompt(s):
    Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
    G, start = Hq // Hkv, 0
    for n in s["rows"]:
        rows = slice(start, start + n)
        q = s["q"][rows].float().view(n, Hkv, G, D).permute(1, 2, 0, 3)                  # [Hkv, G, n, D]
        k = s["kv"][rows, :Hkv].float().transpose(0, 1)[:, None]                         # [Hkv, 1, n, D]
        v = s["kv"][rows, Hkv:].float().transpose(0, 1)[:, None]
        z = torch.matmul(q, k.transpose(-1, -2)) * s["sm_scale"]
        at = torch.arange(n, device=DEV)
        hidden = at > at[:, None]
        if s["window"]:
            hidden |= at <= at[:, None] - s["window"]
        sink = None if s["sink"] is None else s["sink"].view(Hkv, G, 1)
        o, lse = _softmax_product(z.masked_fill_(hidden, -math.inf), v, sink)
        s["o"][rows] = o.permute(2, 0, 1, 3).reshape(n, Hq, D).to(BF16)
        s["lse"][rows] = lse.permute(2, 0, 1).reshape(n, Hq)
        start += n
    return {"out": s["o"], "lse": s["lse"]}


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _own_keeps(s):
    """What a program keeps from call to call: the geometry, the rotation's plan and the workspace."""
    import nvfp4_block_sparse_gb300 as qsa
    k = {"qsa": qsa}
    if s["op"] == "axes":
        more = {"linear": dict(factor=FACTOR),
                "yarn": dict(factor=FACTOR, original_context=ORIGINAL, beta_fast=FAST, beta_slow=SLOW),
                "wavelength": dict(factor=FACTOR, original_context=ORIGINAL, low_freq=LOW, high_freq=HIGH)}
        k["plan"] = qsa.make_rope_axes(s["split"], theta=THETA, layout=s["layout"], scaling=s["scaling"],
                                       **more.get(s["scaling"], {}))
        return k

    def geom(rows):
        return qsa.make_geom(batch=s["B"], rows_per_req=rows, num_q_heads=s.get("Hq", s["Hkv"]),
                             num_kv_heads=s["Hkv"], head_dim=s["D"], index_dim=64,
                             page_size=s.get("P", 64), max_blocks=s.get("MB", 1), num_pages=s.get("NP", 1))
    if s["op"] == "cache":
        k["geom"], k["geom_back"] = geom(1 if s["packed"] else s["hi"]), geom(1 if s["packed"] else s["back"][0])
        return k
    k["geom"] = geom(s.get("R", 1))
    n = (qsa.qsa_dense_attention_fp8_workspace_bytes(k["geom"]) if s["op"] == "dense"
         else qsa.qsa_prompt_attention_workspace_bytes(k["geom"], s["T"]))
    k["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    qsa.qsa_workspace_init(k["workspace"])
    return k


def _own_run(s):
    k, op = s["keeps"], s["op"]
    qsa = k["qsa"]
    if op == "axes":
        qsa.qsa_rope_axes_rows(k["plan"], s["positions"], s["cs"])
        return {"cs": s["cs"]}
    if op == "cache":
        Hkv = s["Hkv"]
        qsa.qsa_store_kv_tokens_fp8(k["geom"], s["kv"][:, :Hkv], s["kv"][:, Hkv:], s["page_table"], s["seqlens"],
                                    *s["pools"], cu_rows=s["cu"])
        qsa.qsa_load_kv_tokens_fp8(k["geom_back"], s["page_table"], s["seqlens"], *s["pools"], *s["out"],
                                   cu_rows=s["cu_back"])
        return {"k": s["out"][0], "v": s["out"][1]}
    if op == "dense":
        qsa.qsa_dense_attention_fp8(k["geom"], s["q"], *s["pools"], s["sm_scale"], s["page_table"], s["seqlens"],
                                    s["o"], s["lse"], k["workspace"], window=s["window"], sinks=s["sink"])
    else:
        Hkv = s["Hkv"]
        qsa.qsa_prompt_attention(k["geom"], s["q"], s["kv"][:, :Hkv], s["kv"][:, Hkv:], s["cu"], s["sm_scale"],
                                 s["o"], s["lse"], k["workspace"], window=s["window"], sinks=s["sink"])
    return {"out": s["o"], "lse": s["lse"]}


def run(state):
    if own:
        return _own_run(state)
    return {"axes": _plain_axes, "cache": _plain_cache, "dense": _plain_dense,
            "prompt": _plain_prompt}[state["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _seen(n, window):
    """Tokens that the rows of a causal sequence of n see, summed."""
    w = min(window or n, n)
    return w * (w + 1) / 2 + (n - w) * w


def work(case):
    op = case["op"]
    if op == "axes":
        split = [int(n) for n in case["pairs"].split(",")]
        n = case["T"] * sum(split)
        return {"bytes": 4 * case["T"] * len(split) + 8 * n, "flops": 10 * n}
    Hkv, D = case["Hkv"], case["D"]
    if op == "cache":
        # keys and values in, as codes out and in again, and out
        T = sum(_spread(case))
        n = 2 * Hkv * D * T
        return {"bytes": n * (2 + 1 + 1 + 2), "flops": 4 * n}
    Hq = case["Hq"]
    if op == "prompt":
        lens = _spread(case)
        T = sum(lens)
        return {"bytes": T * (4 * (Hq + Hkv) * D + 4 * Hq),
                "flops": 4 * D * Hq * sum(_seen(n, case["window"]) for n in lens)}
    B, R = case["B"], case["R"]
    T, L, w = B * R, (case["lo"] + case["hi"]) / 2, case["window"]
    each = min(L, w) if w else L - (R - 1) / 2            # tokens that a row sees
    read = min(L, w + R - 1) if w else L                  # tokens that a request's rows see together
    if case["holes"]:
        each, read = 0.95 * each, 0.95 * read
    return {"bytes": B * Hkv * read * (2 * D + 2 / BLOCK) + T * Hq * (4 * D + 4), "flops": 4 * D * T * Hq * each}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

E4M3 = [m * 2.0**-9 for m in range(8)] + [(8 + m) * 2.0**(x - 10) for x in range(1, 16) for m in range(8)][:-1]


def _exact_rows(q, keys, values, hidden, sink, scale):
    """One KV head: rows q [r, G, D] over keys [n, D]; hidden [r, n]; sink [G] or None."""
    z = torch.einsum("rgd,nd->rgn", q.double(), keys) * scale
    z = torch.where(hidden[:, None], -math.inf, z)
    if sink is not None:
        z = torch.cat([z, sink.double()[None, :, None].expand(z.shape[0], -1, 1)], -1)
    lse = torch.logsumexp(z, -1)
    p = torch.exp(z - lse[..., None]).nan_to_num(0.0)[..., :keys.shape[0]]
    return torch.einsum("rgn,nd->rgd", p, values), lse


def _exact_dense(s):
    B, R, Hq, Hkv, D, P = (s[n] for n in ("B", "R", "Hq", "Hkv", "D", "P"))
    G = Hq // Hkv
    out = torch.zeros(B * R, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B * R, Hq), -math.inf, dtype=torch.float64, device=DEV)
    grid = torch.tensor(E4M3 + [math.nan] + [-m for m in E4M3] + [math.nan], dtype=torch.float64, device=DEV)
    for b in range(B):
        L = int(s["seqlens"][b])
        blocks = torch.arange(-(-L // P), device=DEV)
        pages = s["page_table"][b, blocks].long()
        keep = pages >= 0
        blocks, pages = blocks[keep], pages[keep]
        where = (blocks[:, None] * P + torch.arange(P, device=DEV)).reshape(-1)
        use = where < L
        for h in range(Hkv):
            kv = []
            for i in (0, 2):
                two = torch.exp2(s["pools"][i + 1][pages, h].double() - 127).repeat_interleave(BLOCK, -1)
                kv.append((grid[s["pools"][i][pages, h].long()] * two[..., None]).reshape(-1, D)[use])
            heads = slice(h * G, (h + 1) * G)
            step = max(1, (1 << 28) // max(1, G * int(use.sum())))
            for j in range(0, R, step):
                n = L - R + 1 + torch.arange(j, min(R, j + step), device=DEV)[:, None]
                hidden = (where[use] >= n) | ((where[use] < n - s["window"]) if s["window"] else False)
                rows = slice(b * R + j, b * R + min(R, j + step))
                out[rows, heads], lse[rows, heads] = _exact_rows(
                    s["q"][rows, heads], kv[0], kv[1], hidden, None if s["sink"] is None else s["sink"][heads],
                    s["sm_scale"])
    return {"out": out, "lse": lse}


def _exact_prompt(s):
    Hq, Hkv, G = s["Hq"], s["Hkv"], s["Hq"] // s["Hkv"]
    out = torch.zeros(s["T"], Hq, s["D"], dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["T"], Hq, dtype=torch.float64, device=DEV)
    start = 0
    for n in s["rows"]:
        step = max(1, (1 << 28) // (G * n))
        for h in range(Hkv):
            k, v = (s["kv"][start:start + n, c].double() for c in (h, Hkv + h))
            heads = slice(h * G, (h + 1) * G)
            for j in range(0, n, step):
                i = torch.arange(j, min(n, j + step), device=DEV)[:, None]
                back = i - torch.arange(n, device=DEV)                    # how far a token lies behind a row
                hidden = (back < 0) | ((back >= s["window"]) if s["window"] else False)
                rows = slice(start + j, start + min(n, j + step))
                out[rows, heads], lse[rows, heads] = _exact_rows(
                    s["q"][rows, heads], k, v, hidden, None if s["sink"] is None else s["sink"][heads], s["sm_scale"])
        start += n
    return {"out": out, "lse": lse}


def _exact_cache(s):
    """Each row's value under the exponent that its block ends with, rounded once from the row
    (or, of a row that was there, from its former value)."""
    grid = torch.tensor([-m for m in E4M3[:0:-1]] + E4M3, dtype=torch.float64, device=DEV)
    Hkv, P = s["Hkv"], s["P"]
    res = {}
    for name, i, x in (("k", 0, s["kv"][:, :Hkv]), ("v", 2, s["kv"][:, Hkv:])):
        out, r0 = torch.zeros(sum(s["back"]), Hkv, s["D"], dtype=torch.float64, device=DEV), 0
        done = 0
        for b, n in enumerate(s["rows"]):
            L = int(s["seqlens"][b])
            start = L - n
            low = max(0, (start // BLOCK) * BLOCK)
            old = torch.arange(low - low % BLOCK, start, device=DEV)
            far = torch.arange(max(0, L - s["back"][b]), old[0] if len(old) else start, device=DEV)
            page = lambda p: s["page_table"][b, p // P].long()  # noqa: E731
            codes, exps = s["pools"][i], s["pools"][i + 1]

            def held(p):
                v = codes[page(p), :, p % P].view(F8).double()
                return v * torch.exp2(exps[page(p), :, (p % P) // BLOCK].double() - 127)[..., None]
            new = x[r0:r0 + n].double()
            pos = torch.arange(start, L, device=DEV)
            blk = pos // BLOCK - start // BLOCK
            most = torch.zeros(int(blk[-1]) + 1, Hkv, dtype=torch.float64, device=DEV)
            most.scatter_reduce_(0, blk[:, None].expand(-1, Hkv), new.abs().amax(-1), "amax")
            e = torch.ceil(torch.log2((most / TOP).clamp(min=1e-300))).clamp(E_MIN, E_MAX)
            if len(old):
                e[0] = torch.maximum(e[0], exps[page(old[:1])[0], :, (old[0] % P) // BLOCK].double() - 127)
            new, two = torch.cat([held(old), new]), torch.exp2(e[torch.cat([old // BLOCK - start // BLOCK, blk])])[..., None]
            up = torch.searchsorted(grid, (new / two).contiguous()).clamp(1, grid.numel() - 1)
            lower, upper = grid[up - 1], grid[up]
            t = new / two
            near = torch.where(t - lower < upper - t, lower, upper)
            even = torch.where((up - 1 - (len(E4M3) - 1)) % 2 == 0, lower, upper)        # ties: the even code
            near = torch.where(t - lower == upper - t, even, near) * two
            full = torch.cat([held(far), near])
            want = min(len(full), s["back"][b])
            out[done + s["back"][b] - want:done + s["back"][b]] = full[len(full) - want:]
            r0, done = r0 + n, done + s["back"][b]
        res[name] = out
    return res


def exact(case, seed):
    op = case["op"]
    # within 20 seconds up to this many products, in 64 bits
    if op in ("dense", "prompt") and work(case)["flops"] > 6e11:
        return None
    if op == "dense" and case["B"] * case["Hkv"] * -(-case["R"] * case["hi"] // (1 << 24)) > 5000:
        return None
    s = prepare(case, seed)
    if op == "axes":
        pos = s["positions"].double()
        turn = torch.stack([torch.polar(torch.full_like(pos[0], s["amp"]), pos[a] * f)
                            for a, f in zip(s["axis"].tolist(), s["freqs"].tolist())], 1)
        return {"cs": torch.view_as_real(turn)}
    return {"cache": _exact_cache, "dense": _exact_dense, "prompt": _exact_prompt}[op](s)
