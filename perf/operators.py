"""What a decode or verification step needs around its projections, as measured work.

Four operators: the plan of a paged cache (block tables and slot maps from the
requests' lengths), the store of rotated keys and of values into its pages, the
attention of drafted tokens over it, and the norms around a block with its gate
and residual. ``run`` computes them in their plain form (elementary torch
operations in fp32, rounded once), or, where ``own`` is true, through the
library's entry points; ``exact`` states each from its definition in fp64.
"""
import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# The cases.
# ---------------------------------------------------------------------------

def listed():
    return [
        # A chat's next token, Llama-3-8B heads: one row per kv head group, latency counts.
        dict(name="attn 1 token 1000", op="attn", R=1, lo=1000, hi=1000, n=1, Hq=32, Hkv=8, D=128,
             page=16, layout="nhd", kv="bf16", tree=False),
        # One request verifies a tree of 16 drafted tokens (the GEMVs' largest batch), 64 query heads.
        dict(name="attn tree 16 x 8190", op="attn", R=1, lo=8190, hi=8190, n=16, Hq=64, Hkv=8, D=128,
             page=64, layout="hnd", kv="bf16", tree=True),
        # A served batch of ragged contexts, a few drafted tokens each.
        dict(name="attn ragged 24", op="attn", R=24, lo=17, hi=16111, n=6, Hq=32, Hkv=8, D=128,
             page=32, layout="nhd", kv="bf16", tree=True),
        # Long contexts held in 8 bits, plain decode with short chains, small heads, odd pages.
        dict(name="attn e4m3 long", op="attn", R=11, lo=900, hi=60000, n=3, Hq=32, Hkv=8, D=64,
             page=24, layout="hnd", kv="e4m3", tree=False),
        # Wide trees over long contexts: as many products as bytes.
        dict(name="attn wide trees", op="attn", R=12, lo=2000, hi=16384, n=64, Hq=64, Hkv=8, D=128,
             page=64, layout="nhd", kv="bf16", tree=True),
        # The norm before a projection at batch 1: fp32 residual plus an fp32 GEMV result.
        dict(name="norm 1 x 4096", op="norm", B=1, H=4096, a="f32", r="f32", w="bf16", post=False, gate="none"),
        # Norms on both sides of a block with a gate per channel, 16 rows.
        dict(name="norm 16 x 5120 both", op="norm", B=16, H=5120, a="bf16", r="f32", w="f32", post=True,
             gate="channel"),
        # A prompt chunk: rows enough to be bound by memory, a gate per row and channel.
        dict(name="norm 8191 x 5120", op="norm", B=8191, H=5120, a="bf16", r="bf16", w="bf16", post=True,
             gate="row"),
        # The 16 rows of a step's stacked q | k | v result into their pages, held in 8 bits.
        dict(name="write 16 rows", op="write", T=16, Hq=32, Hkv=8, D=128, page=16, layout="nhd", kv="e4m3",
             rope=True),
        # A prompt chunk into pages of 64, 64 query heads.
        dict(name="write 4001 rows", op="write", T=4001, Hq=64, Hkv=8, D=128, page=64, layout="hnd", kv="bf16",
             rope=True),
        # 16 requests with up to 16 drafted tokens each.
        dict(name="plan 16", op="plan", R=16, n=16, lo=1, hi=9000, page=16, short=False),
        # A full server: decoding requests beside prompt chunks.
        dict(name="plan 2000", op="plan", R=2000, n=300, lo=1, hi=20000, page=32, short=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "norm", "write", "plan"])
    if op == "norm":
        H = 8 * _log(rng, 8, 1024)
        B = _log(rng, 1, min(8191, 22000000 // H))
        return dict(op=op, B=B, H=H, a=rng.choice(["bf16", "f32"]), r=rng.choice(["bf16", "f32"]),
                    w=rng.choice(["bf16", "f32"]), post=rng.random() < 0.5,
                    gate=rng.choice(["none", "channel", "row"]))
    if op == "plan":
        return dict(op=op, R=_log(rng, 1, 2000), n=_log(rng, 1, 300), lo=1, hi=_log(rng, 10, 20000),
                    page=rng.choice([1, 8, 16, 24, 32, 64, 128]), short=rng.random() < 0.25)
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8])
    D = rng.choice([64, 128])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    layout = rng.choice(["nhd", "hnd"])
    kv = rng.choice(["bf16", "bf16", "e4m3"])
    if op == "write":
        return dict(op=op, T=_log(rng, 1, 2000), Hq=Hkv * G, Hkv=Hkv, D=D, page=page, layout=layout, kv=kv,
                    rope=rng.random() < 0.75)
    R = _log(rng, 1, 24)
    hi = _log(rng, 20, min(16000, 120000 // R))
    return dict(op=op, R=R, lo=rng.choice([0, 1, max(1, hi // 8), hi]), hi=hi, n=_log(rng, 1, 40), Hq=Hkv * G,
                Hkv=Hkv, D=D, page=page, layout=layout, kv=kv, tree=rng.random() < 0.6)


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
EPS = 1e-6


def _lens(c):
    """Cached tokens of each request, the same multiset for every seed."""
    R, lo, hi = c["R"], c["lo"], c["hi"]
    if R == 1:
        return [hi]
    a, b = math.log(lo + 1), math.log(hi + 1)
    return [int(round(math.exp(a + (b - a) * i / (R - 1)))) - 1 for i in range(R)]


def _news(c):
    """New tokens of each request: the full count, one, and between."""
    n, R = c["n"], c["R"]
    return [n if i % 3 == 0 else 1 + (7 * i) % n for i in range(R)]


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _dev(rows, dtype=torch.int32):
    return torch.tensor(rows, dtype=dtype).to(DEV)


def _cache(c, pages, gen, fill):
    """Keys and values of every slot, [pages, page, Hkv, D] as a view of the stored order."""
    shape = (pages, c["page"], c["Hkv"], c["D"]) if c["layout"] == "nhd" else (pages, c["Hkv"], c["page"], c["D"])
    got = []
    for _ in range(2):
        x = _randn(gen, *shape) if fill else torch.zeros(*shape, device=DEV)
        x = x.to(TYPES[c["kv"]])
        got.append(x if c["layout"] == "nhd" else x.transpose(1, 2))
    return got


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)
    c = case
    s = {"case": c, "kept": {}}
    if c["op"] == "norm":
        B, H = c["B"], c["H"]
        s["a"] = (_randn(gen, B, H) * 0.5).to(TYPES[c["a"]])
        s["r"] = (_randn(gen, B, H) * 2).to(TYPES[c["r"]])
        wt = TYPES[c["w"]]
        s["w_pre"] = (1 + 0.2 * _randn(gen, H)).to(wt)
        s["w_post"] = (1 + 0.2 * _randn(gen, H)).to(wt) if c["post"] else None
        shape = {"none": None, "channel": (H,), "row": (B, H)}[c["gate"]]
        s["gate"] = _randn(gen, *shape).to(wt) if shape else None
        s["scale"] = 0.5 if c["gate"] == "none" else 1.25
        s["r_out"] = torch.empty_like(s["r"])
        s["x"] = torch.empty(B, H, dtype=torch.bfloat16, device=DEV)
        return s
    if c["op"] == "write":
        T, Hq, Hkv, D, P = c["T"], c["Hq"], c["Hkv"], c["D"], c["page"]
        pages = -(-T // P) + 3
        s["k"], s["v"] = _cache(c, pages, gen, False)
        s["qkv"] = _randn(gen, T, (Hq + 2 * Hkv) * D).to(torch.bfloat16)
        s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
        s["slots"] = torch.randperm(pages * P, generator=host)[:T].to(DEV)
        s["pos"] = torch.randint(0, 32768, (T,), generator=host, dtype=torch.int32).to(DEV)
        s["k_scale"], s["v_scale"] = (0.021, 0.013) if c["kv"] == "e4m3" else (1.0, 1.0)
        s["rope"] = None
        if c["rope"]:  # cos | sin of pos / 500000^(2i/D), angles in fp64
            inv = 500000.0 ** (-torch.arange(0, D, 2, device=DEV, dtype=torch.float64) / D)
            ang = torch.arange(32768, device=DEV, dtype=torch.float64)[:, None] * inv
            s["rope"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        return s
    perm = torch.randperm(c["R"], generator=host).tolist()
    lens, news = _lens(c), _news(c)
    lens, news = [lens[i] for i in perm], [news[i] for i in perm]
    P, R = c["page"], c["R"]
    total = sum(news)
    s["lens"], s["news"] = _dev(lens), _dev(news)
    want = [-(-(l + n) // P) for l, n in zip(lens, news)]
    ld = max(want) + 2
    if c["op"] == "plan":
        held = [-(-l // P) for l in lens]
        short = sum(w - h for w, h in zip(want, held)) // 2
        pages = sum(want) + 5
        ids = torch.randperm(pages, generator=host).int()
        at = sum(held)
        table = torch.full((R, ld), -1, dtype=torch.int32)
        j = 0
        for r in range(R):
            table[r, :held[r]] = ids[j:j + held[r]]
            j += held[r]
        free = torch.full((pages,), -1, dtype=torch.int32)
        free[:pages - at] = ids[at:]
        s["table"], s["free"] = table.to(DEV), free.to(DEV)
        s["held"] = _dev(held)
        s["count"] = _dev([short if c["short"] else pages - at])
        s["depth"] = torch.randint(0, 5, (total,), generator=host, dtype=torch.int32).to(DEV)
        s["pages"], s["T"] = pages, total
        for k, n, t in (("held_out", R, torch.int32), ("count_out", 1, torch.int32), ("cu", R + 1, torch.int32),
                        ("slots", total, torch.int64), ("pos", total, torch.int32), ("req", total, torch.int32)):
            s[k] = torch.zeros(n, dtype=t, device=DEV)
        return s
    pages = sum(want) + 3
    ids = torch.randperm(pages, generator=host).int()
    table = torch.full((R, ld), -1, dtype=torch.int32)
    j = 0
    for r in range(R):
        table[r, :want[r]] = ids[j:j + want[r]]
        j += want[r]
    s["table"] = table.to(DEV)
    s["k"], s["v"] = _cache(c, pages, gen, True)
    s["k_scale"], s["v_scale"] = (0.75, 1.5) if c["kv"] == "e4m3" else (1.0, 1.0)
    s["q"] = (_randn(gen, total, c["Hq"], c["D"]) * 2).to(torch.bfloat16)
    s["scale"] = c["D"] ** -0.5
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    s["cu"] = _dev(cu)
    s["longest"], s["widest"], s["T"] = max(l + n for l, n in zip(lens, news)), max(news), total
    s["tree"] = None
    if c["tree"]:  # bit j of a token's words: draft token j is the token itself or one of its ancestors
        words = (max(news) + 31) // 32
        bits = torch.zeros(total, words * 32, dtype=torch.bool)
        for r in range(R):
            up = (torch.rand(news[r], generator=host) * torch.arange(news[r])).int().tolist()
            for i in range(news[r]):
                if i and up[i] != i - 1 or i % 4:
                    bits[cu[r] + i] = bits[cu[r] + up[i]]
                bits[cu[r] + i, i] = True
        place = torch.arange(32, dtype=torch.int64)
        s["tree"] = (bits.view(total, words, 32).long() << place).sum(-1).to(torch.int32).to(DEV)
    s["out"] = torch.empty(total, c["Hq"], c["D"], dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.empty(total, c["Hq"], dtype=torch.float32, device=DEV)
    return s


# ---------------------------------------------------------------------------
# One pass.
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return {"attn": _own_attn, "norm": _own_norm, "write": _own_write, "plan": _own_plan}[op](s)
    return {"attn": _attn, "norm": _norm, "write": _write, "plan": _plan}[op](s)


def _norm(s):
    u = s["a"].float()
    if s["w_post"] is not None:
        u = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS) * s["w_post"].float()
    if s["gate"] is not None:
        u = u * s["gate"].float()
    r = s["r"].float() + s["scale"] * u
    x = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * s["w_pre"].float()
    return r.to(s["r"].dtype), x.to(torch.bfloat16)


def _rotate(x, rope, pos):
    c = rope[pos.long()][:, None, :]
    half = x.shape[-1] // 2
    lo, hi, cos, sin = x[..., :half], x[..., half:], c[..., :half], c[..., half:]
    return torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1)


def _write(s):
    c = s["case"]
    T, Hq, Hkv, D, P = c["T"], c["Hq"], c["Hkv"], c["D"], c["page"]
    x = s["qkv"].float().view(T, Hq + 2 * Hkv, D)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    if s["rope"] is not None:
        q, k = _rotate(q, s["rope"], s["pos"]), _rotate(k, s["rope"], s["pos"])
    if c["kv"] == "e4m3":
        k, v = (k / s["k_scale"]).clamp(-448, 448), (v / s["v_scale"]).clamp(-448, 448)
    at = s["slots"] // P, s["slots"] % P
    s["k"][at] = k.to(s["k"].dtype)
    s["v"][at] = v.to(s["v"].dtype)
    return q.to(torch.bfloat16), s["k"], s["v"]


def _plan(s):
    P, T, table = s["case"]["page"], s["T"], s["table"]
    lens, news, held, avail = s["lens"].long(), s["news"].long(), s["held"].long(), s["count"].long()
    cu = torch.cat([news.new_zeros(1), news.cumsum(0)])
    want = (lens + news + P - 1) // P
    need = (want - held).clamp(min=0)
    base = need.cumsum(0) - need
    fits = (need == 0) | (base + need <= avail)
    j = torch.arange(table.shape[1], device=DEV)
    at = (avail - 1 - (base[:, None] + j - held[:, None])).clamp(0, s["pages"] - 1)
    fresh = fits[:, None] & (j >= held[:, None]) & (j < want[:, None])
    table.copy_(torch.where(fresh, s["free"][at], table))
    t = torch.arange(T, device=DEV)
    req = torch.searchsorted(cu, t, right=True) - 1
    p = lens[req] + t - cu[req]
    slots = torch.where(fits[req], table[req, p // P].long() * P + p % P, -1)
    left = avail - torch.where(fits, need, 0).sum()
    return (cu.int(), slots, (lens[req] + s["depth"]).int(), req.int(), table,
            torch.where(fits, torch.maximum(held, want), held).int(), left.int())


def _attn(s):
    c = s["case"]
    R, Hq, Hkv, D, P = c["R"], c["Hq"], c["Hkv"], c["D"], c["page"]
    G, L, N, T = Hq // Hkv, s["longest"], s["widest"], s["T"]
    lens, cu = s["lens"].long(), s["cu"].long()
    news = cu[1:] - cu[:-1]
    j = torch.arange(L, device=DEV)
    page = s["table"][:, j // P].long().clamp(min=0)
    k = s["k"][page, j % P].float().permute(0, 2, 3, 1) * s["k_scale"]
    v = s["v"][page, j % P].float().transpose(1, 2) * s["v_scale"]
    v = torch.where((j < (lens + news)[:, None])[:, None, :, None], v, 0)
    i = torch.arange(N, device=DEV)
    tok = (cu[:-1, None] + i).clamp(max=T - 1)
    q = s["q"].float()[tok].view(R, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(R, Hkv, N * G, D)
    back = j - lens[:, None]
    if s["tree"] is None:
        sees = back[:, None, :] <= i[:, None]
    else:
        b = back.clamp(0, s["tree"].shape[1] * 32 - 1)[:, None, :]
        sees = (torch.gather(s["tree"].long()[tok], 2, (b // 32).expand(R, N, L)) >> (b % 32)) & 1 != 0
        sees = sees | (back < 0)[:, None, :]
    sees = sees & (back < news[:, None])[:, None, :]
    w = torch.matmul(q, k).mul_(s["scale"]).view(R, Hkv, N, G, L)
    w.masked_fill_(~sees[:, None, :, None, :], -math.inf)
    m = w.amax(-1, keepdim=True)
    w = w.sub_(m.clamp(min=-1e30)).exp_()
    z = w.sum(-1, keepdim=True)
    o = torch.matmul(w.view(R, Hkv, N * G, L), v).view(R, Hkv, N, G, D) / z.clamp(min=1e-30)
    t = torch.arange(T, device=DEV)
    req = torch.searchsorted(cu, t, right=True) - 1
    out = o.permute(0, 2, 1, 3, 4)[req, t - cu[req]].reshape(T, Hq, D)
    lse = (m + z.log()).permute(0, 2, 1, 3, 4)[req, t - cu[req]].reshape(T, Hq)
    return out.to(torch.bfloat16), lse


def _own_norm(s):
    from activation_sparse_quantized_b200 import sgq
    a, r, x, gate = s["a"], s["r"], s["x"], s["gate"]
    B, H = a.shape
    sgq.sgq_residual_norm(a, H, s["w_post"], gate, H if gate is not None and gate.dim() == 2 else 0, s["scale"],
                          r, H, s["r_out"], H, s["w_pre"], 0.0, x, H, B, H, EPS)
    return s["r_out"], x


def _own_write(s):
    from activation_sparse_quantized_b200 import sgq
    c, kept = s["case"], s["kept"]
    T, Hq, Hkv, D = c["T"], c["Hq"], c["Hkv"], c["D"]
    if not kept:  # the cache's description and views of the stacked projection, made once
        kept["cache"] = sgq.Cache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        x = s["qkv"]
        kept["q"], kept["k"], kept["v"] = x, x[:, Hq * D:], x[:, (Hq + Hkv) * D:]
    ld = s["qkv"].shape[1]
    sgq.sgq_cache_write(kept["q"], ld, kept["k"], ld, kept["v"], ld, T, None, Hq, s["pos"], s["rope"],
                        32768 if s["rope"] is not None else 0, s["slots"], s["q_out"], Hq * D, kept["cache"])
    return s["q_out"], s["k"], s["v"]


def _own_plan(s):
    from activation_sparse_quantized_b200 import sgq
    sgq.sgq_cache_plan(s["lens"], s["news"], s["case"]["R"], s["case"]["page"], s["pages"], s["table"],
                       s["table"].shape[1], s["held"], s["held_out"], s["free"], s["count"], s["count_out"],
                       s["depth"], s["T"], s["cu"], s["slots"], s["pos"], s["req"])
    return s["cu"], s["slots"], s["pos"], s["req"], s["table"], s["held_out"], s["count_out"]


def _own_attn(s):
    from activation_sparse_quantized_b200 import sgq
    c, kept = s["case"], s["kept"]
    R, Hq, Hkv, D, T = c["R"], c["Hq"], c["Hkv"], c["D"], s["T"]
    if not kept:  # the cache's description and the workspace, made once
        kept["cache"] = sgq.Cache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        kept["ws"] = sgq.alloc_tree_attn_workspace(T, R, Hq, Hkv, D)
    tree = s["tree"]
    sgq.sgq_tree_attn(s["q"], Hq * D, T, R, Hq, s["lens"], s["cu"], s["table"], s["table"].shape[1], kept["cache"],
                      tree, tree.shape[1] if tree is not None else 0, s["scale"], s["out"], Hq * D, s["lse"],
                      kept["ws"])
    return s["out"], s["lse"]


# ---------------------------------------------------------------------------
# What a pass cannot do without.
# ---------------------------------------------------------------------------

SIZE = {"bf16": 2, "f32": 4, "e4m3": 1}


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["B"] * c["H"]
        w = SIZE[c["w"]]
        gate = {"none": 0, "channel": c["H"], "row": n}[c["gate"]]
        return {"bytes": n * (SIZE[c["a"]] + 2 * SIZE[c["r"]] + 2) + w * (c["H"] * (2 if c["post"] else 1) + gate),
                "flops": n * (12 if c["post"] else 8)}
    if c["op"] == "write":
        q, kv = c["T"] * c["Hq"] * c["D"], 2 * c["T"] * c["Hkv"] * c["D"]
        rope = c["T"] * c["D"] * 4 if c["rope"] else 0
        return {"bytes": q * 4 + kv * (2 + SIZE[c["kv"]]) + rope + 12 * c["T"],
                "flops": 3 * (q + kv // 2) if c["rope"] else kv}
    lens, news = _lens(c), _news(c)
    T, R, P = sum(news), c["R"], c["page"]
    if c["op"] == "plan":
        fresh = sum(-(-(l + n) // P) - -(-l // P) for l, n in zip(lens, news))
        return {"bytes": 20 * T + 20 * R + 8 * fresh + 4 * R, "flops": 6 * T + 6 * R}
    keys = sum(l + n for l, n in zip(lens, news))
    return {"bytes": keys * c["Hkv"] * c["D"] * 2 * SIZE[c["kv"]] + T * c["Hq"] * (c["D"] * 4 + 4) + 4 * keys // P,
            "flops": 4 * c["Hq"] * c["D"] * sum(n * (l + (n + 1) // 2) for l, n in zip(lens, news))}


# ---------------------------------------------------------------------------
# The definitions in 64 bits.
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "norm": _exact_norm, "write": _exact_write, "plan": lambda s: None}[case["op"]](s)


def _exact_norm(s):
    def rms(y):
        return (torch.linalg.vector_norm(y, dim=1) ** 2 / y.shape[1] + EPS).sqrt()[:, None]

    a = s["a"].double()
    if s["w_post"] is not None:
        a = a / rms(a) * s["w_post"].double()
    if s["gate"] is not None:
        a = a * s["gate"].double()
    r = s["r"].double() + s["scale"] * a
    return r, r / rms(r) * s["w_pre"].double()


def _exact_write(s):
    c = s["case"]
    T, Hq, Hkv, D, P = c["T"], c["Hq"], c["Hkv"], c["D"], c["page"]
    heads = s["qkv"].double().view(T, -1, D)
    if s["rope"] is not None:
        turn = torch.complex(s["rope"][:, :D // 2].double(), s["rope"][:, D // 2:].double())[s["pos"].long()]
        z = torch.complex(heads[:, :Hq + Hkv, :D // 2], heads[:, :Hq + Hkv, D // 2:]) * turn[:, None]
        heads = torch.cat([torch.cat([z.real, z.imag], -1), heads[:, Hq + Hkv:]], 1)
    k = torch.zeros(s["k"].shape[0] * P, Hkv, D, dtype=torch.float64, device=DEV)
    v = torch.zeros_like(k)
    k[s["slots"]] = heads[:, Hq:Hq + Hkv] / s["k_scale"]
    v[s["slots"]] = heads[:, Hq + Hkv:] / s["v_scale"]
    return heads[:, :Hq], k.view(s["k"].shape), v.view(s["v"].shape)


def _exact_attn(s):
    c = s["case"]
    Hq, Hkv, D, P = c["Hq"], c["Hkv"], c["D"], c["page"]
    G = Hq // Hkv
    lens, cu, table = s["lens"].tolist(), s["cu"].tolist(), s["table"].tolist()
    out = torch.zeros(s["T"], Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((s["T"], Hq), -math.inf, dtype=torch.float64, device=DEV)
    for r, l in enumerate(lens):
        n = cu[r + 1] - cu[r]
        ids = torch.tensor(table[r][:-(-(l + n) // P)], device=DEV)
        keys = s["k"][ids].reshape(-1, Hkv, D)[:l + n]
        vals = s["v"][ids].reshape(-1, Hkv, D)[:l + n]
        hidden = torch.zeros(n, l + n, dtype=torch.bool, device=DEV)
        if s["tree"] is None:
            hidden[:, l:] = torch.ones(n, n, device=DEV).triu(1) != 0
        else:
            words = s["tree"][cu[r]:cu[r + 1]].cpu().numpy().view("uint32")
            seen = [[(int(words[i, b // 32]) >> (b % 32)) & 1 for b in range(n)] for i in range(n)]
            hidden[:, l:] = torch.tensor(seen, device=DEV) == 0
        for h in range(Hkv):
            q = s["q"][cu[r]:cu[r + 1], h * G:(h + 1) * G].double()
            w = torch.einsum("ngd,ld->gnl", q, keys[:, h].double()) * (s["scale"] * s["k_scale"])
            w = w.masked_fill(hidden, -math.inf)
            lse[cu[r]:cu[r + 1], h * G:(h + 1) * G] = torch.logsumexp(w, -1).T
            p = torch.softmax(w, -1)
            out[cu[r]:cu[r + 1], h * G:(h + 1) * G] = torch.einsum("gnl,ld->ngd", p, vals[:, h].double()) * s["v_scale"]
    return out, lse
