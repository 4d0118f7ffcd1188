"""fp64 restatements of the step operators on the CPU (test infrastructure).

Each takes CPU tensors or Python lists and follows the definition in
include/sgq.h term by term, without the library's code. The attention and the
norm also return what their error bounds are made of.
"""
from __future__ import annotations

import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4, torch.float32: 2.0 ** -24}
LOWEST_STEP = {torch.bfloat16: 2.0 ** -134, torch.float8_e4m3fn: 2.0 ** -10, torch.float32: 0.0}
U = 2.0 ** -24  # half a step of fp32


def plan(lens, news, page, num_pages, table, table_ld, held, free_pages, free_count, depth,
         max_tokens):
    """(cu, slots, pos, req, table rows, held, free_count, bad) as Python lists; table is copied."""
    R = len(lens)
    table = [list(r) for r in table]
    lens, news, held = list(lens), list(news), list(held)
    bad = set()
    for r in range(R):
        if lens[r] < 0 or news[r] < 0 or held[r] < 0 or held[r] > table_ld or held[r] * page < lens[r]:
            bad.add("count")
            news[r], lens[r], held[r] = 0, max(lens[r], 0), min(max(held[r], 0), table_ld)
    avail = min(max(free_count, 0), num_pages)
    if avail != free_count:
        bad.add("count")
    cu, total = [0], 0
    for n in news:
        total += n
        cu.append(min(total, max_tokens))
    if total > max_tokens:
        bad.add("count")
    slots, pos, req = [], [], []
    left, seen, out_held = avail, 0, list(held)
    for r in range(R):
        n = cu[r + 1] - cu[r]
        want = -(-(lens[r] + n) // page) if n else 0
        need, served = max(0, want - held[r]), True
        if want > table_ld:
            bad.add("count")
            need, served = 0, False
        elif need and seen + need > avail:
            bad.add("pages")
            served = False
        seen += need
        if served and n:
            for j in range(held[r], want):
                table[r][j] = free_pages[left - 1]
                left -= 1
            out_held[r] = max(held[r], want)
        for i in range(n):
            p = lens[r] + i
            slot = -1
            if served:
                pg = table[r][p // page]
                if 0 <= pg < num_pages:
                    slot = pg * page + p % page
                else:
                    bad.add("index")
            slots.append(slot)
            pos.append(lens[r] + (depth[len(pos)] if depth is not None else i))
            req.append(r)
    return cu, slots, pos, req, table, out_held, left, bad


def rotate(x, rope, pos):
    """([T, heads, D] rotated in fp64, sum of the magnitudes of the two products)."""
    D = x.shape[-1]
    c = rope.double()[pos.long()][:, None, :]
    lo, hi, cos, sin = x[..., :D // 2], x[..., D // 2:], c[..., :D // 2], c[..., D // 2:]
    y = torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1)
    mag = torch.cat([(lo * cos).abs() + (hi * sin).abs(), (hi * cos).abs() + (lo * sin).abs()], -1)
    return y, mag


def stored_tolerance(y, mag, dtype):
    """How far the stored value may be from y: three fp32 roundings of at most U of
    the products' magnitudes each and one more (the division by the scale), then
    half a step of the type, taken of a value that is off by as much."""
    d = 4 * U * mag
    return d + HALF_STEP[dtype] * (y.abs() + d) + LOWEST_STEP[dtype]


def attention(q, lens, cu, keys, vals, sees, scale, k_scale=1.0, v_scale=1.0, eight=False):
    """keys, vals: per request [l + n, Hkv, D] fp64; sees: per request bool [n, l + n].
    Returns (out, lse, weighted |v|, largest sum of |q_i k_i| scaled) in fp64, [T, Hq(, D)].
    eight: q is taken in two 8-bit parts, each element off by at most 2^-17 of the
    row's largest; that is added to the sums, as a multiple of what they stand for
    in attention_tolerance ((D + 8) U of them)."""
    T, Hq, D = q.shape
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    mag = torch.zeros_like(out)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    dots = torch.zeros(T, Hq, dtype=torch.float64)
    for r in range(len(lens)):
        t0, n = cu[r], cu[r + 1] - cu[r]
        Hkv = keys[r].shape[1]
        G = Hq // Hkv
        for i in range(n):
            at = torch.nonzero(sees[r][i]).flatten()
            if at.numel() == 0:
                continue
            for h in range(Hq):
                k, v, x = keys[r][at, h // G], vals[r][at, h // G], q[t0 + i, h].double()
                s = (k * x).sum(-1) * (scale * k_scale)
                w = torch.softmax(s, 0)
                out[t0 + i, h] = (w[:, None] * v).sum(0) * v_scale
                mag[t0 + i, h] = (w[:, None] * v.abs()).sum(0) * v_scale
                lse[t0 + i, h] = torch.logsumexp(s, 0)
                d = (k * x).abs().sum(-1)
                if eight:
                    d = d + k.abs().sum(-1) * x.abs().max() * (2.0 ** -17 / ((D + 8) * U))
                dots[t0 + i, h] = (d * abs(scale * k_scale)).max()
    return out, lse, mag, dots


def attention_tolerance(out, lse, mag, dots, D, weight_half_step):
    """(tolerance of out, of lse). A score is a sum of D exact products in fp32
    (at most D U of the magnitudes), scaled, taken from the maximum and raised
    (about 8 U of the score's magnitude, 2^-21 of the power); the same holds for
    the sum below the line. Then the weights' rounding for the product with the
    values (weight_half_step of each, and fp16's lowest step), D and the keys'
    sums in fp32, and the output's half step."""
    e = (2 * (D + 8) * U * dots + 2.0 ** -20)[..., None]
    to = mag * (weight_half_step + 2.0 ** -14 + 2 * e) + 1e-30
    return to + 2.0 ** -8 * (out.abs() + to), e[..., 0] + 8 * U * lse.abs().nan_to_num(0, 0, 0)


def norm(a, w_post, gate, scale, resid, w_pre, w_offset, eps):
    """(r', x, tolerance of the fp32 r', factor of x on r') in fp64. The sums of squares are
    of fp32 squares, at most 64 added one by one and the rest in pairs: off by at
    most 2^-17; the norm's factor by half of that, and the products by 8 U."""
    r = resid.double()
    tol = torch.zeros_like(r)
    if a is not None:
        u = a.double()
        if w_post is not None:
            u = u / torch.sqrt((u * u).mean(-1, keepdim=True) + eps) * (w_offset + w_post.double())
        if gate is not None:
            u = u * gate.double()
        u = scale * u
        r = r + u
        tol = 2.0 ** -17 * u.abs() + U * r.abs()
    x = f = None
    if w_pre is not None:
        f = (w_offset + w_pre.double()) / torch.sqrt((r * r).mean(-1, keepdim=True) + eps)
        x = r * f
    return r, x, tol, f


def attention_by_head(q, cu, keys, vals, sees, scale, k_scale=1.0, v_scale=1.0, eight=False):
    """What ``attention`` returns, with a key head's rows taken together (long contexts,
    many rows)."""
    T, Hq, D = q.shape
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    mag = torch.zeros_like(out)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    dots = torch.zeros(T, Hq, dtype=torch.float64)
    for r in range(len(keys)):
        t0, n = cu[r], cu[r + 1] - cu[r]
        G = Hq // keys[r].shape[1]
        for h in range(keys[r].shape[1]):
            rows = slice(t0, t0 + n), slice(h * G, (h + 1) * G)
            x, k, v = q[rows].double(), keys[r][:, h], vals[r][:, h]
            hidden = ~sees[r][:, None, :]
            s = torch.einsum("ngd,ld->ngl", x, k) * (scale * k_scale)
            s = s.masked_fill(hidden, -math.inf)
            top = s.amax(-1, keepdim=True)
            w = (s - top.clamp(min=-1e300)).exp()
            total = w.sum(-1, keepdim=True)
            w = w / total.clamp(min=1e-300)
            out[rows] = torch.einsum("ngl,ld->ngd", w, v) * v_scale
            mag[rows] = torch.einsum("ngl,ld->ngd", w, v.abs()) * v_scale
            lse[rows] = (top + total.log())[..., 0]
            d = torch.einsum("ngd,ld->ngl", x.abs(), k.abs())
            if eight:
                d = d + k.abs().sum(-1) * x.abs().amax(-1, keepdim=True) * (2.0 ** -17 / ((D + 8) * U))
            dots[rows] = d.masked_fill(hidden, 0.0).amax(-1) * abs(scale * k_scale)
    return out, lse, mag, dots
