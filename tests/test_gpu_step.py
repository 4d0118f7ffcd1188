"""The step entry points on the GPU against their fp64 definitions
(step_oracle): cache plan, cache store, tree attention, residual norm, and a
run of them together with the GEMVs. Tolerances are derived in step_oracle."""
import math
import os
import random
import subprocess
import sys

import pytest
import torch

import step_oracle as so
from activation_sparse_quantized_b200 import build, sgq
from activation_sparse_quantized_b200 import workloads as wl

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    torch.cuda.set_device(0)
    return sgq.load()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def status_word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------------------
# Plan.
# ---------------------------------------------------------------------------

def run_plan(lens, news, page, num_pages, table, held, free, count, depth, max_tokens, in_place=True, rows=None):
    R, ld = len(lens), len(table[0])
    rows = rows or max_tokens
    t = dict(table=i32(table), held=i32(held), count=i32([count]), cu=i32([-7] * (R + 1)),
             slots=torch.full((rows,), -77, dtype=torch.int64, device=DEV), pos=i32([-7] * rows), req=i32([-7] * rows),
             status=status_word())
    held_out, count_out = (t["held"], t["count"]) if in_place else (i32([-7] * R), i32([-7]))
    args = (i32(lens), i32(news), R, page, num_pages, t["table"], ld, t["held"], held_out, i32(free), t["count"],
            count_out, None if depth is None else i32(depth), max_tokens, t["cu"], t["slots"], t["pos"], t["req"], t["status"])
    sgq.sgq_cache_plan(*args)
    torch.cuda.synchronize()
    if not in_place:
        assert t["held"].tolist() == list(held) and t["count"].tolist() == [count]
    return args, dict(t, held=held_out, count=count_out)


def check_plan(got, want, max_tokens):
    cu, slots, pos, req, table, held, left, bad = want
    T = cu[-1]
    assert got["cu"].tolist() == cu
    assert got["slots"].tolist()[:T] == slots and got["pos"].tolist()[:T] == pos and got["req"].tolist()[:T] == req
    # rows behind the last new token stay as they were
    assert (got["slots"][T:] == -77).all() and (got["pos"][T:] == -7).all() and (got["req"][T:] == -7).all()
    assert got["table"].tolist() == table and got["held"].tolist() == held and got["count"].tolist() == [left]
    bits = {"count": 4, "index": 2, "pages": 16}
    assert got["status"].item() == sum(bits[b] for b in bad)


def plan_case(R, page, lo, hi, n, seed, short=False, spare=0):
    rng = random.Random(seed)
    lens = [rng.randint(lo, hi) for _ in range(R)]
    news = [rng.randint(0, n) for _ in range(R)]
    held = [-(-l // page) + rng.randint(0, spare) for l in lens]
    ld = max(max(-(-(l + m) // page), h) for l, m, h in zip(lens, news, held)) + 1
    ids = list(range(sum(held) + sum(-(-m // page) + 1 for m in news) + 2))
    rng.shuffle(ids)
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-1] * (ld - h))
        at += h
    free = ids[at:]
    count = len(free) // 3 if short else len(free)
    return lens, news, page, len(ids), table, held, free + [-1] * at, count


@pytest.mark.parametrize("R,page,lo,hi,n", [
    (1, 16, 0, 0, 1), (1, 16, 15, 15, 2), (3, 1, 0, 9, 5), (16, 16, 0, 300, 16), (33, 24, 5, 1000, 40),
    (257, 64, 0, 5000, 9), (1025, 32, 0, 700, 30), (2049, 8, 0, 64, 3), (5, 128, 0, 0, 4000)])
@pytest.mark.parametrize("in_place", [True, False])
def test_plan(R, page, lo, hi, n, in_place):
    c = plan_case(R, page, lo, hi, n, R + page, spare=2 if R > 3 else 0)
    T = max(1, sum(c[1]))
    depth = [random.Random(i).randint(0, 7) for i in range(T)] if R % 2 else None
    _, got = run_plan(*c, depth, T, in_place, rows=T + 5)
    check_plan(got, so.plan(*c[:5], len(c[4][0]), *c[5:], depth, T), T)


def test_plan_hands_out_the_first_that_fit_and_flags_the_rest():
    c = plan_case(40, 4, 0, 30, 20, 3, short=True)
    T = sum(c[1])
    want = so.plan(*c[:5], len(c[4][0]), *c[5:], None, T)
    assert want[-1] == {"pages"} and -1 in want[1] and want[1][0] >= 0
    args, got = run_plan(*c, None, T)
    check_plan(got, want, T)


def test_plan_of_no_pages_at_all_and_of_no_tokens():
    c = plan_case(4, 8, 3, 8, 9, 1)
    _, got = run_plan(*c[:7], 0, None, sum(c[1]))
    check_plan(got, so.plan(*c[:5], len(c[4][0]), *c[5:7], 0, None, sum(c[1])), sum(c[1]))
    c = plan_case(4, 8, 3, 8, 0, 1)
    _, got = run_plan(*c, None, 6)
    check_plan(got, so.plan(*c[:5], len(c[4][0]), *c[5:], None, 6), 6)


@pytest.mark.parametrize("fault", ["len", "new", "held", "wide", "tokens", "count", "page"])
def test_plan_of_bad_device_state_is_flagged_and_stays_in_bounds(fault):
    lens, news, page, pages, table, held, free, count = plan_case(9, 8, 1, 60, 12, 5)
    T = sum(news)
    if fault == "len":
        lens[3] = -4
    elif fault == "new":
        news[3] = -1
    elif fault == "held":
        held[3] = 0
    elif fault == "wide":
        news[3], T = 8 * len(table[0]) + 1, T + 8 * len(table[0]) + 1
    elif fault == "tokens":
        T -= 5
    elif fault == "count":
        count = pages + 50
        free = free[:count] + [0] * (pages - len(free[:count]))
    elif fault == "page":
        r = next(r for r in range(9) if lens[r] % 8 and news[r])
        table[r][lens[r] // 8] = pages + 3
    _, got = run_plan(lens, news, page, pages, table, held, free, count, None, T, rows=T + 3)
    want = so.plan(lens, news, page, pages, table, len(table[0]), held, free, count, None, T)
    assert want[-1]
    check_plan(got, want, T)


def test_plan_again_on_its_own_result_gives_the_same_rows():
    c = plan_case(20, 16, 0, 200, 16, 8)
    T = sum(c[1])
    args, got = run_plan(*c, None, T)
    first = {k: v.clone() for k, v in got.items()}
    sgq.sgq_cache_plan(*args)
    torch.cuda.synchronize()
    for k in first:
        assert torch.equal(first[k], got[k]), k


# ---------------------------------------------------------------------------
# Store.
# ---------------------------------------------------------------------------

def make_cache(pages, page, Hkv, D, layout, dtype, fill=0.0):
    shape = (pages, page, Hkv, D) if layout == "nhd" else (pages, Hkv, page, D)
    k, v = (torch.full(shape, fill, device=DEV).to(dtype) for _ in range(2))
    return (k, v) if layout == "nhd" else (k.transpose(1, 2), v.transpose(1, 2))


def rope_table(n, D, base=10000.0):
    ang = torch.arange(n, dtype=torch.float64)[:, None] * base ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    return torch.cat([ang.cos(), ang.sin()], 1).float()


@pytest.mark.parametrize("T,Hq,Hkv,D,page,layout,dtype,rope", [
    (1, 8, 2, 64, 16, "nhd", BF16, True), (16, 32, 8, 128, 16, "hnd", BF16, True), (7, 3, 3, 128, 1, "nhd", E4M3, True),
    (130, 5, 1, 64, 24, "hnd", E4M3, False), (33, 0, 2, 64, 8, "nhd", BF16, True), (65, 64, 8, 128, 64, "nhd", BF16, False)])
def test_write(T, Hq, Hkv, D, page, layout, dtype, rope):
    g = torch.Generator().manual_seed(T)
    pages = -(-T // page) + 2
    k, v = make_cache(pages, page, Hkv, D, layout, dtype, 3.0)
    ks, vs = (0.021, 0.013) if dtype == E4M3 else (1.0, 1.0)
    pad = 8
    qkv = (torch.randn(T, (Hq + 2 * Hkv) * D + pad, generator=g) * 3).to(BF16)
    ld = qkv.shape[1]
    table = rope_table(500, D) if rope else None
    pos = torch.randint(0, 500, (T,), generator=g, dtype=torch.int32)
    slots = torch.randperm(pages * page, generator=g)[:T]
    d = qkv.to(DEV)
    q_out = torch.full((T, max(1, Hq) * D + pad), 7.0, dtype=BF16, device=DEV)
    st = status_word()
    before = [x.to(F32).cpu() for x in (k, v)]
    sgq.sgq_cache_write(d if Hq else None, ld, d[:, Hq * D:], ld, d[:, (Hq + Hkv) * D:], ld, T, None, Hq,
                        pos.to(DEV), table.to(DEV) if rope else None, 500, slots.to(DEV), q_out if Hq else None,
                        q_out.shape[1], sgq.Cache(k, v, ks, vs), st)
    torch.cuda.synchronize()
    assert st.item() == 0
    heads = qkv[:, :(Hq + 2 * Hkv) * D].double().view(T, -1, D)
    mag = torch.zeros_like(heads)
    if rope:
        y, m = so.rotate(heads[:, :Hq + Hkv], table, pos)
        heads = torch.cat([y, heads[:, Hq + Hkv:]], 1)
        mag[:, :Hq + Hkv] = m
    if Hq:
        got = q_out[:, :Hq * D].cpu().double().view(T, Hq, D)
        assert ((got - heads[:, :Hq]).abs() <= so.stored_tolerance(heads[:, :Hq], mag[:, :Hq], BF16)).all()
        assert (q_out[:, Hq * D:] == 7.0).all()
    for x, old, part, scale in ((k, before[0], slice(Hq, Hq + Hkv), ks), (v, before[1], slice(Hq + Hkv, None), vs)):
        got = x.to(F32).cpu().reshape(pages * page, Hkv, D)
        want, m = heads[:, part] / scale, (mag[:, part] + (heads[:, part].abs() if dtype == E4M3 else 0)) / scale
        if dtype == E4M3:
            want = want.clamp(-448, 448)
        assert ((got[slots].double() - want).abs() <= so.stored_tolerance(want, m, dtype)).all()
        rest = torch.ones(pages * page, dtype=torch.bool)
        rest[slots] = False
        assert torch.equal(got[rest], old.reshape(pages * page, Hkv, D)[rest])   # other slots untouched


def test_write_skips_what_it_is_told_to_and_flags_the_rest():
    T, Hkv, D, page, pages = 6, 2, 64, 8, 3
    k, v = make_cache(pages, page, Hkv, D, "nhd", BF16, 5.0)
    x = torch.randn(T, Hkv * D, device=DEV).to(BF16)
    run = lambda slots, pos, n, rope=None: sgq.sgq_cache_write(
        None, 0, x, Hkv * D, x, Hkv * D, T, n, 0, pos, rope, 4, torch.tensor(slots, device=DEV), None, 0, sgq.Cache(k, v), st)
    st = status_word()
    run([-1, 3, -1, 5, 9, 9], None, i32([4]))               # -1: skipped; rows behind the count: not read
    assert st.item() == 0 and torch.equal(k.view(-1, Hkv * D)[3], x[1]) and torch.equal(v.view(-1, Hkv * D)[5], x[3])
    assert (k.view(-1, Hkv * D)[[0, 1, 2, 4, 9]] == 5).all()
    run([-2, 0, pages * page, 1, 2, 6], None, None)
    assert st.item() == 2 and torch.equal(k.view(-1, Hkv * D)[0], x[1]) and torch.equal(k.view(-1, Hkv * D)[6], x[5])
    st.zero_()
    k.fill_(5.0)
    run([10, 11, 12, 13, 14, 15], i32([0, 4, -1, 3, 1, 2]), None, rope_table(4, D).to(DEV))
    assert st.item() == 2 and (k.view(-1, Hkv * D)[[11, 12]] == 5).all() and not (k.view(-1, Hkv * D)[13] == 5).all()
    st.zero_()
    run([0, 1, 2, 3, 4, 5], None, i32([7]))
    assert st.item() == 4 and torch.equal(k.view(-1, Hkv * D)[5], x[5])


def test_write_q_in_place_saturation_and_nan():
    T, D = 3, 64
    x = torch.tensor([1e30, -1e30, math.inf, -math.inf, math.nan, 449.0, 463.9, 0.0009], dtype=F32).repeat(8).to(BF16)
    x = x.expand(T, D).contiguous().to(DEV)
    k, v = make_cache(1, 8, 1, D, "nhd", E4M3)
    rope = rope_table(9, D).to(DEV)
    q = torch.randn(T, 2 * D, device=DEV).to(BF16)
    sep = torch.empty_like(q)
    pos = i32([0, 5, 8])
    args = lambda out: (q, 2 * D, x, D, x, D, T, None, 2, pos, rope, 9, torch.arange(T, device=DEV), out, 2 * D, sgq.Cache(k, v))
    sgq.sgq_cache_write(*args(sep))
    sgq.sgq_cache_write(*args(q))                                # q_out may be q
    torch.cuda.synchronize()
    assert torch.equal(q, sep)
    got = v.float().cpu().view(8, D)[:T, :8]
    want = torch.tensor([448, -448, 448, -448, math.nan, 448, 448, 2.0 ** -10 * 0]).expand(T, 8)
    assert torch.equal(got.nan_to_num(-1), want.nan_to_num(-1))


# ---------------------------------------------------------------------------
# Attention.
# ---------------------------------------------------------------------------

class AttnCase:
    def __init__(self, lens, news, Hq, Hkv, D, page, layout="nhd", dtype=BF16, tree="random", seed=0, rows=0, q_scale=1.5):
        g = torch.Generator().manual_seed(seed)
        R = len(lens)
        self.lens, self.news, self.Hq, self.Hkv, self.D, self.page = lens, news, Hq, Hkv, D, page
        self.cu = [0]
        for n in news:
            self.cu.append(self.cu[-1] + n)
        T = self.T = max(1, self.cu[-1]) + rows
        want = [-(-(l + n) // page) for l, n in zip(lens, news)]
        self.pages = sum(want) + 2
        ids = torch.randperm(self.pages, generator=g).tolist()
        self.ld = max(want) + 1
        self.table, at = torch.full((R, self.ld), -1, dtype=torch.int32), 0
        for r in range(R):
            self.table[r, :want[r]] = torch.tensor(ids[at:at + want[r]])
            at += want[r]
        # what no request holds is NaN: a slot that must not be used shows
        self.k, self.v = make_cache(self.pages, page, Hkv, D, layout, dtype, math.nan)
        self.ks, self.vs = (0.75, 1.5) if dtype == E4M3 else (1.0, 1.0)
        self.keys, self.vals = [], []
        for r in range(R):
            L = lens[r] + news[r]
            for x, to in ((self.k, self.keys), (self.v, self.vals)):
                y = torch.randn(L, Hkv, D, generator=g).to(dtype)
                p = torch.arange(L)
                x.view(torch.uint8 if dtype == E4M3 else torch.int16)[self.table[r].long()[p // page].to(DEV), (p % page).to(DEV)] = \
                    y.view(torch.uint8 if dtype == E4M3 else torch.int16).to(DEV)
                to.append(y.to(F32).double())
        self.q = (torch.randn(T, Hq, D, generator=g) * q_scale).to(BF16)
        self.words = max(1, (max(news) + 31) // 32)
        self.tree, self.sees = None, []
        if tree == "random":
            self.tree = torch.zeros(T, self.words, dtype=torch.int64)
        for r in range(R):
            n, L = news[r], lens[r] + news[r]
            see = torch.ones(n, L, dtype=torch.bool)
            if tree == "random":
                bits = torch.rand(n, n, generator=g) < 0.4
                bits |= torch.eye(n, dtype=torch.bool)
                see[:, lens[r]:] = bits
                for i in range(n):
                    for j in range(n):
                        if bits[i, j]:
                            self.tree[self.cu[r] + i, j // 32] |= 1 << (j % 32)
            else:
                see[:, lens[r]:] = torch.ones(n, n).tril() != 0
            self.sees.append(see)
        self.scale = D ** -0.5
        self.ws = sgq.alloc_tree_attn_workspace(T, R, Hq, Hkv, D)
        self.out = torch.full((T, Hq, D), 9.0, dtype=BF16, device=DEV)
        self.lse = torch.full((T, Hq), 9.0, device=DEV)
        self.status = status_word()

    def words_tensor(self):
        return None if self.tree is None else (self.tree & 0xffffffff).to(torch.int64).apply_(
            lambda w: w - (1 << 32) if w >= 1 << 31 else w).to(torch.int32).to(DEV)

    def args(self, **kw):
        a = dict(q=self.q.to(DEV), ld_q=self.Hq * self.D, T=self.T, R=len(self.lens), Hq=self.Hq, lens=i32(self.lens),
                 cu_new=i32(self.cu), table=self.table.to(DEV), table_ld=self.ld, cache=sgq.Cache(self.k, self.v, self.ks, self.vs),
                 tree=self.words_tensor(), tree_words=self.words if self.tree is not None else 0, scale=self.scale, out=self.out,
                 ld_out=self.Hq * self.D, lse=self.lse, workspace=self.ws, status=self.status)
        a.update(kw)
        return a

    def run(self, **kw):
        sgq.sgq_tree_attn(**self.args(**kw))
        torch.cuda.synchronize()
        return self

    def check(self, status=0):
        assert self.status.item() == status
        f8 = self.k.dtype == E4M3
        out, lse, mag, dots = so.attention(self.q, self.lens, self.cu, self.keys, self.vals, self.sees, self.scale, self.ks, self.vs, f8)
        n = self.cu[-1]
        got, gl = self.out.cpu().double(), self.lse.cpu().double()
        to, tl = so.attention_tolerance(out, lse, mag, dots, self.D, 2.0 ** -11 if f8 else 2.0 ** -8)
        assert torch.equal(torch.isfinite(lse[:n]), torch.isfinite(gl[:n]))
        seen = torch.isfinite(lse[:n])
        assert ((got[:n] - out[:n]).abs() <= to[:n]).all(), float(((got[:n] - out[:n]).abs() / to[:n]).max())
        assert ((gl[:n] - lse[:n])[seen].abs() <= tl[:n][seen]).all()
        assert (got[n:] == 9.0).all() and (gl[n:] == 9.0).all()   # rows behind the last request


@pytest.mark.parametrize("Hq,Hkv,D,page,layout,dtype", [
    (8, 8, 64, 16, "nhd", BF16), (8, 2, 128, 16, "hnd", BF16), (6, 2, 64, 24, "hnd", E4M3), (10, 2, 128, 7, "nhd", E4M3),
    (16, 1, 128, 64, "nhd", BF16), (5, 1, 64, 1, "nhd", BF16), (7, 1, 128, 128, "hnd", E4M3),
    (4, 2, 64, 5, "nhd", E4M3), (4, 1, 64, 2, "hnd", E4M3), (4, 4, 128, 12, "nhd", BF16)])
@pytest.mark.parametrize("lens,news", [([0], [1]), ([1], [1]), ([63], [1]), ([64], [1]), ([127, 0, 65], [1, 3, 2]),
                                       ([300, 5, 64, 1000], [7, 16, 1, 33])])
@pytest.mark.parametrize("tree", ["random", None])
def test_attention(Hq, Hkv, D, page, layout, dtype, lens, news, tree):
    AttnCase(lens, news, Hq, Hkv, D, page, layout, dtype, tree, seed=len(lens) + Hq, rows=2).run().check()


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("n,Hq", [(1, 4), (2, 4), (5, 4), (9, 8), (16, 8), (40, 4), (70, 2)])
def test_attention_split_over_a_long_context(dtype, n, Hq):
    AttnCase([4111], [n], Hq, 1, 128, 32, "nhd", dtype, "random", seed=n).run().check()


def test_attention_many_requests_and_requests_without_new_tokens():
    rng = random.Random(4)
    lens = [rng.choice([0, 1, 17, 64, 200]) for _ in range(300)]
    news = [rng.choice([0, 1, 1, 2]) for _ in range(300)]
    AttnCase(lens, news, 4, 2, 64, 16, rows=3, seed=3).run().check()
    AttnCase([5, 9, 30], [0, 0, 0], 4, 2, 64, 16, rows=3).run().check()      # nothing at all to do


def test_attention_rows_that_see_nothing_and_masked_values_that_are_not_finite():
    for dtype in (BF16, E4M3):
        for lens in ([0, 40], [60, 0], [0, 127]):
            c = AttnCase(lens, [6, 5], 4, 2, 128, 16, "nhd", dtype, "random", seed=9)
            # token 1 of request 0 sees no drafted token; where it has no context, nothing at all
            c.tree[1] = 0
            c.sees[0][1, lens[0]:] = False
            # drafted token 3 of both is seen by itself alone, and holds NaN (bf16: and infinities)
            for r in range(2):
                p = lens[r] + 3
                at = int(c.table[r, p // 16]), p % 16
                bad = torch.full((2, 128), math.nan).to(dtype)
                if dtype == BF16:
                    bad[:, ::2] = math.inf
                w = torch.uint8 if dtype == E4M3 else torch.int16
                c.v.view(w)[at] = bad.view(w).to(DEV)
                c.k.view(w)[at] = bad.view(w).to(DEV)
                for i in range(c.news[r]):
                    if i != 3:
                        c.tree[c.cu[r] + i, 0] &= ~(1 << 3)
                        c.sees[r][i, lens[r] + 3] = False
            c.run()
            own = [c.cu[0] + 3, c.cu[1] + 3]
            assert torch.isnan(c.out[own].float()).any(-1).all()    # the rows that see it show it
            for t in own:                                            # the others are as without it
                c.tree[t] = 0
            for r in range(2):
                c.sees[r][3] = False
            got, lse = c.out.clone(), c.lse.clone()
            ref, rl, mag, dots = so.attention(c.q, c.lens, c.cu, c.keys, c.vals, c.sees, c.scale, c.ks, c.vs, dtype == E4M3)
            to, tl = so.attention_tolerance(ref, rl, mag, dots, 128, 2.0 ** -8)
            rest = [t for t in range(c.T) if t not in own]
            assert ((got.cpu().double() - ref).abs() <= to)[rest].all()
            fin = torch.isfinite(rl)
            fin[own] = False
            assert ((lse.cpu().double() - rl).abs() <= tl)[fin].all()
            if lens[0] == 0:
                assert (got[1] == 0).all() and (lse[1] == -math.inf).all()


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("Hq,n", [(1, 5), (8, 9), (8, 40)])    # up to 32, 128 and more rows
@pytest.mark.parametrize("lens", [[0, 40], [61, 0], [250, 130]])
def test_attention_values_that_are_not_finite_reach_only_the_rows_that_see_them(dtype, Hq, n, lens):
    c = AttnCase(lens, [n, n], Hq, 1, 64, 16, "nhd", dtype, "random", seed=n)
    w = torch.uint8 if dtype == E4M3 else torch.int16
    for j in (1, n - 1):            # tokens that see themselves and that no other sees
        for r in range(2):
            p = lens[r] + j
            bad = torch.full((1, 64), math.nan).to(dtype)
            if dtype == BF16:
                bad[:, ::2] = -math.inf
            for x in (c.k, c.v):
                x.view(w)[int(c.table[r, p // 16]), p % 16] = bad.view(w).to(DEV)
            for i in range(n):
                if i != j:
                    c.tree[c.cu[r] + i, j // 32] &= ~(1 << (j % 32))
                    c.sees[r][i, p] = False
    c.run()
    own = [c.cu[r] + j for r in range(2) for j in (1, n - 1)]
    assert torch.isnan(c.out[own].float()).any(-1).all()
    rest = [t for t in range(c.T) if t not in own]
    for r in range(2):              # without their rows the oracle has nothing that is not finite
        for j in (1, n - 1):
            c.sees[r][j] = False
    ref, rl, mag, dots = so.attention(c.q, c.lens, c.cu, c.keys, c.vals, c.sees, c.scale, c.ks, c.vs, dtype == E4M3)
    to, tl = so.attention_tolerance(ref, rl, mag, dots, 64, 2.0 ** -11 if dtype == E4M3 else 2.0 ** -8)
    assert ((c.out.cpu().double() - ref).abs() <= to)[rest].all()
    fin = torch.isfinite(rl)
    fin[own] = False
    assert ((c.lse.cpu().double() - rl).abs() <= tl)[fin].all()


@pytest.mark.parametrize("Hq,n,D,page,dtype", [
    (8, 2, 128, 16, BF16), (8, 2, 64, 24, BF16), (8, 2, 128, 16, E4M3), (8, 2, 64, 24, E4M3), (16, 2, 128, 7, BF16),
    (32, 10, 128, 16, BF16), (32, 10, 64, 24, E4M3), (32, 40, 128, 16, BF16), (32, 40, 64, 12, E4M3)])
def test_attention_of_many_tiles_in_a_row(Hq, n, D, page, dtype):
    # 8 key heads of 25,000 keys in all: every SM goes through its rings several times
    AttnCase([6000, 300, 7001, 5500, 6200], [n, 1, n, n, n - 1], Hq, 8, D, page, "nhd", dtype, None, seed=n + D).run().check()


def test_attention_of_as_many_requests_as_there_may_be_and_of_many_heads():
    rng = random.Random(8)
    R = sgq.SGQ_MAX_REQUESTS
    AttnCase([rng.randint(0, 9) for _ in range(R)], [rng.randint(0, 1) for _ in range(R)], 2, 1, 64, 4, seed=8).run().check()
    AttnCase([33, 2], [2, 1], 128, 64, 64, 8, seed=9).run().check()
    AttnCase([150], [2], 300, 1, 128, 16, seed=10).run().check()    # one key head for 300


FIRST_CALL = '''
import torch
import __graft_entry__ as g
from activation_sparse_quantized_b200 import sgq
torch.cuda.set_device(0)
launched = []
real = {n: getattr(sgq, n) for n in ("sgq_cache_plan", "sgq_cache_write", "sgq_tree_attn", "sgq_residual_norm")}
def captured(name):
    def call(*a):
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            real[name](*a)
        graph.replay()
        launched.append((name, graph))
    return call
for n in real:
    setattr(sgq, n, captured(n))
g.smoke_step("cuda:0")
assert len(launched) == 4
'''


def test_first_call_of_a_process_may_be_captured():
    subprocess.run([sys.executable, "-c", FIRST_CALL], check=True, timeout=120,
                   cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def test_attention_workspace_of_16_byte_alignment_and_shared_by_two_graphs():
    cs = [AttnCase([900, 20], [n, 2], 8, 2, 64, 16, seed=n) for n in (3, 40)]
    need = max(c.ws.numel() for c in cs)
    ws = torch.empty(need + 4, dtype=torch.int32, device=DEV)[4:]
    assert ws.data_ptr() % 32 == 16
    args, graphs = [c.args(workspace=ws) for c in cs], []
    torch.cuda.synchronize()
    for a in args:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            sgq.sgq_tree_attn(**a)
    for g in graphs * 2:            # one after the other on one stream
        g.replay()
    torch.cuda.synchronize()
    for c in cs:
        c.check()


def test_attention_pages_out_of_range_are_masked_and_flagged():
    for dtype in (BF16, E4M3):
        c = AttnCase([100, 70], [3, 2], 4, 2, 64, 16, "nhd", dtype, None, seed=2)
        c.table[0, 2], c.table[1, 0] = c.pages + 5, -3
        c.sees[0][:, 32:48] = False
        c.sees[1][:, 0:16] = False
        c.run().check(status=2)


def test_attention_counts_out_of_range_are_clamped_and_flagged():
    c = AttnCase([20, 30], [3, 2], 4, 2, 64, 16, "nhd", BF16, None, seed=2)
    c.run(lens=i32([-5, 30]))
    assert c.status.item() == 4
    c.status.zero_()
    c.run(lens=i32([20, 1 << 30]))
    assert c.status.item() & 4
    c.status.zero_()
    c.run(cu_new=i32([0, 3, 99]))
    assert c.status.item() == 4
    c.status.zero_()
    c.run(cu_new=i32([0, 4, 2]))
    assert c.status.item() == 4
    c.status.zero_()
    c.run().check()             # the context is as good as before


def test_attention_peaked_and_extreme_scores():
    AttnCase([500], [4], 8, 2, 128, 16, "nhd", BF16, None, seed=1, q_scale=40.0).run().check()
    AttnCase([500], [4], 8, 2, 128, 16, "nhd", E4M3, None, seed=1, q_scale=40.0).run().check()
    for Hq, n, dtype in ((4, 2, BF16), (4, 2, E4M3), (8, 9, BF16), (8, 40, BF16), (8, 9, E4M3)):   # negative and zero scales
        for scale in (-0.3, 0.0):
            c = AttnCase([300], [n], Hq, 1, 64, 16, "nhd", dtype, "random", seed=n)
            c.scale = scale
            c.run().check()
    for big in (1e30, 1e-30):       # q far outside fp16, scale bringing the scores back
        c = AttnCase([130], [2], 4, 1, 64, 16, "nhd", E4M3, None, seed=1)
        c.q = (c.q.float() * big).to(BF16)
        c.scale = c.scale / big
        c.run().check()


def test_attention_strides_streams_and_graphs():
    c = AttnCase([200, 77], [5, 2], 8, 2, 128, 16, "hnd", BF16, "random", seed=6)
    wide_q = torch.full((c.T, 8 * 128 + 64), math.nan, dtype=BF16, device=DEV)
    wide_q[:, :1024] = c.q.view(c.T, 1024).to(DEV)
    wide_o = torch.full((c.T, 8 * 128 + 24), 4.0, dtype=BF16, device=DEV)
    side = torch.cuda.Stream()
    a = c.args(q=wide_q, ld_q=wide_q.shape[1], out=wide_o, ld_out=wide_o.shape[1])
    torch.cuda.synchronize()
    sgq.sgq_tree_attn(**a, stream=side)
    side.synchronize()
    c.out = wide_o[:, :1024].reshape(c.T, 8, 128)
    c.check()
    assert (wide_o[:, 1024:] == 4.0).all()
    # captured once, replayed on other lengths and pages (device data)
    c.out = torch.full((c.T, 8, 128), 9.0, dtype=BF16, device=DEV)
    a = c.args()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sgq.sgq_tree_attn(**a)
    for lens in ([200, 77], [3, 130], [0, 0]):
        d = AttnCase(lens, [5, 2], 8, 2, 128, 16, "hnd", BF16, "random", seed=sum(lens))
        n = min(d.table.shape[1], c.ld)
        m = d.pages
        a["table"].fill_(-1)
        a["table"][:, :n] = d.table[:, :n].to(DEV)
        a["cache"].k[:m], a["cache"].v[:m] = d.k[:a["cache"].k.shape[0]], d.v[:a["cache"].k.shape[0]]
        a["lens"].copy_(i32(lens))
        a["q"].copy_(d.q.to(DEV))
        a["tree"].copy_(d.words_tensor())
        g.replay()
        torch.cuda.synchronize()
        d.out, d.lse, d.status = a["out"], a["lse"], a["status"]
        d.check()


def test_attention_two_streams_with_their_own_workspaces():
    cs = [AttnCase([900 + 50 * i], [4], 8, 2, 128, 16, seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cs]
    args = [c.args() for c in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, a in zip(streams, args):
            sgq.sgq_tree_attn(**a, stream=s)
    torch.cuda.synchronize()
    for c in cs:
        c.check()


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_attention_and_store_beyond_32_bit_offsets(dtype):
    # a cache of which the used pages lie beyond 2^31 elements and 2^32 bytes
    Hkv, D, page = 1, 128, 16
    pages = (2 ** 31 // (page * Hkv * D) + 64) * (1 if dtype == BF16 else 2)
    k, v = (torch.empty(pages, page, Hkv, D, dtype=dtype, device=DEV) for _ in range(2))
    c = AttnCase([150], [3], 2, Hkv, D, page, "nhd", dtype, None, seed=5)
    far = pages - 40
    w = torch.uint8 if dtype == E4M3 else torch.int16
    k.view(w)[far:far + c.pages], v.view(w)[far:far + c.pages] = c.k.view(w), c.v.view(w)
    c.table = torch.where(c.table >= 0, c.table + far, c.table)
    x = torch.randn(3, Hkv * D, device=DEV).to(BF16)
    slots = torch.tensor([(int(c.table[0, (150 + i) // page]) * page + (150 + i) % page) for i in range(3)], device=DEV)
    cache = sgq.Cache(k, v, c.ks, c.vs)
    sgq.sgq_cache_write(None, 0, x, Hkv * D, x, Hkv * D, 3, None, 0, None, None, 0, slots, None, 0, cache)
    torch.cuda.synchronize()
    for i in range(3):
        for t, to, s in ((k, c.keys, c.ks), (v, c.vals, c.vs)):
            row = t[int(slots[i]) // page, int(slots[i]) % page].float().cpu()
            assert ((row.double() - x[i].cpu().double() / s).abs() <=
                    so.stored_tolerance(x[i].cpu().double() / s, x[i].cpu().double().abs() / s, dtype)).all()
            to[0][150 + i] = row.double()
    c.k, c.v = k, v
    c.run(cache=cache, table=c.table.to(DEV)).check()


# ---------------------------------------------------------------------------
# Norm.
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("B,H", [(1, 8), (1, 4096), (3, 264), (16, 5120), (2, 8200), (2, 16392), (1, 32768), (300, 1024)])
@pytest.mark.parametrize("at,rt,wt", [(F32, F32, BF16), (BF16, F32, F32), (BF16, BF16, BF16), (F32, BF16, F32)])
@pytest.mark.parametrize("post,gate", [(False, None), (True, None), (False, "channel"), (True, "row")])
def test_norm(B, H, at, rt, wt, post, gate):
    g = torch.Generator().manual_seed(B + H)
    rn = lambda *s: torch.randn(*s, generator=g)
    pad = 16
    a, r = rn(B, H + pad).to(at), (rn(B, H + pad) * 2).to(rt)
    wp, wx = (rn(H) * 0.3).to(wt) if post else None, (rn(H) * 0.3).to(wt)
    gt = None if gate is None else (rn(H) if gate == "channel" else rn(B, H + 8)).to(wt)
    eps, off, scale = 1e-5, 1.0, 0.75
    ro = torch.full((B, H + 8), 3.0, dtype=rt, device=DEV)
    x = torch.full((B, H + 8), 3.0, dtype=BF16, device=DEV)
    dv = lambda t: None if t is None else t.to(DEV)
    sgq.sgq_residual_norm(dv(a), H + pad, dv(wp), dv(gt), 0 if gate != "row" else H + 8, scale, dv(r), H + pad, ro, H + 8,
                          dv(wx), off, x, H + 8, B, H, eps)
    torch.cuda.synchronize()
    r64, x64, tol, f = so.norm(a[:, :H], wp, None if gt is None else gt[..., :H], scale, r[:, :H], wx, off, eps)
    st = so.HALF_STEP[rt]
    assert ((ro[:, :H].cpu().double() - r64).abs() <= tol + st * (r64.abs() + tol)).all()
    tx = f.abs() * tol + 2.0 ** -17 * x64.abs()
    assert ((x[:, :H].cpu().double() - x64).abs() <= tx + 2.0 ** -8 * (x64.abs() + tx)).all()
    assert (ro[:, H:] == 3.0).all() and (x[:, H:] == 3.0).all()


def test_norm_in_place_without_a_block_without_an_x_and_zero_rows():
    H = 1024
    r = torch.randn(5, H, device=DEV)
    r[2] = 0
    w = torch.randn(H, device=DEV).to(BF16)
    x = torch.empty(5, H, dtype=BF16, device=DEV)
    keep = r.clone()
    sgq.sgq_residual_norm(None, 0, None, None, 0, 1.0, r, H, None, 0, w, 0.0, x, H, 5, H, 0.5)       # the first norm
    torch.cuda.synchronize()
    _, x64, _, _ = so.norm(None, None, None, 1.0, r.cpu(), w.cpu(), 0.0, 0.5)
    assert torch.equal(r, keep) and ((x.cpu().double() - x64).abs() <= (2.0 ** -8 + 2.0 ** -16) * x64.abs()).all()
    a = torch.randn(5, H, device=DEV)
    a[1] = 0                                                                                          # a zero block through its norm
    sgq.sgq_residual_norm(a, H, w, None, 0, 2.0, r, H, r, H, None, 0.0, None, 0, 5, H, 1e-6)         # in place, no x
    torch.cuda.synchronize()
    r64, _, tol, _ = so.norm(a.cpu(), w.cpu(), None, 2.0, keep.cpu(), None, 0.0, 1e-6)
    assert ((r.cpu().double() - r64).abs() <= tol + 2.0 ** -24 * r64.abs()).all() and torch.equal(r[1], keep[1])


def test_norm_in_a_graph_on_a_side_stream():
    H = 4096
    a, r, w = torch.randn(1, H, device=DEV), torch.randn(1, H, device=DEV), torch.ones(H, device=DEV)
    x = torch.empty(1, H, dtype=BF16, device=DEV)
    g = torch.cuda.CUDAGraph()
    r0 = r.clone()
    with torch.cuda.graph(g):
        for _ in range(3):
            sgq.sgq_residual_norm(a, H, None, None, 0, 1.0, r, H, r, H, w, 0.0, x, H, 1, H, 1e-6)
    g.replay()
    torch.cuda.synchronize()
    want = r0.double() + 3 * a.double()
    assert ((r.double() - want).abs() <= 3 * 2.0 ** -24 * (r0.abs() + 3 * a.abs()).double()).all()


# ---------------------------------------------------------------------------
# Together: two steps of one layer's attention half, as a decoder runs them.
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_a_step_together(dtype):
    g = torch.Generator().manual_seed(11)
    hidden, Hq, Hkv, D, page, group = 256, 4, 2, 64, 8, 64
    R, ld, pages, rope_len = 3, 12, 40, 128
    N = (Hq + 2 * Hkv) * D
    W = [(torch.randn(n, k, generator=g) * 0.1).to(torch.float16) for n, k in ((N, hidden), (hidden, Hq * D))]
    packed = []
    for w in W:
        qw, sz = sgq.alloc_packed(*w.shape, group)
        sgq.sgq_pack(w.to(DEV), *w.shape, group, qw, sz)
        packed.append((qw, sz))
    rope = rope_table(rope_len, D)
    w_pre, w_post = (1 + 0.1 * torch.randn(hidden, generator=g)).to(BF16), (1 + 0.1 * torch.randn(hidden, generator=g)).to(BF16)
    k, v = make_cache(pages, page, Hkv, D, "hnd", dtype, math.nan)
    ks, vs = (0.25, 0.25) if dtype == E4M3 else (1.0, 1.0)
    cache = sgq.Cache(k, v, ks, vs)
    table, held = torch.full((R, ld), -1, dtype=torch.int32, device=DEV), i32([0] * R)
    free, count = torch.randperm(pages, generator=g).int().to(DEV), i32([pages])
    status = status_word()
    lens, keys, vals = [0, 0, 0], [[] for _ in range(R)], [[] for _ in range(R)]
    for news, chain in (([9, 3, 4], True), ([4, 0, 8], False)):
        T, rows = sum(news), 16
        depth = None if chain else [0, 1, 1, 2] + [0, 1, 2, 2, 3, 1, 2, 3]
        up = None if chain else [[-1, 0, 0, 1], [], [-1, 0, 1, 1, 2, 0, 5, 6]]
        d_lens = i32(lens)
        cu, slots = i32([0] * (R + 1)), torch.full((rows,), -1, dtype=torch.int64, device=DEV)
        pos, req = i32([0] * rows), i32([0] * rows)
        sgq.sgq_cache_plan(d_lens, i32(news), R, page, pages, table, ld, held, held, free, count, count,
                           None if depth is None else i32(depth + [0] * (rows - T)), rows, cu, slots, pos, req, status)
        resid = torch.randn(rows, hidden, generator=g).to(DEV)
        r0 = resid.clone()
        x = torch.empty(rows, hidden, dtype=BF16, device=DEV)
        sgq.sgq_residual_norm(None, 0, None, None, 0, 1.0, resid, hidden, None, 0, w_pre.to(DEV), 0.0, x, hidden, rows, hidden, 1e-6)
        qkv, y32 = torch.empty(rows, N, dtype=BF16, device=DEV), torch.empty(rows, N, device=DEV)
        sgq.sgq_gemv_dense(*packed[0], N, hidden, group, x, rows, qkv, y32, sgq.alloc_workspace(N, hidden, rows), status)
        q = torch.empty(rows, Hq * D, dtype=BF16, device=DEV)
        sgq.sgq_cache_write(qkv, N, qkv[:, Hq * D:], N, qkv[:, (Hq + Hkv) * D:], N, rows, cu[R:], Hq, pos, rope.to(DEV), rope_len,
                            slots, q, Hq * D, cache, status)
        tree = None
        if not chain:
            bits = []
            for p in up:
                for i in range(len(p)):
                    b, j = 0, i
                    while j >= 0:
                        b, j = b | 1 << j, p[j]
                    bits.append(b)
            tree = i32(bits + [0] * (rows - T)).view(rows, 1)
        att, lse = torch.empty(rows, Hq * D, dtype=BF16, device=DEV), torch.empty(rows, Hq, device=DEV)
        ws = sgq.alloc_tree_attn_workspace(rows, R, Hq, Hkv, D)
        sgq.sgq_tree_attn(q, Hq * D, rows, R, Hq, d_lens, cu, table, ld, cache, tree, 1, D ** -0.5, att, Hq * D, lse, ws, status)
        o, o32 = torch.empty(rows, hidden, dtype=BF16, device=DEV), torch.empty(rows, hidden, device=DEV)
        att[T:] = 0
        sgq.sgq_gemv_dense(*packed[1], hidden, Hq * D, group, att, rows, o, o32, sgq.alloc_workspace(hidden, Hq * D, rows), status)
        sgq.sgq_residual_norm(o32, hidden, w_post.to(DEV), None, 0, 1.0, resid, hidden, resid, hidden, w_pre.to(DEV), 0.0, x, hidden,
                              rows, hidden, 1e-6)
        torch.cuda.synchronize()
        assert status.item() == 0
        # each operator against its definition on the values it was given
        want = so.plan(lens, news, page, pages, [[0] * ld] * R, ld, [ld] * R, [0] * pages, 0, depth, rows)
        assert cu.tolist() == want[0] and pos.tolist()[:T] == want[2] and req.tolist()[:T] == want[3]
        heads = qkv[:T].cpu().double().view(T, -1, D)
        rot, mag = so.rotate(heads[:, :Hq + Hkv], rope, pos[:T].cpu())
        assert ((q[:T].cpu().double().view(T, Hq, D) - rot[:, :Hq]).abs() <= so.stored_tolerance(rot[:, :Hq], mag[:, :Hq], BF16)).all()
        at = slots[:T].cpu()
        assert len(set(at.tolist())) == T and (at >= 0).all()
        kk, vv = (t[(at // page).to(DEV), (at % page).to(DEV)].float().cpu().double() for t in (k, v))
        kr = rot[:, Hq:] / ks
        assert ((kk - kr).abs() <= so.stored_tolerance(kr, (mag[:, Hq:] + rot[:, Hq:].abs()) / ks, dtype)).all()
        vr = heads[:, Hq + Hkv:] / vs
        assert ((vv - vr).abs() <= so.stored_tolerance(vr, vr.abs() if dtype == E4M3 else 0 * vr, dtype)).all()
        sees, b = [], 0
        for r in range(R):
            for i in range(news[r]):
                keys[r].append(kk[b + i])
                vals[r].append(vv[b + i])
            see = torch.ones(news[r], len(keys[r]), dtype=torch.bool)
            for i in range(news[r]):
                for j in range(news[r]):
                    see[i, lens[r] + j] = j <= i if chain else bool(bits[b + i] >> j & 1)
            sees.append(see)
            b += news[r]
        ref, rl, mg, dots = so.attention(q[:T].cpu().view(T, Hq, D), lens, cu.tolist(), [torch.stack(z) for z in keys],
                                         [torch.stack(z) for z in vals], sees, D ** -0.5, ks, vs, dtype == E4M3)
        to, tl = so.attention_tolerance(ref, rl, mg, dots, D, 2.0 ** -11 if dtype == E4M3 else 2.0 ** -8)
        assert ((att[:T].cpu().double().view(T, Hq, D) - ref).abs() <= to).all() and ((lse[:T].cpu().double() - rl).abs() <= tl).all()
        r64, x64, tol, f = so.norm(o32.cpu(), w_post, None, 1.0, r0.cpu(), w_pre, 0.0, 1e-6)
        assert ((resid.cpu().double() - r64).abs() <= tol + 2.0 ** -24 * r64.abs()).all()
        tx = f.abs() * tol + 2.0 ** -17 * x64.abs()
        assert ((x.cpu().double() - x64).abs() <= tx + 2.0 ** -8 * (x64.abs() + tx)).all()
        # the chain is accepted whole; of the tree, its first path: what was drafted behind it is dropped
        if chain:
            lens = [l + n for l, n in zip(lens, news)]
