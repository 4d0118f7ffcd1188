"""The step entry points where sums, references and hand-offs are stretched:
maxima that grow along a run, weights far below the largest, scores and queries
at the ends of their types, many tokens, long runs, waits that run out. Against
the fp64 definitions (step_oracle), as in test_gpu_step."""
import math

import pytest
import torch

import step_oracle as so
from activation_sparse_quantized_b200 import build, sgq
from test_gpu_step import AttnCase, check_plan, i32, make_cache, plan_case, rope_table, run_plan, status_word
from test_gpu_step import test_write as check_write

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


class Attn(AttnCase):
    """An AttnCase whose keys and values can be put in place, checked a key head at a time."""

    def put(self, r, keys=None, vals=None):
        """Keys, values [L, Hkv, D] of request r, rounded to the cache's type."""
        w = torch.uint8 if self.k.dtype == E4M3 else torch.int16
        p = torch.arange(self.lens[r] + self.news[r])
        at = self.table[r].long()[p // self.page].to(DEV), (p % self.page).to(DEV)
        for x, y, to in ((self.k, keys, self.keys), (self.v, vals, self.vals)):
            if y is not None:
                y = y.to(self.k.dtype)
                x.view(w)[at] = y.view(w).to(DEV)
                to[r] = y.to(F32).double()

    def expected(self):
        f8 = self.k.dtype == E4M3
        out, lse, mag, dots = so.attention_by_head(self.q, self.cu, self.keys, self.vals, self.sees, self.scale, self.ks, self.vs, f8)
        return out, lse, *so.attention_tolerance(out, lse, mag, dots, self.D, 2.0 ** -11 if f8 else 2.0 ** -8)

    def check(self, status=0, rows=None):
        assert self.status.item() == status
        out, lse, to, tl = self.expected()
        rows = list(range(self.cu[-1])) if rows is None else rows
        d = ((self.out.cpu().double() - out).abs() / to)[rows]
        assert (d <= 1).all(), float(d.nan_to_num(math.inf).max())
        assert ((self.lse.cpu().double() - lse).abs() <= tl)[rows].all()
        n = self.cu[-1]
        assert (self.out[n:] == 9.0).all() and (self.lse[n:] == 9.0).all()


# ---- maxima that grow along a run ----

@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,n", [(16, 2), (32, 20), (32, 40)])   # tiles of 32, 128 and 256 rows
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_attention_maxima_that_outgrow_their_reference(dtype, D, Hq, n, sign):
    # Eight key heads of 20,000 keys are eight tiles and more in a row on every SM. The
    # scores climb by 100 binary orders in 1100 keys and fall back, at another pace and
    # from another place for each row and head, so that what is summed so far is scaled
    # down many times over, and the top of every climb counts in the result.
    L, Hkv = 20000, 8
    c = Attn([L], [n], Hq, Hkv, D, 32, "nhd", dtype, None, seed=n + D)
    g = torch.Generator().manual_seed(n)
    ones = torch.ones(D)
    climb = ((torch.arange(L + n)[:, None] + 137 * torch.arange(Hkv)) % 1100) / 1100 * 100
    unit = math.log(2) / (D * c.scale * c.ks)              # a key of this, times ones, is one binary order
    c.put(0, (climb * unit)[..., None] * ones + 0.05 * torch.randn(L + n, Hkv, D, generator=g))
    pace = 0.3 + torch.rand(n, Hq, 1, generator=g)
    c.q = (sign * pace * ones).to(BF16)
    c.scale *= sign
    c.run().check()
    first = c.out.clone(), c.lse.clone()
    for _ in range(4):
        c.run()
        assert torch.equal(c.out, first[0]) and torch.equal(c.lse, first[1])


# ---- scores of any size ----

@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("Hq,n", [(4, 2), (8, 9), (8, 40)])
@pytest.mark.parametrize("power", [12, 26, 34, 60, 110])
def test_attention_scores_far_beyond_the_exponents_range(dtype, Hq, n, power):
    # Small whole numbers times powers of two: every product and sum is exact, scores
    # differ by 2^power times a whole number over D or not at all, and a row's result is
    # the mean of the values at its highest score. (D = 64: scale 1/8 is exact too.)
    g = torch.Generator().manual_seed(power + n)
    c = Attn([1500, 200], [n, n], Hq, 1, 64, 16, "nhd", dtype, None, seed=n)
    for r in range(2):
        c.put(r, torch.randint(-3, 4, (c.lens[r] + n, 1, 64), generator=g).float())
    c.q = (torch.randint(-3, 4, (2 * n, Hq, 64), generator=g) * 2.0 ** power).to(BF16)
    c.ks = 1.0
    c.run()
    assert c.status.item() == 0
    out, lse, _, _ = so.attention_by_head(c.q, c.cu, c.keys, c.vals, c.sees, c.scale, c.ks, c.vs)
    got = c.out.cpu().double()
    # a weight's and the result's rounding, and the sums', as in attention_tolerance without a score's error
    most = max(float(v.abs().max()) for v in c.vals) * c.vs
    to = ((2.0 ** -11 if dtype == E4M3 else 2.0 ** -8) + 2.0 ** -14) * most
    assert ((got - out).abs() <= to + 2.0 ** -8 * (out.abs() + to)).all()
    assert ((c.lse.cpu().double() - lse).abs() <= 2.0 ** -20 + 8 * so.U * lse.abs()).all()


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("Hq,n", [(4, 2), (8, 9), (8, 40)])
def test_attention_rows_whose_scores_leave_fp32_are_not_finite(dtype, Hq, n):
    # Products of 9 x 64 x 2^117 and a scale of 8: 2^129 and more, in base 2. Row 0's are all
    # above the range, row 1's all below it; the others are ordinary. The context is cut into
    # parts, one key head to many SMs.
    c = Attn([20000, 200], [n, n], Hq, 1, 64, 16, "nhd", dtype, None, seed=n)
    keys = [k.clone() for k in c.keys]
    for r in range(2):
        keys[r][:] = 3.0
        c.put(r, keys[r])
    c.q = c.q * 2.0 ** -10
    c.q[0], c.q[1] = 3 * 2.0 ** 117, -3 * 2.0 ** 117
    c.scale = 8.0
    c.run()
    assert torch.isnan(c.out[:2].float()).all() and not torch.isfinite(c.lse[:2]).any()
    c.q[:2] = 0                     # the oracle needs scores there
    c.check(rows=list(range(2, c.cu[-1])))


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("Hq,n", [(4, 2), (8, 9), (8, 40)])
@pytest.mark.parametrize("scale", [0.0, 1e-38, -3e-39, 1e-35])
def test_attention_scales_next_to_zero(dtype, Hq, n, scale):
    # the products reach 2^117 (q 2^57 times k up to 2^53; 8-bit k up to 8 and q 2^110)
    g = torch.Generator().manual_seed(n)
    c = Attn([300], [n], Hq, 1, 64, 16, "nhd", dtype, None, seed=n)
    c.put(0, torch.randint(-7, 8, (300 + n, 1, 64), generator=g).float() * (2.0 ** 50 if dtype == BF16 else 1.0))
    c.q = (torch.randint(-7, 8, (n, Hq, 64), generator=g) * 2.0 ** (57 if dtype == BF16 else 107)).to(BF16)
    c.scale = scale
    c.run().check()


# ---- weights far below the largest ----

def share(c, R):
    """The one request of c, of one new token, R times over the same pages, with a q each."""
    c.lens, c.news, c.cu, c.T = c.lens * R, c.news * R, list(range(R + 1)), R
    c.table = c.table.expand(R, -1).contiguous()
    c.keys, c.vals, c.sees = c.keys * R, c.vals * R, c.sees * R
    c.ws = sgq.alloc_tree_attn_workspace(R, R, c.Hq, c.Hkv, c.D)
    c.out = torch.full((R, c.Hq, c.D), 9.0, dtype=BF16, device=DEV)
    c.lse = torch.full((R, c.Hq), 9.0, device=DEV)
    return c


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_a_long_tail_below_one_key_whose_value_is_zero(dtype, D):
    # One key, the first, 10 to 20 nats above 60,000 others: its value is zero, so the
    # result is the others'. Two requests a SM, so that most are not cut into parts
    # (each part has a reference of its own).
    L, R = 60000, 2 * torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator().manual_seed(D)
    c = Attn([L], [1], 1, 1, D, 64, "nhd", dtype, None, seed=D)
    keys = -1 + 0.0625 * torch.randint(0, 2, (L + 1, 1, D), generator=g)
    vals = 1 + 0.25 * torch.randint(-2, 3, (L + 1, 1, D), generator=g)
    keys[0], vals[0] = 1.0, 0.0
    c.put(0, keys, vals)
    c = share(c, R)
    nats = 10 + 10 * torch.arange(R) / (R - 1)                     # the distance to the lowest key
    c.q = (nats / (2 * D * c.scale * c.ks))[:, None, None].expand(R, 1, D).to(BF16)
    c.run()
    assert c.status.item() == 0
    out, lse, to, tl = c.expected()
    # The largest weight is 2^7 at least and one below 2^-14 is off by at most 2^-25
    # (fp16's steps), so each of the keys' weights by 2^-32 of the largest.
    low = 1.5 * c.vs * L * 2.0 ** -32 if dtype == E4M3 else 0.0
    assert ((c.out.cpu().double() - out).abs() <= to + low * (1 + 2.0 ** -8)).all()
    assert ((c.lse.cpu().double() - lse).abs() <= tl).all()
    assert low < 0.2 * out.abs().min()                             # the bound says something of every row


# ---- a q that is not finite ----

@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("Hq,n", [(4, 3), (8, 9), (8, 40)])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_attention_rows_of_q_that_are_not_finite(dtype, Hq, n, bad):
    c = Attn([1000, 70], [n, n], Hq, 1, 64, 16, "nhd", dtype, "random", seed=n)
    rows = [0, n - 1, n + 1]
    keys = [k.clone() for k in c.keys]
    for r in range(2):              # one channel's keys are small: products of 448 with them do not overflow
        keys[r][:, :, 5] *= 0.0625
        c.put(r, keys[r])
    for t in rows:
        c.q[t, :, 5] = bad
    c.run()
    assert torch.isnan(c.out[rows].float()).all() and not torch.isfinite(c.lse[rows]).any()
    c.q[rows] = 0                   # the oracle needs numbers there
    c.check(rows=[t for t in range(c.cu[-1]) if t not in rows])


# ---- runs of a second ----

def test_attention_over_contexts_of_two_hundred_million_keys():
    # Two contexts of 2^28 keys a SM, all of them 256 times over the one page there is (table
    # rows may name a page again): each takes about half a second, longer than the limit
    # of a wait for data. One key in 4096 counts, the others are 250 nats below.
    R, page, D, times = 2 * torch.cuda.get_device_properties(0).multi_processor_count, 1 << 20, 64, 256
    g = torch.Generator().manual_seed(1)
    at = torch.arange(0, page, 4096)
    keys, vals = torch.full((page, 1, D), -8.0), torch.ones(page, 1, D)
    keys[at], vals[at] = 0.3 * torch.randn(len(at), 1, D, generator=g), torch.randn(len(at), 1, D, generator=g)
    keys, vals = keys.to(BF16), vals.to(BF16)
    q = (4 + 0.25 * torch.randn(R, 1, D, generator=g)).to(BF16)
    out, lse, status = torch.zeros(R, 1, D, dtype=BF16, device=DEV), torch.zeros(R, 1, device=DEV), i32([0])
    sgq.sgq_tree_attn(q.to(DEV), D, R, R, 1, i32([times * page - 1] * R), i32(list(range(R + 1))),
                      torch.zeros(R, times, dtype=torch.int32, device=DEV), times,
                      sgq.Cache(keys[None].to(DEV), vals[None].to(DEV)), None, 0, D ** -0.5, out, D, lse,
                      sgq.alloc_tree_attn_workspace(R, R, 1, 1, D), status)
    torch.cuda.synchronize()
    assert status.item() == 0
    k, v = keys[at].float().double(), vals[at].float().double()
    ref, rl, mag, dots = so.attention_by_head(q, list(range(R + 1)), [k] * R, [v] * R, [torch.ones(1, len(at), dtype=torch.bool)] * R, D ** -0.5)
    to, tl = so.attention_tolerance(ref, rl, mag, dots, D, 2.0 ** -8)
    # 2^16 weights that are not zero are added one after the other, each time with one
    # rounding of the sum so far: by half a step in l, by a whole one in the tensor core.
    long = 2.0 ** 16 * so.U
    assert ((out.cpu().double() - ref).abs() <= to + 3 * long * mag).all()
    assert ((lse.cpu().double() - rl - math.log(times)).abs() <= tl + long).all()


# ---- waits that run out ----

@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("page", [16, 3])                          # bulk copies, and others
@pytest.mark.parametrize("Hq,n", [(4, 2), (8, 9), (8, 40)])
def test_attention_wait_limits_set_timeout_and_the_context_survives(dtype, page, Hq, n):
    # Host-side injection: the kernel's issuer never passes scores on, so the waits for them
    # run out. The call returns, and the next one, on the same workspace, is right.
    c = Attn([3000] + [40] * 30, [n] * 31, Hq, 1, 128, page, "nhd", dtype, "random", seed=n, rows=3)
    a = c.args()
    sgq.sgq_debug_tree_attn_withhold(**a)
    torch.cuda.synchronize()
    assert c.status.item() == sgq.SGQ_STATUS_TIMEOUT
    n_rows = c.cu[-1]
    assert (c.out[n_rows:] == 9.0).all() and (c.lse[n_rows:] == 9.0).all()
    c.status.zero_()
    c.run().check()


# ---- a prompt's chunk ----

@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("lens,news", [([0], [513]), ([777], [300]), ([50, 1030, 0, 3], [1, 1, 400, 1])])
def test_attention_of_a_long_chain(dtype, lens, news):
    Attn(lens, news, 8, 2, 128, 16, "hnd", dtype, None, seed=sum(news), rows=1).run().check()


# ---- the store of many tokens ----

@pytest.mark.parametrize("T,Hq,Hkv,D,page,layout,dtype,rope", [
    (296, 32, 8, 128, 16, "nhd", BF16, True), (700, 8, 2, 64, 24, "hnd", BF16, True), (513, 64, 8, 128, 64, "hnd", E4M3, True),
    (1000, 6, 3, 64, 16, "nhd", E4M3, False), (301, 0, 2, 128, 8, "nhd", BF16, False), (600, 7, 1, 128, 7, "nhd", E4M3, True),
    (299, 200, 40, 64, 16, "hnd", BF16, True)])
def test_write_of_many_tokens(T, Hq, Hkv, D, page, layout, dtype, rope):
    # several heads a thread, from 2 tokens a SM on
    check_write(T, Hq, Hkv, D, page, layout, dtype, rope)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_write_of_many_tokens_skips_flags_and_writes_q_in_place(dtype):
    # What few tokens and many are told to skip is the same, and the rest too: against calls
    # of 100 rows each (a kernel of one head a thread) on the same values.
    T, Hq, Hkv, D, page = 1000, 8, 2, 64, 16
    pages = T // page + 2
    g = torch.Generator().manual_seed(3)
    qkv = (torch.randn(T, (Hq + 2 * Hkv) * D, generator=g) * 300).to(BF16)
    qkv[5, 7], qkv[400, Hq * D + 3], qkv[401, -1] = math.nan, math.inf, -math.inf
    slots, pos = torch.randperm(pages * page, generator=g)[:T], torch.randint(0, 50, (T,), generator=g, dtype=torch.int32)
    slots[torch.arange(0, T, 9)] = -1
    slots[123], slots[777] = pages * page, -2
    pos[50], pos[600] = 50, -1
    n, ld = 901, qkv.shape[1]
    table, got = rope_table(50, D).to(DEV), []
    for step in (T, 100):
        k, v = make_cache(pages, page, Hkv, D, "nhd", dtype, 5.0)
        cache, st = sgq.Cache(k, v, *((0.7, 1.3) if dtype == E4M3 else (1.0, 1.0))), status_word()
        d, ds, dp = qkv.to(DEV), slots.to(DEV), pos.to(DEV)
        for t in range(0, T, step):
            rows = d[t:t + step]
            sgq.sgq_cache_write(rows, ld, rows[:, Hq * D:], ld, rows[:, (Hq + Hkv) * D:], ld, step, i32([max(0, min(step, n - t))]), Hq,
                                dp[t:], table, 50, ds[t:], rows, ld, cache, st)
        torch.cuda.synchronize()
        assert st.item() == sgq.SGQ_STATUS_BAD_INDEX
        w = torch.uint8 if dtype == E4M3 else torch.int16
        got.append((d.view(torch.int16), k.view(w), v.view(w)))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert torch.equal(got[0][0][n:].cpu(), qkv[n:].view(torch.int16))       # rows behind the count


# ---- padded batches ----

@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("rows", [60, 300])
def test_attention_of_a_batch_padded_behind(dtype, rows):
    # many rows behind the last request: the rows a request has on average, and so the row
    # tile, are not what the requests have
    Attn([500, 0, 33], [3, 1, 2], 8, 2, 128, 16, "nhd", dtype, "random", seed=rows, rows=rows).run().check()


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_attention_of_a_batch_padded_in_front(dtype):
    c = Attn([300, 5], [4, 9], 8, 2, 64, 16, "nhd", dtype, "random", seed=4)
    pad = 5
    c.q = torch.cat([torch.full((pad, 8, 64), math.nan, dtype=BF16), c.q])
    c.tree = torch.cat([torch.full((pad, c.words), 7), c.tree])
    c.T += pad
    out, lse = torch.full((c.T, 8, 64), 9.0, dtype=BF16, device=DEV), torch.full((c.T, 8), 9.0, device=DEV)
    c.ws = sgq.alloc_tree_attn_workspace(c.T, 2, 8, 2, 64)
    c.run(cu_new=i32([t + pad for t in c.cu]), out=out, lse=lse)
    assert (out[:pad] == 9.0).all() and (lse[:pad] == 9.0).all()
    c.q, c.out, c.lse = c.q[pad:], out[pad:], lse[pad:]
    c.check()


# ---- plans of many tokens (a second kernel writes the tokens' rows) ----

@pytest.mark.parametrize("fault", ["short", "len", "new", "held", "wide", "tokens", "count", "page"])
def test_plan_of_many_tokens_with_bad_state_or_too_few_pages(fault):
    lens, news, page, pages, table, held, free, count = plan_case(900, 8, 1, 60, 40, 5, short=fault == "short")
    T, r = sum(news), 333
    if fault == "len":
        lens[r] = -4
    elif fault == "new":
        news[r] = -1
    elif fault == "held":
        held[r] = 0
    elif fault == "wide":
        more = 8 * len(table[0]) + 1 - news[r]
        news[r], T = news[r] + more, T + more
    elif fault == "tokens":
        T -= 4001
    elif fault == "count":
        count = pages + 50
        free = free[:pages] + [0] * (pages - len(free[:pages]))
    elif fault == "page":
        r = next(i for i in range(r, 900) if lens[i] % 8 and news[i])
        table[r][lens[r] // 8] = pages + 3
    assert T > 8192
    depth = [i % 5 for i in range(T + 3)] if fault in ("short", "page") else None
    _, got = run_plan(lens, news, page, pages, table, held, free, count, depth, T, rows=T + 3)
    want = so.plan(lens, news, page, pages, table, len(table[0]), held, free, count, depth, T)
    assert want[-1]
    check_plan(got, want, T)
