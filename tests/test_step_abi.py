"""The step entry points (cache plan and store, tree attention, residual norm):
what they refuse, on the host, before anything is enqueued (no GPU needed), and
the fp64 oracle's own pins."""
import ctypes
import math

import pytest
import torch

import step_oracle as so
from activation_sparse_quantized_b200 import build as sgq_build
from activation_sparse_quantized_b200 import sgq

P, F = ctypes.c_void_p, ctypes.c_float
FAKE, ODD = P(1 << 20), P((1 << 20) + 8)   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    sgq_build.build()
    return sgq.load()


def cache(**kw):
    c = dict(k=1 << 20, v=1 << 21, type=0, page=16, num_pages=64, heads=8, dim=128,
             page_stride=16 * 8 * 128, slot_stride=8 * 128, head_stride=128, k_scale=1.0, v_scale=1.0)
    c.update(kw)
    s = sgq._CacheStruct(*[c[f] for f, _ in sgq._CacheStruct._fields_])
    return ctypes.byref(s)


def attn_args(lib, **kw):
    a = dict(q=FAKE, ld_q=4096, T=16, R=2, Hq=32, lens=FAKE, cu=FAKE, table=FAKE, table_ld=64,
             cache=cache(), tree=FAKE, words=1, scale=F(0.1), out=FAKE, ld_out=4096, lse=None, ws=FAKE,
             wsb=lib.sgq_tree_attn_workspace_bytes(16, 2, 32, 8, 128), status=None, stream=None)
    a.update(kw)
    return list(a.values())


CACHE_FAULTS = [
    (dict(type=1), -11), (dict(type=7), -11), (dict(dim=96), -2), (dict(dim=256), -2), (dict(heads=0), -2),
    (dict(page=0), -2), (dict(num_pages=0), -2), (dict(k=None), -1), (dict(v=None), -1), (dict(k=(1 << 20) + 2), -4),
    (dict(slot_stride=1028), -4), (dict(head_stride=64), -2), (dict(slot_stride=0), -2), (dict(page_stride=-8), -2),
    (dict(page_stride=0), -2), (dict(page_stride=(1 << 38) + 8), -2), (dict(k_scale=0.5), -2), (dict(type=2, k_scale=0.0), -2),
    (dict(type=2, v_scale=math.nan), -2), (dict(type=2, k_scale=math.inf), -2), (dict(type=2, head_stride=136), -4),
]


@pytest.mark.parametrize("fault,code", CACHE_FAULTS, ids=[str(f[0]) for f in CACHE_FAULTS])
def test_cache_descriptions_are_refused(lib, fault, code):
    assert lib.sgq_tree_attn(*attn_args(lib, cache=cache(**fault))) == code
    assert lib.sgq_cache_write(FAKE, 4096, FAKE, 1024, FAKE, 1024, 4, None, 32, None, None, 0, FAKE, FAKE, 4096,
                               cache(**fault), None, None) == code


ATTN_FAULTS = [
    (dict(cache=None), -1), (dict(R=0), -5), (dict(R=8193), -5), (dict(T=0), -2), (dict(Hq=4), -2), (dict(Hq=36), -2),
    (dict(table_ld=0), -2), (dict(table_ld=1 << 27), -2), (dict(words=0), -2), (dict(q=None), -1), (dict(lens=None), -1),
    (dict(cu=None), -1), (dict(table=None), -1), (dict(out=None), -1), (dict(ws=None), -1), (dict(q=ODD), -4),
    (dict(out=ODD), -4), (dict(ws=ODD), -4), (dict(ld_q=4095), -2), (dict(ld_q=4100), -2), (dict(ld_out=64), -2),
    (dict(T=1 << 30), -2), (dict(wsb=1 << 20), -6), (dict(scale=F(math.nan)), -2), (dict(scale=F(math.inf)), -2),
    (dict(scale=F(-2e37)), -2),
]


@pytest.mark.parametrize("fault,code", ATTN_FAULTS, ids=[str(list(f[0])[0]) + str(f[1]) for f in ATTN_FAULTS])
def test_attention_refusals(lib, fault, code):
    assert lib.sgq_tree_attn(*attn_args(lib, **fault)) == code


def test_attention_workspace_sizes(lib):
    ws = lib.sgq_tree_attn_workspace_bytes
    assert ws(16, 2, 32, 8, 128) > 0 and ws(16, 2, 32, 8, 128) % 16 == 0
    assert ws(1, 8192, 8, 8, 64) > 0
    for bad in ((0, 1, 8, 8, 64), (1, 0, 8, 8, 64), (1, 1, 8, 3, 64), (1, 1, 8, 8, 80), (1, 8193, 8, 8, 64)):
        assert ws(*bad) == 0


def test_write_refusals(lib):
    def call(**kw):
        a = dict(q=FAKE, ld_q=6144, k=FAKE, ld_k=6144, v=FAKE, ld_v=6144, T=4, nt=None, Hq=32, pos=FAKE, rope=FAKE,
                 rope_len=100, slots=FAKE, q_out=FAKE, ld_qo=4096, cache=cache(), status=None, stream=None)
        a.update(kw)
        return lib.sgq_cache_write(*a.values())
    assert call(cache=None) == -1 and call(k=None) == -1 and call(v=None) == -1 and call(slots=None) == -1
    assert call(q_out=None) == -1 and call(pos=None) == -1          # a rotation needs positions
    assert call(T=0) == -2 and call(Hq=0) == -2 and call(rope_len=0) == -2
    assert call(ld_q=4088) == -2 and call(ld_k=1020) == -2 and call(ld_v=1032 + 4) == -2 and call(ld_qo=8) == -2
    assert call(k=ODD) == -4 and call(q=ODD) == -4 and call(rope=ODD) == -4 and call(q_out=ODD) == -4


def test_plan_refusals(lib):
    def call(**kw):
        a = dict(lens=FAKE, news=FAKE, R=4, page=16, num_pages=64, table=FAKE, ld=8, held=FAKE, held_out=FAKE, free=FAKE,
                 count=FAKE, count_out=FAKE, depth=None, T=64, cu=FAKE, slots=FAKE, pos=None, req=None, status=None, stream=None)
        a.update(kw)
        return lib.sgq_cache_plan(*a.values())
    assert call(R=0) == -5 and call(R=8193) == -5
    for k in ("page", "num_pages", "ld", "T"):
        assert call(**{k: 0}) == -2
    assert call(ld=1 << 27) == -2 and call(T=(1 << 30) + 1) == -2
    for k in ("lens", "news", "table", "held", "held_out", "free", "count", "count_out", "cu", "slots"):
        assert call(**{k: None}) == -1


def test_norm_refusals(lib):
    def call(**kw):
        a = dict(a=FAKE, ld_a=64, at=0, wp=FAKE, gate=FAKE, ldg=0, scale=F(1), r=FAKE, ldr=64, rt=1, ro=FAKE, ldro=64,
                 wpre=FAKE, wt=0, off=F(0), x=FAKE, ldx=64, B=2, H=64, eps=F(1e-6), stream=None)
        a.update(kw)
        return lib.sgq_residual_norm(*a.values())
    for k in ("at", "rt", "wt"):
        assert call(**{k: 2}) == -11
    assert call(B=0) == -2 and call(H=60) == -2 and call(H=0) == -2 and call(H=32776) == -2
    assert call(eps=F(-1)) == -2 and call(eps=F(math.nan)) == -2
    assert call(r=None) == -1 and call(ro=None) == -1 and call(wpre=None) == -1
    assert call(a=None) == -1                         # a gate or a norm of nothing
    assert call(a=None, wp=None, gate=None, x=None) == -1
    for k in ("a", "wp", "gate", "r", "ro", "wpre", "x"):
        assert call(**{k: ODD}) == -4
    assert call(ld_a=56) == -2 and call(ldr=66) == -2 and call(ldx=68) == -2 and call(ldg=8) == -2 and call(ldro=0) == -2


def test_status_strings(lib):
    assert b"type" in lib.sgq_status_string(-11) and b"unknown" in lib.sgq_status_string(-99)


def test_binding_refuses_types_devices_and_shapes():
    cpu = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError, match="lens"):
        sgq._dev("lens", cpu.float(), torch.int32, 0)
    with pytest.raises(ValueError, match="current device"):
        sgq._dev("lens", cpu, torch.int32, 0)
    assert sgq._dev("tree", None, torch.int32, 0) is None
    with pytest.raises(TypeError, match="resid"):
        sgq._float_type("resid", cpu)
    k = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sgq.Cache(k, k[:2])
    with pytest.raises(ValueError):
        sgq.Cache(k, torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16).transpose(1, 2))   # other strides
    with pytest.raises(TypeError):
        sgq.Cache(k.float(), k.float())
    with pytest.raises(ValueError):
        sgq.Cache(k.transpose(2, 3), k.transpose(2, 3))
    c = sgq.Cache(k, k)
    assert (c.struct.page, c.struct.num_pages, c.struct.heads, c.struct.dim) == (16, 3, 2, 64)
    assert (c.struct.page_stride, c.struct.slot_stride, c.struct.head_stride) == (2048, 128, 64)
    with pytest.raises(ValueError, match="current device"):
        c.on(0)


def test_cache_of_one_page_head_or_slot_takes_any_stride_there():
    one = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    k = one.as_strided((1, 2, 1, 64), (7, 64, 3, 1))
    v = one.as_strided((1, 2, 1, 64), (64, 64, 1, 1))
    c = sgq.Cache(k, v)
    assert (c.struct.page_stride, c.struct.slot_stride, c.struct.head_stride) == (64, 64, 64)


# ---- the oracle's pins ----

def test_oracle_plan_by_hand():
    # pages of 4; request 0 holds 5 tokens in 2 pages and takes 4 more (one new
    # page), request 1 nothing, request 2 is new with 5 (two pages), request 3 wants more than is left
    cu, slots, pos, req, table, held, left, bad = so.plan(
        [5, 3, 0, 1], [4, 0, 5, 9], 4, 10, [[7, 3, -1], [9, -1, -1], [-1] * 3, [8, -1, -1]], 3, [2, 1, 0, 1],
        [0, 1, 2, 4, 0, 0, 0, 0, 0, 0], 4, None, 100)
    assert cu == [0, 4, 4, 9, 18] and left == 1 and held == [3, 1, 2, 1] and bad == {"pages"}
    assert table == [[7, 3, 4], [9, -1, -1], [2, 1, -1], [8, -1, -1]]
    assert slots == [13, 14, 15, 16, 8, 9, 10, 11, 4] + [-1] * 9
    assert pos[:9] == [5, 6, 7, 8, 0, 1, 2, 3, 4] and req == [0] * 4 + [2] * 5 + [3] * 9


def test_oracle_attention_closed_forms():
    # equal scores: the mean of the values seen; one key: its value; none: zero
    q = torch.zeros(3, 2, 64)
    keys, vals = [torch.randn(4, 1, 64).double()], [torch.arange(4.).double()[:, None, None].expand(4, 1, 64)]
    sees = [torch.tensor([[1, 1, 1, 1], [0, 0, 1, 0], [0, 0, 0, 0]]).bool()]
    out, lse, _, _ = so.attention(q, [1], [0, 3], keys, vals, sees, 1.0, 1.0, 2.0)
    assert torch.allclose(out[0], torch.full((2, 64), 3.0).double()) and torch.allclose(out[1], torch.full((2, 64), 4.0).double())
    assert (out[2] == 0).all() and (lse[2] == -math.inf).all()
    assert torch.allclose(lse[0], torch.full((2,), math.log(4.0)).double()) and (lse[1] == 0).all()


def test_oracle_norm_and_rotation_closed_forms():
    # a constant row has rms equal to its magnitude
    r, x, _, _ = so.norm(torch.full((1, 8), -3.0), torch.ones(8), None, 2.0, torch.full((1, 8), 5.0), torch.full((8,), 0.5), 0.0, 0.0)
    assert torch.allclose(r, torch.full((1, 8), 3.0).double()) and torch.allclose(x, torch.full((1, 8), 0.5).double())
    # a quarter turn swaps the halves; it keeps the length
    rope = torch.cat([torch.zeros(1, 4), torch.ones(1, 4)], 1)
    v = torch.arange(8.).double().view(1, 1, 8)
    y, _ = so.rotate(v, rope, torch.zeros(1))
    assert torch.equal(y[0, 0], torch.tensor([-4., -5, -6, -7, 0, 1, 2, 3]).double())
