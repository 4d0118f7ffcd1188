"""The step entry points' binding: what it refuses of tensors, on the host, and the
calls around the entry points (no GPU needed: CPU tensors and a recording library
stand in for the device's)."""
import ctypes

import pytest
import torch

from activation_sparse_quantized_b200 import build as sgq_build
from activation_sparse_quantized_b200 import sgq
from test_step_abi import ATTN_FAULTS, attn_args

I32, I64, F32, BF16, E4M3 = torch.int32, torch.int64, torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    sgq_build.build()
    return sgq.load()


@pytest.mark.parametrize("fault,code", ATTN_FAULTS, ids=[str(list(f[0])[0]) + str(f[1]) for f in ATTN_FAULTS])
def test_the_attention_test_hook_refuses_what_the_entry_point_refuses(lib, fault, code):
    assert lib.sgq_debug_tree_attn_withhold(*attn_args(lib, **fault)) == code


def test_a_number_of_requests_out_of_range_is_called_that(lib):
    assert lib.sgq_tree_attn(*attn_args(lib, R=8193)) == -5
    words = lib.sgq_status_string(-5)
    assert b"requests" in words and str(sgq.SGQ_MAX_REQUESTS).encode() in words and str(sgq.SGQ_MAX_BATCH).encode() in words


@pytest.mark.parametrize("Hq,heads,dim", [(32, 8, 128), (8, 8, 64), (128, 2, 128)])
def test_a_workspace_for_the_largest_step_takes_every_smaller_one(lib, Hq, heads, dim):
    sizes = [1, 2, 5, 16, 40, 64, 300, 8192]
    small = dict(k=1 << 20, v=1 << 21, type=0, page=16, num_pages=64, heads=heads, dim=dim, page_stride=16 * heads * dim,
                 slot_stride=heads * dim, head_stride=dim, k_scale=1.0, v_scale=1.0)
    c = ctypes.byref(sgq._CacheStruct(*[small[f] for f, _ in sgq._CacheStruct._fields_]))
    for T in sizes:
        for R in sizes:
            ws = lib.sgq_tree_attn_workspace_bytes(T, R, Hq, heads, dim)
            for t in sizes[:sizes.index(T) + 1]:
                for r in sizes[:sizes.index(R) + 1]:
                    # no GPU here: a call that passes its checks fails later, for another reason
                    a = attn_args(lib, T=t, R=r, Hq=Hq, ld_q=Hq * dim, ld_out=Hq * dim, cache=c, wsb=ws, status=None)
                    assert ws >= lib.sgq_tree_attn_workspace_bytes(t, r, Hq, heads, dim)
                    if not torch.cuda.is_available():
                        assert lib.sgq_tree_attn(*a) in (-8, -9), (T, R, t, r)


class Recorder:
    """Stands in for the library: takes every call and keeps its arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*a):
            self.calls.append((name, a))
            return 0
        return call


@pytest.fixture(params=["module", "python"])
def calls(request, monkeypatch, lib):
    """The entry points on CPU tensors, checked by the helper module or in Python."""
    rec = Recorder()
    monkeypatch.setattr(sgq, "load", lambda: rec)
    monkeypatch.setattr(sgq, "_current_device", lambda: -1)       # what a CPU tensor's get_device() says
    monkeypatch.setattr(sgq, "_stream", lambda stream, dev=None: 0)
    if request.param == "module":
        from activation_sparse_quantized_b200._tensors import addresses
        monkeypatch.setattr(sgq, "_fast", addresses)
    else:
        monkeypatch.setattr(sgq, "_fast", lambda *a: None)
    return rec.calls


def cache(dtype=BF16, heads=2, dim=64):
    k, v = (torch.zeros(6, 8, heads, dim, dtype=dtype) for _ in range(2))
    return sgq.Cache(k, v)


def plan_args():
    R, ld, pages, T = 3, 4, 6, 10
    z = lambda n, t=I32: torch.zeros(n, dtype=t)
    return dict(lens=z(R), news=z(R), R=R, page=8, num_pages=pages, table=z(R * ld).view(R, ld), table_ld=ld, held=z(R),
                held_out=z(R), free_pages=z(pages), free_count=z(1), free_count_out=z(1), depth=z(4), max_tokens=T, cu_new=z(R + 1),
                slots=z(T, I64), pos=z(T), req=z(T), status=z(1))


def write_args():
    T, Hq, D = 5, 4, 64
    x = torch.zeros(T, (Hq + 4) * D, dtype=BF16)
    z = lambda n, t=I32: torch.zeros(n, dtype=t)
    return dict(q=x, ld_q=x.shape[1], k=x[:, Hq * D:], ld_k=x.shape[1], v=x[:, (Hq + 2) * D:], ld_v=x.shape[1], T=T, n_tokens=z(1),
                Hq=Hq, pos=z(T), rope=z(7 * D, F32), rope_len=7, slots=z(T, I64), q_out=z(T * Hq * D, BF16), ld_qo=Hq * D,
                cache=cache(), status=z(1))


def attn_call_args():
    T, R, Hq, D, ld = 5, 2, 4, 64, 3
    z = lambda n, t=I32: torch.zeros(n, dtype=t)
    return dict(q=z(T * Hq * D, BF16).view(T, Hq, D), ld_q=Hq * D, T=T, R=R, Hq=Hq, lens=z(R), cu_new=z(R + 1),
                table=z(R * ld).view(R, ld), table_ld=ld, cache=cache(), tree=z(T).view(T, 1), tree_words=1, scale=0.1,
                out=z(T * Hq * D, BF16).view(T, Hq * D), ld_out=Hq * D, lse=z(T * Hq, F32).view(T, Hq), workspace=z(4096), status=z(1))


def norm_args():
    B, H = 3, 16
    z = lambda *n, t=BF16: torch.zeros(*n, dtype=t)
    return dict(a=z(B, H, t=F32), ld_a=H, w_post=z(H), gate=z(B, H), ld_gate=H, scale=1.0, resid=z(B, H, t=F32), ld_r=H,
                resid_out=z(B, H, t=F32), ld_ro=H, w_pre=z(H), w_offset=0.0, x=z(B, H), ld_x=H, B=B, H=H, eps=1e-6)


ENTRIES = {"sgq_cache_plan": plan_args, "sgq_cache_write": write_args, "sgq_tree_attn": attn_call_args, "sgq_residual_norm": norm_args}
TENSORS = [(e, n) for e, make in ENTRIES.items() for n, t in make().items() if isinstance(t, torch.Tensor)]


def strided(t):
    """Every other element of a tensor of twice as many, of t's shape."""
    return torch.zeros(*t.shape, 2, dtype=t.dtype)[..., 0]


@pytest.mark.parametrize("entry", ENTRIES)
def test_dense_tensors_and_views_of_rows_pass(calls, entry):
    make = ENTRIES[entry]
    a = make()
    getattr(sgq, entry)(**a)
    (name, got), = calls
    assert name == entry
    addresses = {t.data_ptr() for t in a.values() if isinstance(t, torch.Tensor)}
    assert addresses <= set(got)


@pytest.mark.parametrize("entry,name", TENSORS)
def test_short_strided_and_mistyped_tensors_are_refused_by_name(calls, entry, name):
    a = ENTRIES[entry]()
    t = a[name]
    if name not in ("depth", "workspace"):        # (of these the entry point alone knows how many it needs)
        need = t.numel()
        if entry == "sgq_cache_write" and name in "qkv":       # the last row ends with its own part
            need = 4 * a["ld_q"] + (4 if name == "q" else 2) * 64
        with pytest.raises(ValueError, match=f"^{name}: "):
            getattr(sgq, entry)(**dict(a, **{name: torch.zeros(need - 1, dtype=t.dtype)}))
    if t.numel() > 1:
        with pytest.raises(ValueError, match=f"^{name}: "):
            getattr(sgq, entry)(**dict(a, **{name: strided(t)}))
    if t.dim() == 1 and t.numel() > 1:
        with pytest.raises(ValueError, match=f"^{name}: "):
            getattr(sgq, entry)(**dict(a, **{name: torch.zeros(1, dtype=t.dtype).expand(t.numel())}))
    with pytest.raises(TypeError):
        getattr(sgq, entry)(**dict(a, **{name: t.to(torch.int16)}))
    assert not calls


@pytest.mark.parametrize("entry", ENTRIES)
def test_tensors_of_another_device_are_refused(calls, monkeypatch, entry):
    monkeypatch.setattr(sgq, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="expected the current device, cuda:0"):
        getattr(sgq, entry)(**ENTRIES[entry]())
    assert not calls


OPTIONAL = {"sgq_cache_plan": ["depth", "pos", "req", "status"], "sgq_cache_write": ["n_tokens", "rope", "status"],
            "sgq_tree_attn": ["tree", "lse", "status"], "sgq_residual_norm": ["w_post", "gate", "x"]}


@pytest.mark.parametrize("entry,name", [(e, n) for e, names in OPTIONAL.items() for n in names])
def test_optional_tensors_may_be_none(calls, entry, name):
    getattr(sgq, entry)(**dict(ENTRIES[entry](), **{name: None}))
    assert len(calls) == 1 and None in calls[0][1]


def test_a_missing_tensor_reaches_the_entry_point(calls):
    # which says so itself (SGQ_ERR_NULL)
    sgq.sgq_cache_plan(**dict(plan_args(), lens=None))
    sgq.sgq_tree_attn(**dict(attn_call_args(), workspace=None))
    assert calls[0][1][0] is None and calls[1][1][-4] is None and calls[1][1][-3] == 0


def test_rows_may_be_views_of_wider_ones_with_leading_dimensions(calls):
    a = attn_call_args()
    T, width, ld = a["T"], a["ld_q"], a["ld_q"] + 64
    wide = torch.zeros(T, ld, dtype=BF16)
    for q in (wide, wide[:, :width], wide[:, 32:32 + width], wide[None, :, :width], wide.view(-1)[64:], wide[:, :width].unflatten(1, (4, 64))):
        sgq.sgq_tree_attn(**dict(a, q=q, ld_q=ld))
        assert calls[-1][1][0] == q.data_ptr()
    with pytest.raises(ValueError, match="^q: "):        # the last row ends behind the storage
        sgq.sgq_tree_attn(**dict(a, q=wide[:, 65:], ld_q=ld))
    with pytest.raises(ValueError, match="^q: "):        # heads and tokens the other way round
        sgq.sgq_tree_attn(**dict(a, q=torch.zeros(4, T, 64, dtype=BF16).transpose(0, 1)))
    with pytest.raises(ValueError, match="^table: "):
        sgq.sgq_tree_attn(**dict(a, table=a["table"].t().contiguous().t()))
    with pytest.raises(ValueError, match="^q: "):        # rows at another distance than is said
        sgq.sgq_tree_attn(**dict(a, q=wide[:, :width], ld_q=width))
    wider = torch.zeros(a["R"], 9, dtype=I32)
    sgq.sgq_tree_attn(**dict(a, table=wider[:, :3], table_ld=9))


def test_one_gate_for_all_rows(calls):
    a = norm_args()
    for gate in (torch.zeros(16, dtype=BF16), torch.zeros(16, dtype=BF16).expand(3, 16), torch.zeros(3, 20, dtype=BF16)[:, :16]):
        sgq.sgq_residual_norm(**dict(a, gate=gate, ld_gate=0))
    with pytest.raises(ValueError, match="^gate: "):
        sgq.sgq_residual_norm(**dict(a, gate=torch.zeros(16, dtype=BF16).expand(3, 16)))


def test_tree_words_of_either_type(calls):
    a = attn_call_args()
    for t in (I32, torch.uint32):
        sgq.sgq_tree_attn(**dict(a, tree=torch.zeros(a["T"], 1, dtype=t)))
    with pytest.raises(TypeError, match="^tree: "):
        sgq.sgq_tree_attn(**dict(a, tree=torch.zeros(a["T"], 1, dtype=I64)))


def test_the_helper_module_refuses_what_is_no_call():
    from activation_sparse_quantized_b200 import _tensors
    t = torch.zeros(4, dtype=I32)
    for bad in ((), (0,), (0, [t], (I32,), (4,)), (0, (t,), (I32, I32), (4,)), ("x", (t,), (I32,), (4,))):
        with pytest.raises(TypeError):
            _tensors.addresses(*bad)
    with pytest.raises(TypeError):
        _tensors.addresses(-1, (t,), (I32,), ("four",))
    assert _tensors.addresses(-1, (t,), ("int32",), (4,)) is None
    assert _tensors.addresses(-1, (3,), (I32,), (4,)) is None
    assert _tensors.addresses(-1, (t, None), (I32, I32), (4, 4)) == (t.data_ptr(), None)
