"""The step entry points' binding: what it refuses of tensors, on the host, and the
calls around the entry points (no GPU needed)."""
import pytest

from activation_sparse_quantized_b200 import build as sgq_build
from activation_sparse_quantized_b200 import sgq
from test_step_abi import ATTN_FAULTS, attn_args


@pytest.fixture(scope="module")
def lib():
    sgq_build.build()
    return sgq.load()


@pytest.mark.parametrize("fault,code", ATTN_FAULTS, ids=[str(list(f[0])[0]) + str(f[1]) for f in ATTN_FAULTS])
def test_the_attention_test_hook_refuses_what_the_entry_point_refuses(lib, fault, code):
    assert lib.sgq_debug_tree_attn_withhold(*attn_args(lib, **fault)) == code
