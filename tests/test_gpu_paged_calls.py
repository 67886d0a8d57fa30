"""Paged calls that the documentation allows and that are easy to get wrong at the edges."""
import math

import pytest
import torch

import paged_ref as ref
from dynamic_sparse_attention_est_b200 import minf

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)
BF, HF = torch.bfloat16, torch.float16


def test_one_element_arrays_may_have_any_stride():
    """One sequence's length out of an array of several, and a one-column table seen from a row."""
    c = ref.Case([1, 1], [13, 9], 4, 2, 16, BF, seed=1)
    want, _ = minf.minf_paged_attention(c.q, c.k_cache, c.v_cache, *c.meta(), scale=SCALE)
    column = c.tables[:, 0].clone().view(1, 2).t()
    assert column.shape == (2, 1) and column.stride(1) == 2
    got, _ = minf.minf_paged_attention(c.q, c.k_cache, c.v_cache, column, c.cu, c.kv_lens, 1, scale=SCALE)
    assert torch.equal(got, want)
    apart = torch.tensor([13, 0, 0, 9], dtype=torch.int32, device="cuda")
    got, _ = minf.minf_paged_attention(c.q[:1], c.k_cache, c.v_cache, c.tables[:1], c.cu[:2], apart[::4], 1, scale=SCALE)
    assert apart[::4].stride(0) == 4 and torch.equal(got, want[:1])
    with pytest.raises(ValueError, match="contiguous last"):
        minf.minf_paged_attention(c.q, c.k_cache, c.v_cache, c.tables, c.cu, apart[::3], 1, scale=SCALE)


def test_a_fault_in_a_call_without_a_workspace_goes_unreported_and_no_further():
    """The call returns, the rows left out keep what they held, and the next call finds no trace of it; with
    a workspace the same call is reported."""
    c = ref.Case([1, 1], [300, 90], 4, 2, 64, BF, seed=2)
    want, _ = minf.minf_paged_attention(c.q, c.k_cache, c.v_cache, *c.meta(), scale=SCALE)
    bad = c.kv_lens.clone()
    bad[1] = -1
    out = torch.full((2, 4, 128), 9.0, dtype=BF, device="cuda")
    minf.minf_paged_attention(c.q, c.k_cache, c.v_cache, c.tables, c.cu, bad, 1, scale=SCALE, out=out)
    assert torch.equal(out[0], want[0]) and (out[1] == 9).all()
    ws = minf.workspace(minf.paged_workspace_bytes(minf.OP_PAGED_ATTENTION, 4, 2, 2, 2, 1), "cuda")
    got, _ = minf.minf_paged_attention(c.q, c.k_cache, c.v_cache, *c.meta(), scale=SCALE, ws=ws)
    assert torch.equal(got, want) and minf.minf_status(ws) == 0
    minf.minf_paged_attention(c.q, c.k_cache, c.v_cache, c.tables, c.cu, bad, 1, scale=SCALE, out=out, ws=ws)
    assert minf.minf_status(ws) == minf.MINF_ERR_INVALID
