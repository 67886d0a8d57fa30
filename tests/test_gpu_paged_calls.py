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


@pytest.mark.parametrize("reps,n,hq,hkv,steps", [
    (1 << 20, 1, 4, 1, 4800),       # 296 shares, six warps each
    (1 << 13, 3, 4, 2, 80),
    (1 << 10, 1024, 64, 16, 8192),  # row tiles uncut over 131,072 keys
    (1 << 15, 64, 4, 1, 8192),      # two row tiles, cut into 32 parts
])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_contexts_of_up_to_2_27_tokens(reps, n, hq, hkv, steps, dtype):
    """One page that a table names over and over: each of its keys counts as often as it is seen, so the 64-bit
    form needs the page alone.

    Beside the errors of `ref.attention`: O grows in the tensor cores' fp32 taken to truncate, so that each of
    the `steps` of 16 keys of a part loses up to 2^-23 of the sum so far, which is half of the final one on
    average.  The sum of weights loses half of that.  fp16 weights end at 2^-25 of a scale that lies 2^6 below
    the row's largest at the least."""
    P = 128
    g = torch.Generator(device="cuda").manual_seed(reps)
    k, v = (torch.randn(1, hkv, P, 128, generator=g, device="cuda").to(dtype) for _ in "kv")
    q = torch.randn(n, hq, 128, generator=g, device="cuda").to(dtype)
    table = torch.zeros(1, reps, dtype=torch.int32, device="cuda")
    cu, kv = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n], [reps * P]))
    ws = minf.workspace(minf.paged_workspace_bytes(minf.OP_PAGED_ATTENTION, hq, hkv, n, 1, n), "cuda")
    out, lse = minf.minf_paged_attention(q, k, v, table, cu, kv, n, scale=SCALE, ws=ws)
    assert minf.minf_status(ws) == 0
    x = torch.einsum("nhgd,hkd->nhgk", q.double().view(n, hkv, -1, 128), k[0].double()) * SCALE
    seen = (torch.arange(reps * P - n, reps * P, device="cuda")[:, None] + P - torch.arange(P, device="cuda")) // P
    w = x + seen.double().log()[:, None, None, :]
    z = torch.logsumexp(w, -1)
    p = (w - z[..., None]).exp()
    want, mag = (torch.einsum("nhgk,hkd->nhgd", p, t).reshape(n, hq, 128) for t in (v[0].double(), v[0].double().abs()))
    dots = torch.einsum("nhgd,hkd->nhgk", q.double().abs().view(n, hkv, -1, 128), k[0].double().abs()).amax(-1) * SCALE
    d = (dots * 2 ** -19 + x.abs().amax(-1) * 2 ** -23 + 2 ** -20).reshape(n, hq)
    u = ref.u(dtype)
    tol = u * want.abs() + (u + 2 * d[..., None] + steps * 2 ** -24) * mag + 1e-7
    if dtype == HF:
        weights = (z - x.amax(-1)).exp().reshape(n, hq, 1)  # in units of the largest
        tol += 2 ** -25 + reps * P * 2 ** -31 / weights * v.double().abs().max()
    assert ((out.double() - want).abs() <= tol).all()
    tol = d + steps * 2 ** -25 + 64 * 2 ** -24 + z.reshape(n, hq).abs() * 2 ** -22 + 2 ** -20
    assert ((lse.double() - z.reshape(n, hq)).abs() <= tol).all()
