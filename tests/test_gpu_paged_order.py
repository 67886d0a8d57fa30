"""What follows a paged call in its stream sees its results whole and may overwrite what it read: also where no
part of the work was cut, so that the kernel launched behind the first has nothing to wait for."""
import math

import pytest
import torch

import paged_ref as ref
from dynamic_sparse_attention_est_b200 import minf

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)
BF = torch.bfloat16


# short sequences: one share each, nothing to join; long ones with a few lists: some cut, some not
@pytest.mark.parametrize("lens,kv", [([1], [9]), ([1, 1, 1], [1, 16, 40]), ([1] * 6, [3000, 5, 900, 64, 1, 2000])])
def test_caches_may_change_right_behind_attention(lens, kv):
    c = ref.Case(lens, kv, 8, 2, 64, BF, seed=2)
    kc, vc = torch.nan_to_num(c.k_cache), torch.nan_to_num(c.v_cache)
    idx = torch.zeros(c.total, 2, 1, dtype=torch.int32, device="cuda")
    cnt = torch.ones(c.total, 2, dtype=torch.int32, device="cuda")
    ws = minf.workspace(max(minf.paged_workspace_bytes(op, 8, 2, c.total, len(lens), c.max_q, c.width, 1)
                            for op in (minf.OP_PAGED_ATTENTION, minf.OP_PAGED_BLOCK_ATTENTION)), "cuda")
    calls = [lambda k, v, o: minf.minf_paged_attention(c.q, k, v, *c.meta(), scale=SCALE, out=o, ws=ws),
             lambda k, v, o: minf.minf_paged_block_attention(c.q, k, v, *c.meta(), idx, cnt, scale=SCALE, out=o, ws=ws)]
    for call in calls:
        want = [t.clone() for t in call(kc, vc, None)]
        torch.cuda.synchronize()
        seen = []
        for _ in range(30):
            k, v, o = kc.clone(), vc.clone(), torch.full_like(c.q, 7.0).contiguous()
            got, lse = call(k, v, o)
            copy, lse = got.clone(), lse.clone()
            k.fill_(float("nan"))
            v.fill_(float("nan"))
            seen.append((copy, lse))
        for a, b in seen:
            assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    assert minf.minf_status(ws) == 0


@pytest.mark.parametrize("lens,pages", [([1, 2], 30), ([300], 60)])
def test_workspace_serves_the_next_call_right_behind_a_selection(lens, pages):
    """Every row keeps all its pages, so no row needs the scores that the first kernel still writes."""
    c = ref.Case(lens, [16 * pages + n for n in lens], 8, 8 if len(lens) == 1 else 2, 16, BF, seed=3)
    kb = torch.nan_to_num(ref.bounds(c))
    ws = minf.workspace(max(minf.paged_workspace_bytes(op, c.hq, c.hkv, c.total, len(lens), c.max_q, c.width, c.width)
                            for op in (minf.OP_PAGED_ATTENTION, minf.OP_PAGED_BLOCK_ESTIMATE)), "cuda")
    want = [t.clone() for t in minf.minf_paged_attention(c.q, c.k_cache, c.v_cache, *c.meta(), scale=SCALE, ws=ws)]
    wi, wc = ref.estimate(c, kb, c.width)
    for _ in range(20):
        idx, cnt = minf.minf_paged_block_estimate(c.q, kb, *c.meta(), page_size=16, topk=c.width, ws=ws)
        o, l = minf.minf_paged_attention(c.q, c.k_cache, c.v_cache, *c.meta(), scale=SCALE, ws=ws)
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])
        assert torch.equal(idx, wi) and torch.equal(cnt, wc)
    assert minf.minf_status(ws) == 0


# ------------------------------------------------------------------ starts that name the same rows over and over
def alternating(n_seqs, n):
    """Every other sequence claims all n rows, the ones between end before they begin."""
    return torch.tensor([0, n] * (n_seqs // 2) + [0], dtype=torch.int32, device="cuda")


def test_append_counts_rows_named_over_and_over():
    """2,048 sequences of 2^20 pages each: their sum passes 32 bits.  No table entry is a page."""
    n_seqs, n = 4096, 1 << 24
    k = torch.zeros(n * 8 + 128, dtype=BF, device="cuda").as_strided((n, 1, 128), (8, 128, 1))
    kc = torch.zeros(2, 1, 16, 128, dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    tables = torch.full((n_seqs, n // 16), -1, dtype=torch.int32, device="cuda")
    kv = torch.full((n_seqs,), n, dtype=torch.int32, device="cuda")
    ws = minf.workspace(minf.paged_workspace_bytes(minf.OP_PAGED_APPEND, 1, 1, n, n_seqs, n), "cuda")
    minf.minf_paged_append(k, k, kc, vc, tables, alternating(n_seqs, n), kv, n, ws=ws)
    assert minf.minf_status(ws) == minf.MINF_ERR_INVALID
    assert (kc == 0).all() and (vc == 0).all()


def test_chunk_works_on_no_rows_named_over_and_over():
    """2,048 sequences that claim the same 4,096 tokens: more row tiles than the rows make."""
    n_seqs, n = 4096, 4096
    q = torch.zeros(n, 4, 128, dtype=BF, device="cuda")
    kc = torch.zeros(256, 1, 16, 128, dtype=BF, device="cuda")
    tables = torch.arange(256, dtype=torch.int32, device="cuda").expand(n_seqs, 256).contiguous()
    kv = torch.full((n_seqs,), n, dtype=torch.int32, device="cuda")
    ws = minf.workspace(minf.paged_workspace_bytes(minf.OP_PAGED_ATTENTION, 4, 1, n, n_seqs, n), "cuda")
    out = torch.full_like(q, 7.0)
    minf.minf_paged_attention(q, kc, kc, tables, alternating(n_seqs, n), kv, n, out=out, ws=ws)
    assert minf.minf_status(ws) == minf.MINF_ERR_INVALID
    assert (out == 7).all()
    # the same workspace serves a call that makes sense
    minf.minf_paged_attention(q, kc, kc, tables[:1], alternating(2, n)[:2], kv[:1], n, out=out, ws=ws)
    assert minf.minf_status(ws) == 0 and (out == 0).all()


# ------------------------------------------------------------------ the binding
def test_flags_without_a_truth_value_raise_their_own_error():
    c = ref.Case([1], [20], 4, 2, 16, BF, seed=1)
    no_truth = torch.zeros(2)
    with pytest.raises(RuntimeError, match="ambiguous"):
        minf.minf_paged_append(c.k_new, c.v_new, c.k_cache, c.v_cache, *c.meta(), interleaved=no_truth)
    with pytest.raises(RuntimeError, match="ambiguous"):
        minf.minf_paged_attention(c.q, c.k_cache, c.v_cache, *c.meta(), want_lse=no_truth)
    with pytest.raises(ValueError, match="integer"):
        minf.minf_paged_attention(c.q, c.k_cache, c.v_cache, c.tables, c.cu, c.kv_lens, "one")
    with pytest.raises(TypeError):
        minf.minf_paged_attention(c.q, c.k_cache, c.v_cache, *c.meta(), scale="a")
