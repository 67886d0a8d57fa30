"""The workspace of the paged calls: what a call without one costs, and what a call finds in one."""
import math

import pytest
import torch

import paged_ref as ref
from dynamic_sparse_attention_est_b200 import minf

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)
BF = torch.bfloat16
POISON = 171


def poisoned(need):
    """Leaves a freed block of `need` bytes of POISON for the next allocation of that size; its address."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    block = torch.full((need,), POISON, dtype=torch.uint8, device="cuda")
    return block.data_ptr()


@pytest.mark.parametrize("lens,kv", [([40, 33], [300, 90]), ([1, 1], [300, 65])])
def test_a_call_without_a_workspace_clears_the_status_block_only(lens, kv):
    """The buffer that the call takes from the allocator keeps what it held wherever the kernels have nothing
    to write (partial slots that no part of the work takes).  The results are those of a cleared workspace."""
    c = ref.Case(lens, kv, 8, 2, 64, BF, seed=1)
    kb = torch.nan_to_num(ref.bounds(c))
    lists = torch.zeros(c.total, 2, 64, dtype=torch.int32, device="cuda")
    cnt = torch.ones(c.total, 2, dtype=torch.int32, device="cuda")
    args = (8, 2, c.total, len(lens), c.max_q)
    calls = [
        (minf.paged_workspace_bytes(minf.OP_PAGED_ATTENTION, *args),
         lambda ws: minf.minf_paged_attention(c.q, c.k_cache, c.v_cache, *c.meta(), scale=SCALE, ws=ws)),
        (minf.paged_workspace_bytes(minf.OP_PAGED_BLOCK_ESTIMATE, *args, c.width, 2),
         lambda ws: minf.minf_paged_block_estimate(c.q, kb, *c.meta(), topk=2, ws=ws)),
        (minf.paged_workspace_bytes(minf.OP_PAGED_BLOCK_ATTENTION, *args, c.width, 64),
         lambda ws: minf.minf_paged_block_attention(c.q, c.k_cache, c.v_cache, *c.meta(), lists, cnt, scale=SCALE,
                                                    ws=ws)),
    ]
    seen = 0
    for need, call in calls:
        want = [t.clone() for t in call(minf.workspace(need, "cuda"))]
        n = sum(lens)
        assert all(torch.equal(a[:n], b[:n]) for a, b in zip(call(None), want))
        if need < 2 << 20:  # the allocator hands the same block out again from there on
            continue
        at = poisoned(need)
        got = call(None)
        block = torch.empty(need, dtype=torch.uint8, device="cuda")
        assert block.data_ptr() == at  # the call's own buffer, given back
        assert (block == POISON).float().mean() > 0.1  # 1 / 256 of random bytes, none of cleared ones
        assert all(torch.equal(a[:n], b[:n]) for a, b in zip(got, want))
        del block
        seen += 1
    assert seen >= 1
