"""A sequence that contradicts itself costs the others nothing: their results beside it, in all four calls."""
import math

import pytest
import torch

import paged_ref as ref
from dynamic_sparse_attention_est_b200 import minf

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)
BF = torch.bfloat16
P, TOPK = 64, 4


def faulty(lens, kv, fault):
    """The case with its fault in; the rows whose results stand, as (sequence, row, position); and the rows
    that are left out."""
    c = ref.Case(lens, kv, 4, 2, P, BF, seed=12)
    rows = list(c.rows())
    if fault == "starts":  # sequence 1 ends before it begins, and 2 takes its rows and one of sequence 0
        c.cu[2] = c.cu[1] - 1
        at, end = lens[0] - 1, sum(lens[:3])
        n = end - at
        rows = [x for x in rows if x[1] < at or x[1] >= end]
        if n > c.max_q:
            return c, rows, list(range(at + 1, end))
        return c, rows + [(2, r, kv[2] - n + r - at) for r in range(at + 1, end)], []
    bad = 1
    if fault == "length":
        c.kv_lens[1] = c.width * P + 1
    elif fault == "negative":
        c.kv_lens[1] = -5
    elif fault == "page":
        c.tables[1, 0] = c.num_pages
    else:
        c.max_q -= 1
        bad = lens.index(max(lens))
    out = [] if fault == "page" else [r for s, r, _ in rows if s == bad]
    return c, [x for x in rows if x[0] != bad], out


@pytest.mark.parametrize("fault", ["length", "negative", "page", "starts", "max_q"])
@pytest.mark.parametrize("lens,kv", [([1, 1, 2], [300, 90, 400]), ([90, 5, 70], [300, 90, 400]),
                                     ([1, 1, 2], [9000, 90, 7000]), ([90, 5, 70], [9000, 90, 7000])])
def test_other_sequences_results_stand(lens, kv, fault):
    """Short sequences (whole items) and long ones (cut into parts and joined: which parts an item has follows
    from the lengths of all the others)."""
    c, rows, out_rows = faulty(lens, kv, fault)
    c.rows = lambda: iter(rows)  # the 64-bit forms go over these alone
    keep = torch.tensor([r for _, r, _ in rows], dtype=torch.long, device="cuda")
    gone = torch.tensor(out_rows, dtype=torch.long, device="cuda")
    ws = minf.workspace(max(minf.paged_workspace_bytes(op, 4, 2, c.total, 3, max(lens), c.width, TOPK) for op in
                            (minf.OP_PAGED_ATTENTION, minf.OP_PAGED_BLOCK_ESTIMATE, minf.OP_PAGED_BLOCK_ATTENTION)),
                        "cuda")

    def agrees(got, want):
        o, l = got
        ro, rl, to, tl = want
        assert ((o[keep].double() - ro[keep]).abs() <= to[keep]).all()
        assert ((l[keep].double() - rl[keep]).abs() <= tl[keep]).all()
        assert (o[gone] == 9).all()
        assert minf.minf_status(ws) == minf.MINF_ERR_INVALID

    def buffer():
        return torch.full((c.total, 4, 128), 9.0, dtype=BF, device="cuda")

    agrees(minf.minf_paged_attention(c.q, c.k_cache, c.v_cache, *c.meta(), scale=SCALE, out=buffer(), ws=ws),
           ref.attention(c, SCALE))

    tables = c.tables.clone()
    c.tables.clamp_(max=c.num_pages - 1)  # the 64-bit forms' own reads
    kb = torch.nan_to_num(ref.bounds(c))
    wi, wc = ref.estimate(c, kb, TOPK)
    c.tables.copy_(tables)
    idx, cnt = minf.minf_paged_block_estimate(c.q, kb, *c.meta(), page_size=P, topk=TOPK, ws=ws)
    assert torch.equal(idx[keep], wi[keep]) and torch.equal(cnt[keep], wc[keep])
    assert minf.minf_status(ws) == minf.MINF_ERR_INVALID

    sets = [[set(wi[r, h, :wc[r, h]].tolist()) for h in range(2)] for r in range(c.total)]

    def pick(s, r, h, pos):
        return torch.tensor([(i // P) in sets[r][h] for i in range(pos + 1)], dtype=torch.bool, device="cuda")

    li, lc = wi.clone(), wc.clone()
    rest = torch.ones(c.total, dtype=torch.bool, device="cuda")
    rest[keep] = False
    li[rest], lc[rest] = torch.arange(TOPK, dtype=torch.int32, device="cuda"), TOPK
    agrees(minf.minf_paged_block_attention(c.q, c.k_cache, c.v_cache, *c.meta(), li, lc, scale=SCALE, out=buffer(), ws=ws),
           ref.attention(c, SCALE, pick))


@pytest.mark.parametrize("fault", ["length", "negative", "page", "starts", "max_q"])
@pytest.mark.parametrize("lens", [[1, 1, 2], [90, 5, 70], [700] + [1] * 60 + [70]])
def test_appends_beside_a_bad_sequence(lens, fault):
    """Rows stored and bounds kept for the others, nothing for the one left out (the last case finds its pages
    by counting over all sequences)."""
    kv = [len_ + 95 + 31 * (i % 9) for i, len_ in enumerate(lens)]
    c, rows, out_rows = faulty(lens, kv, fault)
    kc, vc = torch.nan_to_num(c.k_cache), torch.nan_to_num(c.v_cache)
    kb = torch.stack(kc.aminmax(dim=2), 2).contiguous()
    kc0, vc0, kb0 = kc.clone(), vc.clone(), kb.clone()
    q_out = torch.full((c.total, 4, 128), 9.0, dtype=BF, device="cuda")
    ws = minf.workspace(256, "cuda")
    minf.minf_paged_append(c.k_new, c.v_new, kc, vc, *c.meta(), q=c.q, q_out=q_out, k_bounds=kb, ws=ws)
    # the append stores into sequence 1's second page and later ones only: the bad first one it has no use for
    assert minf.minf_status(ws) == (0 if fault == "page" else minf.MINF_ERR_INVALID)
    keep = torch.tensor([r for _, r, _ in rows], dtype=torch.long, device="cuda")
    assert torch.equal(q_out[keep], c.q[keep])
    assert (q_out[torch.tensor(out_rows, dtype=torch.long, device="cuda")] == 9).all()
    seq = torch.tensor([s for s, _, _ in rows], dtype=torch.long, device="cuda")
    pos = torch.tensor([p for _, _, p in rows], dtype=torch.long, device="cuda")
    page = c.tables[seq, pos // P].long()
    assert torch.equal(kc[page, :, pos % P], c.k_new[keep]) and torch.equal(vc[page, :, pos % P], c.v_new[keep])
    others = torch.ones(c.num_pages, P, dtype=torch.bool, device="cuda")
    others[page, pos % P] = False
    touched = torch.zeros(c.num_pages, dtype=torch.bool, device="cuda")
    touched[page] = True
    if fault in ("page", "starts"):  # sequence 1 is stored all the same; rows of two sequences are unspecified
        for s in ((1,) if fault == "page" else (0, 2)):
            mine = c.tables[s][(c.tables[s] >= 0) & (c.tables[s] < c.num_pages)].long()
            others[mine] = False
            touched[mine] = True
            page = page[~torch.isin(page, mine)]
    assert torch.equal(kc.transpose(1, 2)[others], kc0.transpose(1, 2)[others])
    assert torch.equal(vc.transpose(1, 2)[others], vc0.transpose(1, 2)[others])
    assert torch.equal(kb[~touched], kb0[~touched])
    for pg in page.unique().tolist():
        new = ~others[pg]
        lo, hi = kc[pg, :, new].amin(1), kc[pg, :, new].amax(1)
        if not new[0]:  # the page held keys before
            lo, hi = torch.minimum(lo, kb0[pg, :, 0]), torch.maximum(hi, kb0[pg, :, 1])
        assert torch.equal(kb[pg, :, 0], lo) and torch.equal(kb[pg, :, 1], hi)
