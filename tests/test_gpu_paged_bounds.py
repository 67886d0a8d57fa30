"""Page selection on bounds that are hard: not finite, and made so that approximate scores come out badly."""
import ctypes
import math

import pytest
import torch

import paged_ref as ref
from dynamic_sparse_attention_est_b200 import minf

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def estimate_into(c, kb, topk, ws, idx, cnt):
    """The C call, into lists that the caller filled."""
    q = c.q.contiguous()
    seqs = minf.PagedSeqs(c.cu.data_ptr(), c.kv_lens.data_ptr(), c.tables.data_ptr(), c.tables.stride(0), c.width,
                          len(c.lens), c.total, c.max_q, c.page, c.num_pages)
    rows = minf.Rows(q.data_ptr(), q.stride(0), q.stride(1))
    rc = minf.lib().minf_paged_block_estimate(
        ctypes.byref(seqs), minf.MINF_FP16 if c.dtype == HF else minf.MINF_BF16, c.hq, c.hkv, 128, ctypes.byref(rows),
        kb.data_ptr(), topk, idx.data_ptr(), cnt.data_ptr(), ws.data_ptr(), ws.numel(),
        torch.cuda.current_stream().cuda_stream)
    assert rc == 0, minf.lib().minf_last_error()
    torch.cuda.synchronize()


# few rows and few new tokens; a CTA per row behind the tensor-core scores; a warp per row, 32 and 64 keys a lane
@pytest.mark.parametrize("lens,pages", [([2], 60), ([300], 300), ([600], 700), ([600], 1500)])
@pytest.mark.parametrize("what", ["inf", "nan", "all_inf", "all_nan", "minus_inf", "every_kind"])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_lists_are_whole_whatever_the_bounds_hold(lens, pages, what, dtype):
    """Bounds that are not finite leave open which pages are taken, not what a list is: as many entries as
    there are pages up to topk, ascending and distinct, the token's own page last, -1 behind."""
    c = ref.Case(lens, [16 * pages + lens[0]], 4, 2, 16, dtype, seed=1, extra_rows=1)
    kb = torch.nan_to_num(ref.bounds(c))
    g = torch.Generator(device="cuda").manual_seed(pages)
    if what in ("inf", "nan"):
        kb[::3, :, 1, 5] = float(what)
    elif what == "minus_inf":
        kb[::2, :, 0, 7] = -math.inf
    elif what == "every_kind":
        kinds = torch.tensor([math.inf, -math.inf, math.nan, 0.0], device="cuda", dtype=dtype)
        at = torch.rand(kb.shape, generator=g, device="cuda") < 0.01
        kb[at] = kinds[torch.randint(0, 4, (int(at.sum()),), generator=g, device="cuda")]
    else:
        kb[:, :, 1] = float(what[4:])
    topk, poison = 20, 123456789
    ws = minf.workspace(minf.paged_workspace_bytes(minf.OP_PAGED_BLOCK_ESTIMATE, 4, 2, c.total, 1, c.max_q, c.width,
                                                   topk), "cuda")
    idx = torch.full((c.total, 2, topk), poison, dtype=torch.int32, device="cuda")
    cnt = torch.full((c.total, 2), poison, dtype=torch.int32, device="cuda")
    estimate_into(c, kb, topk, ws, idx, cnt)
    assert minf.minf_status(ws) == 0
    n = lens[0]
    assert (idx[n:] == poison).all() and (cnt[n:] == poison).all()  # the row of no sequence
    idx, cnt = idx[:n].long(), cnt[:n].long()
    own = torch.arange(c.kv[0] - n, c.kv[0], device="cuda")[:, None] // 16
    assert (cnt == (own + 1).clamp(max=topk)).all()
    at = torch.arange(topk, device="cuda")
    listed = at < cnt[..., None]
    assert (idx[~listed] == -1).all()
    assert (idx[listed] >= 0).all()
    assert ((idx[..., 1:] > idx[..., :-1]) | ~listed[..., 1:]).all()
    assert (idx.gather(2, cnt[..., None] - 1)[..., 0] == own).all()


# ------------------------------------------------------------------ the approximate scores' error
def made(kind, c, g):
    """Queries and bounds (min <= max) of a kind."""
    def rnd(*s):
        return torch.randn(*s, generator=g, device="cuda")

    q, kb = rnd(*c.q.shape), rnd(c.num_pages, c.hkv, 2, 128)
    if kind == "cancelling":  # large terms of both signs, small sums
        kb = kb.sign() * (1 + kb.abs() / 64)
        q = q.sign() * (1 + q.abs() / 64)
    elif kind == "one_sign":  # every rounding in the running sum falls the same way
        kb, q = 1 + kb.abs() / 8, 1 + q.abs() / 8
    elif kind == "one_large":  # one product so large that the others' last bits fall out
        q, kb = torch.rand(q.shape, generator=g, device="cuda") * 2 ** -9, 0.5 + torch.rand(kb.shape, generator=g, device="cuda") / 2
        q[..., 3], kb[..., 3] = 255 / 256, 255 / 256
    elif kind == "wide":
        q, kb = q * torch.exp2(4 * rnd(*q.shape)).clamp(2 ** -8, 2 ** 6), kb * torch.exp2(4 * rnd(*kb.shape)).clamp(2 ** -8, 2 ** 6)
    return q.to(c.dtype), kb.sort(dim=2).values.to(c.dtype)


@pytest.mark.parametrize("kind", ["normal", "cancelling", "one_sign", "one_large", "wide"])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (64, 1)])
@pytest.mark.parametrize("lens", [[3], [70]])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_approximate_scores_keep_within_the_bound_that_decides(lens, dtype, hq, hkv, kind, record_property):
    """The scores as the first kernel leaves them in the workspace (its other output, the lists, hides their
    error): off from the 64-bit ones by at most E = (2^-15 + G 2^-23) |Q|_1 max |bound|."""
    c = ref.Case(lens, [16 * 300 + lens[0]], hq, hkv, 16, dtype, seed=3)
    c.q, kb = made(kind, c, torch.Generator(device="cuda").manual_seed(len(kind) + hq))
    topk, n = 5, lens[0]
    ws = minf.workspace(minf.paged_workspace_bytes(minf.OP_PAGED_BLOCK_ESTIMATE, hq, hkv, c.total, 1, c.max_q, c.width,
                                                   topk), "cuda")
    idx = torch.empty(c.total, hkv, topk, dtype=torch.int32, device="cuda")
    cnt = torch.empty(c.total, hkv, dtype=torch.int32, device="cuda")
    estimate_into(c, kb, topk, ws, idx, cnt)
    stride = -(-c.width // 4) * 4
    got = ws[256:256 + 4 * n * hkv * stride].view(torch.float32).view(n, hkv, stride)[:, :, :300].double()
    x = c.q.double().view(n, hkv, hq // hkv, 128)
    up, down = x.clamp(min=0).sum(2), x.clamp(max=0).sum(2)
    if dtype == HF:  # these scores carry a power of two that brings a row's largest sum below 2^14
        top = torch.maximum(up.amax(-1), (-down).amax(-1))
        got = got / torch.exp2(14 - torch.frexp(top).exponent.double())[..., None]
    b = kb[c.tables[0, :300].long()].double()
    want = torch.einsum("nhd,phd->nhp", up, b[:, :, 1]) + torch.einsum("nhd,phd->nhp", down, b[:, :, 0])
    norm = (up - down).sum(-1)
    err = (2 ** -15 + hq // hkv * 2 ** -23) * norm * b.abs().amax((0, 2, 3))
    worst = float(((got - want).abs() / err[..., None]).max())
    record_property("share_of_the_bound", worst)
    print(f"share {worst:.4f}")
    assert worst <= 1.0
    wi, wc = ref.estimate(c, kb, topk)
    assert torch.equal(cnt, wc) and torch.equal(idx, wi)
