"""Refusals of the paged calls, on the host: through the C ABI before any CUDA call, and in the binding."""
import ctypes
import random

import pytest
import torch

from dynamic_sparse_attention_est_b200 import minf

FAKE = 1 << 20  # 256-byte aligned, never dereferenced
BIG = 1 << 40


def seqs(**kw):
    a = dict(cu_q=FAKE, kv_lens=FAKE, block_tables=FAKE, table_stride=8, width=8, n_seqs=2, total=3, max_q=2,
             page_size=64, num_pages=20)
    a.update(kw)
    return minf.PagedSeqs(**a)


def rows(heads=4, **kw):
    a = dict(data=FAKE, token_stride=heads * 128, head_stride=128)
    a.update(kw)
    return minf.Rows(**a)


def cache(page=64, hkv=2, **kw):
    a = dict(k=FAKE, v=FAKE, k_page_stride=page * hkv * 128, v_page_stride=page * hkv * 128)
    a.update(kw)
    return minf.PagedCache(**a)


def ref(x):
    return None if x is None else ctypes.byref(x)


def attention(s=None, dtype=0, hq=4, hkv=2, d=128, q=None, c=None, scale=0.1, out=None, ws=FAKE, wsb=BIG, **kw):
    s = seqs(**kw) if s is None else s
    q = rows() if q is None else q
    out = rows() if out is None else out
    c = cache(s.page_size) if c is None else c
    return minf.lib().minf_paged_attention(ref(s), dtype, hq, hkv, d, ref(q), ref(c), scale, ref(out), None, ws, wsb, None)


INV, UNS, WS = minf.MINF_ERR_INVALID, minf.MINF_ERR_UNSUPPORTED, minf.MINF_ERR_WORKSPACE

COMMON = [
    (dict(dtype=2), UNS), (dict(dtype=-1), UNS), (dict(hkv=3), INV), (dict(hq=0), INV), (dict(hq=512, hkv=1), INV),
    (dict(hq=256, hkv=1), UNS), (dict(d=64), UNS), (dict(page_size=8), UNS), (dict(page_size=48), UNS),
    (dict(n_seqs=-1), INV), (dict(n_seqs=4097), UNS), (dict(total=-1), INV), (dict(cu_q=None), INV),
    (dict(kv_lens=None), INV), (dict(block_tables=None), INV), (dict(width=0), INV), (dict(table_stride=7), INV),
    (dict(num_pages=0), INV), (dict(max_q=0), INV), (dict(max_q=4), INV),
    (dict(width=1 << 25, table_stride=1 << 25), UNS), (dict(total=1 << 29, max_q=1), UNS),
]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(scale=0.0), INV), (dict(scale=float("inf")), INV), (dict(q=rows(data=None)), INV),
    (dict(q=rows(data=FAKE + 8)), INV), (dict(q=rows(token_stride=516)), INV), (dict(q=rows(head_stride=0)), INV),
    (dict(q=rows(token_stride=-512)), INV), (dict(out=rows(data=None)), INV),
    (dict(out=rows(token_stride=256)), INV),                      # rows overlap
    (dict(out=rows(head_stride=64, token_stride=512)), INV),
    (dict(c=cache(k=None)), INV), (dict(c=cache(v=FAKE + 2)), INV), (dict(c=cache(k_page_stride=128)), INV),
    (dict(c=cache(v_page_stride=64 * 2 * 128 + 4)), INV), (dict(ws=None), INV), (dict(ws=FAKE + 64), INV),
    (dict(wsb=256), WS),
])
def test_attention_refusals(minf_lib, kw, code):
    assert attention(**kw) == code
    assert minf.lib().minf_last_error()


def test_nothing_to_do_is_not_an_error(minf_lib):
    assert attention(total=0) == 0 and attention(n_seqs=0) == 0
    assert minf.lib().minf_paged_attention(None, 0, 4, 2, 128, None, None, 0.1, None, None, FAKE, BIG, None) == INV


def append(dtype=0, hq=4, hkv=2, d=128, k=None, v=None, q=None, qo=None, c=None, kb=None, rope=None, rrows=0, rot=0,
           ws=FAKE, wsb=256, **kw):
    s = seqs(**kw)
    k = rows(hkv) if k is None else k
    v = rows(hkv) if v is None else v
    c = cache(s.page_size) if c is None else c
    return minf.lib().minf_paged_append(ref(s), dtype, hq, hkv, d, ref(k), ref(v), ref(q), ref(qo), ref(c), kb, rope,
                                        rrows, rot, 0, ws, wsb, None)


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(rope=FAKE, rrows=10, rot=8), UNS), (dict(rope=FAKE, rrows=10, rot=144), UNS),
    (dict(rope=FAKE, rrows=10, rot=40), UNS), (dict(rope=FAKE, rrows=0, rot=64), INV),
    (dict(rope=FAKE + 4, rrows=9, rot=64), INV), (dict(q=rows()), INV), (dict(qo=rows()), INV),
    (dict(q=rows(), qo=rows(token_stride=128)), INV), (dict(k=rows(2, data=None)), INV),
    (dict(v=rows(2, head_stride=100)), INV), (dict(kb=FAKE + 8), INV), (dict(wsb=16), WS), (dict(ws=None), INV),
])
def test_append_refusals(minf_lib, kw, code):
    assert append(**kw) == code


def estimate(dtype=0, hq=4, hkv=2, d=128, q=None, kb=FAKE, topk=4, idx=FAKE, cnt=FAKE, ws=FAKE, wsb=BIG, **kw):
    return minf.lib().minf_paged_block_estimate(ref(seqs(**kw)), dtype, hq, hkv, d, ref(q or rows()), kb, topk, idx, cnt,
                                                ws, wsb, None)


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(topk=0), INV), (dict(kb=None), INV), (dict(kb=FAKE + 8), INV), (dict(idx=None), INV), (dict(cnt=None), INV),
    (dict(width=32769, table_stride=32769, page_size=16), UNS), (dict(wsb=256), WS), (dict(q=rows(data=None)), INV),
])
def test_estimate_refusals(minf_lib, kw, code):
    assert estimate(**kw) == code


def block_attention(dtype=0, hq=4, hkv=2, d=128, topk=4, idx=FAKE, cnt=FAKE, ws=FAKE, wsb=BIG, scale=0.1, **kw):
    s = seqs(**kw)
    return minf.lib().minf_paged_block_attention(ref(s), dtype, hq, hkv, d, ref(rows()), ref(cache(s.page_size)), scale,
                                                 idx, cnt, topk, ref(rows()), None, ws, wsb, None)


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(topk=0), INV), (dict(idx=None), INV), (dict(cnt=None), INV), (dict(scale=-1.0), INV), (dict(wsb=256), WS),
])
def test_block_attention_refusals(minf_lib, kw, code):
    assert block_attention(**kw) == code


def test_workspace_sizes(minf_lib):
    f = minf.paged_workspace_bytes
    assert f(minf.OP_PAGED_APPEND, 32, 8, 10, 2, 5) == minf.MINF_STATUS_BYTES
    assert f(minf.OP_PAGED_ATTENTION, 32, 8, 0, 0, 0) == minf.MINF_STATUS_BYTES
    a = f(minf.OP_PAGED_ATTENTION, 32, 8, 64, 64, 1)      # streaming
    b = f(minf.OP_PAGED_ATTENTION, 32, 8, 2048, 1, 2048)  # chunks
    assert minf.MINF_STATUS_BYTES < a < b
    assert f(minf.OP_PAGED_BLOCK_ESTIMATE, 32, 8, 16, 16, 1, 2048, 100) > 16 * 8 * 2048 * 4
    # rejected arguments size to 0
    assert f(minf.OP_PAGED_BLOCK_ESTIMATE, 32, 8, 16, 16, 1, 2048, 0) == 0
    assert f(minf.OP_PAGED_BLOCK_ESTIMATE, 32, 8, 16, 16, 1, 40000, 4) == 0
    assert f(minf.OP_PAGED_BLOCK_ATTENTION, 32, 8, 16, 16, 1, 2048, 0) == 0
    assert f(minf.OP_PAGED_ATTENTION, 32, 7, 16, 16, 1) == 0 and f(99, 32, 8, 16, 16, 1) == 0


def test_binding_refuses_cpu_tensors_and_wrong_counts(minf_lib):
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    kc = torch.zeros(3, 2, 64, 128, dtype=torch.bfloat16)
    t, cu, kv = torch.zeros(1, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA bf16 or fp16"):
        minf.minf_paged_attention(q, kc, kc, t, cu, kv, 1)
    with pytest.raises(ValueError, match="CUDA bf16 or fp16"):
        minf.minf_paged_append(q, q, kc, kc, t, cu, kv, 1)
    with pytest.raises(ValueError, match="must be a tensor"):
        minf.minf_paged_block_estimate(None, kc, t, cu, kv, 1)
    with pytest.raises(ValueError, match="arguments"):
        minf._paged().attention(q)


def test_block_attention_refuses_lists_longer_than_a_table_can_name(minf_lib):
    """2^26 pages of 16 tokens are all that a table names; longer lists would overflow the count of 16-key groups."""
    most = 1 << 26
    assert block_attention(topk=most + 1) == UNS and block_attention(topk=1 << 28) == UNS
    assert block_attention(topk=most, wsb=256) == WS  # the limit itself only lacks its workspace here
    f = minf.paged_workspace_bytes
    assert f(minf.OP_PAGED_BLOCK_ATTENTION, 4, 2, 3, 2, 2, 8, most) > 0
    assert f(minf.OP_PAGED_BLOCK_ATTENTION, 4, 2, 3, 2, 2, 8, most + 1) == 0


def sizes(rng):
    hkv = rng.choice([1, 2, 3, 8, 32, 128])
    group = rng.choice([1, 2, 4, 7, 8, 9, 16, 33, 128])
    total, width = int(2 ** rng.uniform(0, 14)), int(2 ** rng.uniform(0, 15))
    return min(256 // hkv, group) * hkv, hkv, total, rng.randint(1, min(total, 4096)), rng.randint(1, total), width, rng.randint(1, 300)


@pytest.mark.parametrize("seed", range(4))
def test_workspace_of_the_largest_step_serves_every_smaller_one(minf_lib, seed):
    """Sizes do not fall with the tokens, sequences, new tokens, table columns or list entries of a step, and
    a call takes a buffer that was sized for a larger one (past that check there is no device memory here)."""
    rng = random.Random(seed)
    f = minf.paged_workspace_bytes
    steps = [(8, 32, 200, 200, 1, 2048, 100, [(147, 147, 1, 2048, 100), (1, 1, 1, 2048, 100), (20, 4, 1, 2048, 100)])]
    for _ in range(300):
        hq, hkv, total, n_seqs, max_q, width, topk = sizes(rng)
        small = []
        for _ in range(4):
            t = rng.choice([total, rng.randint(1, total)])
            q = rng.randint(1, min(max_q, t))
            small.append((t, rng.randint(1, min(n_seqs, t)), q, rng.choice([width, rng.randint(1, width)]),
                          rng.choice([topk, rng.randint(1, topk)])))
        steps.append((hkv, hq, total, n_seqs, max_q, width, topk, small))
    for hkv, hq, total, n_seqs, max_q, width, topk, small in steps:
        for op in (minf.OP_PAGED_ATTENTION, minf.OP_PAGED_BLOCK_ESTIMATE, minf.OP_PAGED_BLOCK_ATTENTION):
            have = f(op, hq, hkv, total, n_seqs, max_q, width, topk)
            for t, n, q, w, k in small:
                assert 0 < f(op, hq, hkv, t, n, q, w, k) <= have, (op, hq, hkv, total, t, n, q, w, k)
                kw = dict(hq=hq, hkv=hkv, total=t, n_seqs=n, max_q=q, width=w, table_stride=w, wsb=have)
                page = rng.choice([16, 32, 64, 128])
                if op == minf.OP_PAGED_ATTENTION:
                    rc = attention(page_size=page, q=rows(hq), out=rows(hq), c=cache(page, hkv), **kw)
                elif op == minf.OP_PAGED_BLOCK_ESTIMATE:
                    rc = estimate(page_size=page, q=rows(hq), topk=k, **kw)
                else:
                    s = seqs(page_size=page, **{x: kw[x] for x in ("total", "n_seqs", "max_q", "width", "table_stride")})
                    rc = minf.lib().minf_paged_block_attention(ref(s), 0, hq, hkv, 128, ref(rows(hq)), ref(cache(page, hkv)),
                                                               0.1, FAKE, FAKE, k, ref(rows(hq)), None, FAKE, have, None)
                assert rc not in (0, WS, UNS), (op, rc, minf.lib().minf_last_error())
