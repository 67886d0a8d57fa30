"""The paged calls as a program uses them: together, in other layouts, on other streams, captured, over
long caches, and on arrays that contradict themselves."""
import math

import pytest
import torch

import paged_ref as ref
from dynamic_sparse_attention_est_b200 import minf, synth

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)
BF, HF = torch.bfloat16, torch.float16


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ together
def test_prompt_chunks_and_decoding_agree_with_the_prompt_kernels():
    """A prompt stored in three chunks and continued token by token: every chunk's attention equals the
    dense prompt kernel's rows over the same tokens, and with every page listed the selected-page
    attention equals the full one."""
    hq, hkv, n, page = 8, 2, 64 * 9, 64
    w = synth.Workload("t", "vs", hq, hkv, n, "vertical", n_heavy=8)
    x = synth.generate(w, seed=3)
    q, k, v = (x[i].cuda() for i in "qkv")  # [heads][n][128], keys rotated already
    dense, dense_lse = minf.minf_dense_attention(q, k, v, scale=SCALE)
    pages = n // page
    kc = torch.zeros(pages + 2, hkv, page, 128, dtype=BF, device="cuda")
    vc, kb = torch.zeros_like(kc), torch.zeros(pages + 2, hkv, 2, 128, dtype=BF, device="cuda")
    perm = torch.randperm(pages + 2, generator=torch.Generator().manual_seed(0))[:pages]
    table = perm.to(torch.int32).cuda().view(1, -1)
    qt, kt, vt = q.transpose(0, 1), k.transpose(0, 1), v.transpose(0, 1)  # views: tokens first
    got, got_lse, sel = torch.empty_like(qt.contiguous()), torch.empty(n, hq, device="cuda"), []
    edges = [0, 200, 201, 500] + list(range(501, n + 1))
    for a, b in zip(edges, edges[1:]):
        cu, kv = i32(0, b - a), i32(b)
        minf.minf_paged_append(kt[a:b], vt[a:b], kc, vc, table, cu, kv, b - a, k_bounds=kb)
        o, l = minf.minf_paged_attention(qt[a:b], kc, vc, table, cu, kv, b - a, scale=SCALE)
        got[a:b], got_lse[a:b] = o, l
        idx, cnt = minf.minf_paged_block_estimate(qt[a:b], kb, table, cu, kv, b - a, page_size=page, topk=pages)
        o2, l2 = minf.minf_paged_block_attention(qt[a:b], kc, vc, table, cu, kv, b - a, idx, cnt, scale=SCALE)
        assert torch.equal(cnt, (torch.arange(a, b, device="cuda") // page + 1)[:, None].expand(-1, hkv).int())
        sel.append((o2, l2))
    # two 16-bit roundings of the same sums on each side: outputs, and weights against sum p |v| <= max |v|
    tol = 2 * ref.u(BF) * (dense.float().abs() + v.float().abs().max())
    want, want_lse = dense.transpose(0, 1).float(), dense_lse.T
    assert ((got.float() - want).abs() <= tol.transpose(0, 1)).all()
    # a logit's error (2^-19 sum |q| |k| scale, and the exponential) on either side
    mag = (q.float().abs().sum(-1).max() * k.float().abs().max()) * SCALE
    assert ((got_lse - want_lse).abs() <= 2 * (float(mag) * 2 ** -19 + 2 ** -15)).all()
    o2, l2 = torch.cat([s[0] for s in sel]), torch.cat([s[1] for s in sel])
    assert ((o2.float() - want).abs() <= tol.transpose(0, 1)).all()
    assert ((l2 - want_lse).abs() <= 2 * (float(mag) * 2 ** -19 + 2 ** -15)).all()


def test_selection_finds_the_page_of_a_planted_key():
    """A key that a query asks for brings its page into the list, through append's bounds."""
    c = ref.Case([1], [64 * 40 + 7], 4, 1, 64, BF, seed=4)
    c.k_cache[int(c.tables[0, 17]), :, 33] = 6 * torch.nn.functional.normalize(c.q[0].float().sum(0), dim=0).to(BF) * 3
    kb = torch.nan_to_num(ref.bounds(c))
    idx, cnt = minf.minf_paged_block_estimate(c.q, kb, *c.meta(), topk=4)
    assert 17 in idx[0, 0].tolist() and idx[0, 0, 3] == 40


# ------------------------------------------------------------------ layouts
@pytest.mark.parametrize("lens,kv", [([1, 1], [300, 65]), ([40, 90], [300, 90])])
def test_head_major_rows_page_strides_and_output_views(lens, kv):
    """q and out as [heads][tokens] tensors seen tokens first, K and V of a page side by side, table rows
    inside a wider table."""
    c = ref.Case(lens, kv, 8, 2, 64, BF, seed=6, cache_gap=True)
    q = c.q.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.full((2, c.width + 5), -7, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + c.width] = c.tables
    buf = torch.zeros(8, c.total + 3, 128, dtype=BF, device="cuda")
    out = buf[:, 1:1 + c.total].transpose(0, 1)
    o, l = minf.minf_paged_attention(q, c.k_cache, c.v_cache, wide[:, 2:2 + c.width], c.cu, c.kv_lens, c.max_q,
                                     scale=SCALE, out=out)
    assert o.data_ptr() == out.data_ptr()
    ref.check(c, (o, l), ref.attention(c, SCALE))
    assert (buf[:, 0] == 0).all() and (buf[:, c.total + 1:] == 0).all()
    o2, none = minf.minf_paged_attention(q, c.k_cache, c.v_cache, *c.meta(), want_lse=False)
    assert none is None and torch.equal(o2, o.contiguous())


def test_offsets_past_32_bits():
    """Pages a gigabyte apart: element offsets of the last ones pass 2^32."""
    stride, pages = 1 << 29, 10  # elements; 10 GB each for keys and values
    big = torch.empty((pages - 1) * stride + 2 * 64 * 128, dtype=BF, device="cuda")
    bigv = torch.empty_like(big)
    kc = big.as_strided((pages, 2, 64, 128), (stride, 64 * 128, 128, 1))
    vc = bigv.as_strided((pages, 2, 64, 128), (stride, 64 * 128, 128, 1))
    for lens, n in (([1], 64 * 9 + 5), ([70], 64 * 9 + 60)):
        c = ref.Case(lens, [n], 4, 2, 64, BF, seed=n)
        c.tables = torch.arange(10, dtype=torch.int32, device="cuda").view(1, -1)
        for p in range(10):
            kc[p], vc[p] = 0, 0
        g = torch.Generator().manual_seed(1)
        k, v = torch.randn(n, 2, 128, generator=g).to(BF).cuda(), torch.randn(n, 2, 128, generator=g).to(BF).cuda()
        minf.minf_paged_append(k, v, kc, vc, c.tables, i32(0, n), i32(n), n)
        assert torch.equal(kc[9, :, 3], k[64 * 9 + 3]) and torch.equal(vc[9, :, 3], v[64 * 9 + 3])
        c.k_cache, c.v_cache = kc, vc
        ref.check(c, minf.minf_paged_attention(c.q, kc, vc, *c.meta(), scale=SCALE), ref.attention(c, SCALE))
        idx = torch.arange(10, dtype=torch.int32, device="cuda").expand(c.total, 2, 10).contiguous()
        cnt = torch.full((c.total, 2), 10, dtype=torch.int32, device="cuda")
        ref.check(c, minf.minf_paged_block_attention(c.q, kc, vc, *c.meta(), idx, cnt, scale=SCALE),
                  ref.attention(c, SCALE))


def test_values_that_reach_far():
    """Logits of hundreds, one key that outweighs the rest by far, weights below fp16's range."""
    for dtype in (BF, HF):
        for lens in ([1], [80]):
            c = ref.Case(lens, [700], 4, 1, 64, dtype, seed=9)
            c.q *= 8
            c.k_cache[:, :, 5] *= 4
            ref.check(c, minf.minf_paged_attention(c.q, c.k_cache, c.v_cache, *c.meta(), scale=SCALE),
                      ref.attention(c, SCALE))


# ------------------------------------------------------------------ streams, graphs, repeats
def test_equal_calls_give_equal_bits_on_any_stream():
    cases = [ref.Case([1] * 5, [3000, 64, 777, 1, 2000], 8, 2, 64, BF, seed=1),
             ref.Case([50, 200, 3], [50, 1500, 900], 8, 2, 64, BF, seed=2)]
    for c in cases:
        kb = torch.nan_to_num(ref.bounds(c))
        first = None
        for i in range(3):
            st = torch.cuda.Stream()
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                o, l = minf.minf_paged_attention(c.q, c.k_cache, c.v_cache, *c.meta())
                idx, cnt = minf.minf_paged_block_estimate(c.q, kb, *c.meta(), topk=8)
                o2, l2 = minf.minf_paged_block_attention(c.q, c.k_cache, c.v_cache, *c.meta(), idx, cnt)
            torch.cuda.current_stream().wait_stream(st)
            torch.cuda.synchronize()
            now = [t.clone() for t in (o, l, idx, cnt, o2, l2)]
            if first is None:
                first = now
            assert all(torch.equal(a, b) for a, b in zip(first, now))


def test_two_calls_at_once_with_their_own_workspaces():
    cases = [ref.Case([1] * 8, [4000 + 100 * i for i in range(8)], 8, 2, 64, BF, seed=1),
             ref.Case([300], [2500], 8, 2, 64, BF, seed=2)]
    want = [minf.minf_paged_attention(c.q, c.k_cache, c.v_cache, *c.meta()) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = []
        for c, st in zip(cases, streams):
            with torch.cuda.stream(st):
                got.append(minf.minf_paged_attention(c.q, c.k_cache, c.v_cache, *c.meta()))
        torch.cuda.synchronize()
        for (a, la), (b, lb) in zip(want, got):
            assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("new", [1, 24])
def test_captured_step_follows_the_lengths(new):
    """One captured step (append, attention, selection, selected-page attention) replayed as the sequences
    grow: every replay equals the eager step on the same state."""
    hq, hkv, page, n_seqs, steps = 8, 2, 16, 3, 4
    start = [5, 200, 77]
    g = torch.Generator().manual_seed(3)
    width, pages = 24, 80
    tables = torch.randperm(pages, generator=g)[:n_seqs * width].to(torch.int32).view(n_seqs, width).cuda()
    tab = ref.rope_table(width * page, 128)
    total = new * n_seqs
    cu = i32(*range(0, total + 1, new))
    rows = [torch.randn(total, hq + 2 * hkv, 128, generator=g).to(BF).cuda() for _ in range(steps)]

    def caches():
        kc = torch.randn(pages, hkv, page, 128, generator=torch.Generator().manual_seed(5)).to(BF).cuda()
        vc = torch.randn(pages, hkv, page, 128, generator=torch.Generator().manual_seed(6)).to(BF).cuda()
        return kc, vc, torch.stack(kc.aminmax(dim=2), 2).contiguous()

    def step(x, kc, vc, kb, kv):
        q = minf.minf_paged_append(x[:, hq:hq + hkv], x[:, hq + hkv:], kc, vc, tables, cu, kv, new, rope=tab, q=x[:, :hq],
                                   k_bounds=kb, ws=ws)
        o, l = minf.minf_paged_attention(q, kc, vc, tables, cu, kv, new, ws=ws)
        idx, cnt = minf.minf_paged_block_estimate(q, kb, tables, cu, kv, new, page_size=page, topk=5, ws=ws)
        o2, l2 = minf.minf_paged_block_attention(q, kc, vc, tables, cu, kv, new, idx, cnt, ws=ws)
        return o, l, idx, cnt, o2, l2

    need = max(minf.paged_workspace_bytes(op, hq, hkv, total, n_seqs, new, width, 5)
               for op in (minf.OP_PAGED_APPEND, minf.OP_PAGED_ATTENTION, minf.OP_PAGED_BLOCK_ESTIMATE,
                          minf.OP_PAGED_BLOCK_ATTENTION))
    ws = minf.workspace(need, "cuda")  # one after the other: the four calls and both graphs share it
    eager = []
    kc, vc, kb = caches()
    kv = i32(*start)
    for x in rows:
        kv += new
        eager.append([t.clone() for t in step(x, kc, vc, kb, kv)])
    x_in, kc, vc, kb = rows[0].clone(), *caches()
    kv = i32(*start)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kv += new
        outs = step(x_in, kc, vc, kb, kv)
    with torch.cuda.graph(other, stream=side):
        minf.minf_paged_attention(x_in[:, :hq], kc, vc, tables, cu, kv, new, ws=ws)
    for x, want in zip(rows, eager):
        x_in.copy_(x)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        other.replay()
    assert minf.minf_status(ws) == 0


# ------------------------------------------------------------------ arrays that contradict themselves
def run_all(c, ws, topk=4):
    kb = torch.zeros(c.num_pages, c.hkv, 2, 128, dtype=c.dtype, device="cuda")
    kc, vc = torch.nan_to_num(c.k_cache), torch.nan_to_num(c.v_cache)
    idx = torch.zeros(c.total, c.hkv, topk, dtype=torch.int32, device="cuda")
    cnt = torch.ones(c.total, c.hkv, dtype=torch.int32, device="cuda")
    yield minf.minf_paged_append(c.k_new, c.v_new, kc, vc, *c.meta(), q=c.q, k_bounds=kb, ws=ws)
    yield minf.minf_paged_attention(c.q, kc, vc, *c.meta(), ws=ws)
    yield minf.minf_paged_block_estimate(c.q, kb, *c.meta(), page_size=c.page, topk=topk, ws=ws)
    yield minf.minf_paged_block_attention(c.q, kc, vc, *c.meta(), idx, cnt, ws=ws)


@pytest.mark.parametrize("lens", [[1, 1, 2], [90, 5, 70]])
@pytest.mark.parametrize("fault", ["length", "negative", "page", "starts", "max_q"])
def test_bad_lengths_and_pages_are_reported_and_left_out(lens, fault):
    """Sequence 1 carries the fault: the status says so, and the other sequences' results stand."""
    kv = [300, 90, 400]
    c = ref.Case(lens, kv, 4, 2, 64, BF, seed=12)
    want = ref.attention(c, SCALE)
    if fault == "length":
        c.kv_lens[1] = c.width * 64 + 1
    elif fault == "negative":
        c.kv_lens[1] = -5
    elif fault == "page":
        c.tables[1, 0] = c.num_pages
    elif fault == "starts":
        c.cu[2] = c.cu[1] - 1  # sequence 1 ends before it begins, and 2 takes its rows
    else:
        c.max_q -= 1
    ws = minf.workspace(max(minf.paged_workspace_bytes(op, 4, 2, c.total, 3, max(lens), c.width, 4) for op in
                            (minf.OP_PAGED_ATTENTION, minf.OP_PAGED_BLOCK_ESTIMATE, minf.OP_PAGED_BLOCK_ATTENTION)),
                        "cuda")
    for call, _ in enumerate(run_all(c, ws)):
        # the append stores into the sequence's second page only: it has no use for the bad first one
        unread = fault == "page" and call == 0
        assert minf.minf_status(ws) == (0 if unread else minf.MINF_ERR_INVALID), call
        assert minf.minf_status(ws) == 0  # reported once
    if fault == "page":
        out, lse = minf.minf_paged_attention(c.q, c.k_cache, c.v_cache, *c.meta(), scale=SCALE, ws=ws)
        keep = torch.cat([torch.arange(lens[0]), torch.arange(lens[0] + lens[1], sum(lens))])
        ref_o, ref_l, to, tl = (t[keep] for t in want)
        assert ((out[keep].double() - ref_o).abs() <= to).all() and ((lse[keep].double() - ref_l).abs() <= tl).all()
        minf.minf_status(ws)


def test_bad_list_counts_are_reported():
    c = ref.Case([1], [200], 4, 1, 64, BF, seed=1)
    ws = minf.workspace(minf.paged_workspace_bytes(minf.OP_PAGED_BLOCK_ATTENTION, 4, 1, 1, 1, 1, c.width, 2), "cuda")
    idx = i32(0, 1).view(1, 1, 2)
    for n in (-3, 7):
        minf.minf_paged_block_attention(c.q, c.k_cache, c.v_cache, *c.meta(), idx, i32(n).view(1, 1), ws=ws)
        assert minf.minf_status(ws) == minf.MINF_ERR_INVALID
        assert "list" in minf.lib().minf_last_error().decode()


def test_append_reports_positions_it_has_no_rotation_for():
    c = ref.Case([2], [40], 4, 2, 16, BF, seed=1)
    ws = minf.workspace(256, "cuda")
    before = c.k_cache.clone()
    minf.minf_paged_append(c.k_new, c.v_new, c.k_cache, c.v_cache, *c.meta(), rope=ref.rope_table(39, 128), ws=ws)
    assert minf.minf_status(ws) == minf.MINF_ERR_INVALID
    assert torch.equal(c.k_cache.view(torch.int16), before.view(torch.int16))
    c.kv_lens[0] = 1  # two new tokens, one stored
    minf.minf_paged_append(c.k_new, c.v_new, c.k_cache, c.v_cache, *c.meta(), ws=ws)
    assert minf.minf_status(ws) == minf.MINF_ERR_INVALID


# ------------------------------------------------------------------ many sequences, many tokens
def test_many_sequences():
    """4,096 sequences in one call (prefix sums of several sequences to a thread)."""
    lens, kv = [1] * 4096, [1 + (i * 7) % 40 for i in range(4096)]
    c = ref.Case(lens, kv, 2, 1, 16, BF, seed=3)
    out, lse = minf.minf_paged_attention(c.q, c.k_cache, c.v_cache, *c.meta(), scale=SCALE)
    some = list(range(0, 4096, 37)) + [4095]
    for s in some:
        k, v = c.stored(s, 0, kv[s])
        x = c.q[s].double() @ k.T * SCALE
        p = torch.softmax(x, 1)
        tol = ref.u(BF) * ((p @ v).abs() + p @ v.abs()) + 1e-4
        assert ((out[s].double() - p @ v).abs() <= tol).all(), s
        assert ((lse[s].double() - torch.logsumexp(x, 1)).abs() <= 1e-4).all()
    # the chunk kernel on the same sequences (two tokens in one of them make it the larger call)
    c2 = ref.Case([1] * 4095 + [17], kv[:-1] + [30], 2, 1, 16, BF, seed=3)
    out2, _ = minf.minf_paged_attention(c2.q, c2.k_cache, c2.v_cache, *c2.meta(), scale=SCALE)
    for s in some[:-1]:
        k, v = c2.stored(s, 0, kv[s])
        p = torch.softmax(c2.q[s].double() @ k.T * SCALE, 1)
        tol = ref.u(BF) * ((p @ v).abs() + p @ v.abs()) + 1e-4
        assert ((out2[s].double() - p @ v).abs() <= tol).all(), s


def test_estimate_in_batches_of_tokens():
    """A table so wide that the scores of 64 tokens fill the scratch: three batches, tiles cut at their edges."""
    c = ref.Case([90, 1, 60], [1000, 500, 60], 8, 8, 16, BF, seed=8, gap=32600)
    kb = torch.nan_to_num(ref.bounds(c))
    idx, cnt = minf.minf_paged_block_estimate(c.q, kb, *c.meta(), page_size=16, topk=9)
    wi, wc = ref.estimate(c, kb, 9)
    assert torch.equal(cnt, wc) and torch.equal(idx, wi)


def test_estimate_decides_scores_that_differ_in_the_last_bits():
    """Pages equal but for one step of one channel: far closer than the approximate scores resolve."""
    c = ref.Case([3], [16 * 300 + 2], 4, 2, 16, BF, seed=8)
    base = torch.sort(torch.randn(2, 2, 128, generator=torch.Generator().manual_seed(1)), dim=1).values.to(BF).cuda()
    kb = base.expand(c.num_pages, 2, 2, 128).contiguous()
    bits = kb.view(torch.int16)
    g = torch.Generator().manual_seed(2)
    ch = torch.randint(0, 128, (c.num_pages,), generator=g).cuda()
    bits[torch.arange(c.num_pages, device="cuda"), :, 1, ch] += torch.randint(0, 2, (c.num_pages, 1), generator=g).cuda().to(torch.int16)
    idx, cnt = minf.minf_paged_block_estimate(c.q, kb, *c.meta(), page_size=16, topk=40)
    wi, wc = ref.estimate(c, kb, 40)
    assert torch.equal(cnt, wc) and torch.equal(idx, wi)


@pytest.mark.parametrize("lens,pages", [([2], 60), ([300], 300), ([300], 1500)])
@pytest.mark.parametrize("what", ["inf", "nan", "all_inf"])
def test_estimate_stays_in_its_lists_whatever_the_bounds_hold(lens, pages, what):
    """Bounds that are not finite: which pages are taken is unspecified, but the lists are lists of pages
    before the token's own, ascending and distinct, with the own page last."""
    c = ref.Case(lens, [16 * pages + lens[0]], 4, 2, 16, HF, seed=1)
    kb = torch.nan_to_num(ref.bounds(c))
    bad = {"inf": math.inf, "nan": math.nan, "all_inf": math.inf}[what]
    if what == "all_inf":
        kb[:, :, 1] = bad
    else:
        kb[::3, :, 1, 5] = bad
    idx, cnt = minf.minf_paged_block_estimate(c.q, kb, *c.meta(), page_size=16, topk=20)
    pos = torch.arange(c.kv[0] - lens[0], c.kv[0], device="cuda") // 16
    assert (cnt <= 20).all() and (cnt >= 1).all()
    own = idx.gather(2, (cnt - 1).long()[..., None])[..., 0]
    assert torch.equal(own, pos[:, None].expand_as(own).int())
