"""The paged key/value cache operators on the GPU against their plain 64-bit forms."""
import math

import pytest
import torch

import paged_ref as ref
from dynamic_sparse_attention_est_b200 import minf

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)
BF, HF = torch.bfloat16, torch.float16


rope_table = ref.rope_table


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("lens,kv,hq,hkv,page,dtype,rot,inter", [
    ([1], [1], 4, 1, 64, BF, 128, False),
    ([1, 1, 1], [64, 65, 300], 8, 2, 64, BF, 128, False),
    ([130, 0, 3], [130, 77, 67], 6, 2, 64, BF, 64, False),
    ([5, 40, 1], [15, 57, 33], 2, 2, 16, HF, 96, True),
    ([200], [333], 12, 4, 128, HF, 16, False),
    ([33, 31], [33, 63], 4, 4, 32, BF, 128, True),
])
def test_append(lens, kv, hq, hkv, page, dtype, rot, inter):
    c = ref.Case(lens, kv, hq, hkv, page, dtype, seed=len(lens) + page, extra_rows=2)
    tab = rope_table(max(kv), rot)
    kc0, vc0 = c.k_cache.clone(), c.v_cache.clone()
    # bounds as they stood before: over the tokens stored until now, NaN-free elsewhere
    c0 = ref.Case(lens, kv, hq, hkv, page, dtype, seed=len(lens) + page, extra_rows=2)
    c0.kv = [x - n for x, n in zip(kv, lens)]
    kb = torch.nan_to_num(ref.bounds(c0), nan=7.0)
    kb0 = kb.clone()
    fused = torch.cat([c.q, c.k_new, c.v_new], 1)  # strided slices of one projection
    q, k, v = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    q_out = torch.full((c.total, hq, 128), 3.0, dtype=dtype, device="cuda")
    ws = minf.workspace(256, c.dev)
    got = minf.minf_paged_append(k, v, c.k_cache, c.v_cache, *c.meta(), rope=tab, interleaved=inter, q=q, q_out=q_out,
                                 k_bounds=kb, ws=ws)
    assert got is q_out and minf.minf_status(ws) == 0
    rows = list(c.rows())
    pos = torch.tensor([p for _, _, p in rows], device="cuda")
    n = len(rows)
    yq, tq = ref.rotate(q[:n], tab, pos, rot, inter)
    yk, tk = ref.rotate(k[:n], tab, pos, rot, inter)
    assert ((q_out[:n].double() - yq).abs() <= tq).all()
    assert (q_out[n:] == 3.0).all()  # rows of no sequence
    touched = torch.zeros(c.num_pages, page, dtype=torch.bool, device="cuda")
    for (s, r, p) in rows:
        pg = int(c.tables[s, p // page])
        touched[pg, p % page] = True
        assert ((c.k_cache[pg, :, p % page].double() - yk[r]).abs() <= tk[r]).all()
        assert torch.equal(c.v_cache[pg, :, p % page], v[r])
    keep = ~touched[:, None, :, None].expand_as(c.k_cache)
    assert torch.equal(c.k_cache[keep].view(torch.int16), kc0[keep].view(torch.int16))
    assert torch.equal(c.v_cache[keep].view(torch.int16), vc0[keep].view(torch.int16))
    for s, (m, x) in enumerate(zip(lens, kv)):
        first, last = (x - m) // page, (x - 1) // page
        for b in range(-(-x // page)):
            pg = int(c.tables[s, b])
            if m == 0 or not first <= b <= last:
                assert torch.equal(kb[pg], kb0[pg])
                continue
            keys = c.k_cache[pg, :, :min(page, x - b * page)]
            assert torch.equal(kb[pg, :, 0], keys.amin(1)) and torch.equal(kb[pg, :, 1], keys.amax(1))


def test_append_without_rotation_in_place_and_split_calls():
    """No table: rows are copied; q rotated in place; tokens appended one by one leave what one call leaves."""
    c = ref.Case([9], [25], 4, 2, 16, BF, seed=3)
    tab = rope_table(25, 128)
    a = minf.minf_paged_append(c.k_new, c.v_new, c.k_cache, c.v_cache, *c.meta())
    assert a is None
    for s, r, p in c.rows():
        assert torch.equal(c.k_cache[int(c.tables[0, p // 16]), :, p % 16], c.k_new[r])
    kb1 = torch.zeros(c.num_pages, 2, 2, 128, dtype=BF, device="cuda")
    kb2 = kb1.clone()
    q = c.q.clone()
    out = minf.minf_paged_append(c.k_new, c.v_new, c.k_cache, c.v_cache, *c.meta(), rope=tab, q=c.q, k_bounds=kb1)
    minf.minf_paged_append(c.k_new, c.v_new, c.k_cache, c.v_cache, *c.meta(), rope=tab, q=q, q_out=q)
    assert torch.equal(q, out)
    k2, v2 = torch.nan_to_num(c.k_cache) * 0, torch.nan_to_num(c.v_cache) * 0
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for s, r, p in c.rows():
        n = torch.tensor([p + 1], dtype=torch.int32, device="cuda")
        minf.minf_paged_append(c.k_new[r:r + 1], c.v_new[r:r + 1], k2, v2, c.tables, one, n, 1, rope=tab, k_bounds=kb2)
    for s, r, p in c.rows():
        at = (int(c.tables[0, p // 16]), slice(None), p % 16)
        assert torch.equal(k2[at], c.k_cache[at]) and torch.equal(v2[at], c.v_cache[at])
    assert torch.equal(kb1, kb2)


# ------------------------------------------------------------------ attention, few rows
DECODE = [
    # lens, kv, hq, hkv, page, dtype
    ([1], [1], 1, 1, 64, BF),
    ([1], [129], 8, 2, 64, BF),
    ([1, 1, 1, 1], [5, 64, 1000, 4097], 8, 2, 64, BF),
    ([1, 0, 1], [17, 40, 33], 7, 7, 16, HF),
    ([2, 1, 4, 3], [100, 2, 4, 77], 8, 2, 32, BF),
    ([1, 1], [700, 300], 16, 1, 128, HF),
    ([1, 1], [700, 300], 10, 1, 128, BF),
    ([3, 2, 1], [1, 0, 50], 4, 2, 16, BF),      # fewer stored tokens than new ones: rows that see no key
    ([1] * 40, list(range(1, 41)), 4, 4, 16, BF),
]


@pytest.mark.parametrize("lens,kv,hq,hkv,page,dtype", DECODE)
def test_decode(lens, kv, hq, hkv, page, dtype):
    c = ref.Case(lens, kv, hq, hkv, page, dtype, seed=sum(kv), extra_rows=1, gap=1)
    out = torch.full((c.total, hq, 128), 9.0, dtype=dtype, device="cuda")
    ws = minf.workspace(minf.paged_workspace_bytes(minf.OP_PAGED_ATTENTION, hq, hkv, c.total, len(lens), c.max_q),
                        c.dev)
    got = minf.minf_paged_attention(c.q, c.k_cache, c.v_cache, *c.meta(), scale=SCALE, out=out, ws=ws)
    assert minf.minf_status(ws) == 0
    ref.check(c, got, ref.attention(c, SCALE))
    assert (out[sum(lens):] == 9.0).all()


# ------------------------------------------------------------------ attention over selected pages
@pytest.mark.parametrize("lens,kv,hq,hkv,page,dtype,topk", [
    ([1], [1], 4, 1, 64, BF, 1),
    ([1], [5000], 8, 2, 64, BF, 20),             # split over CTAs
    ([3, 0, 5], [400, 9, 333], 8, 2, 16, HF, 7),
    ([40], [700], 32, 1, 32, BF, 9),             # four row tiles to a group
    ([2, 2], [1, 260], 6, 2, 128, BF, 3),        # a token that sees no key
])
def test_block_attention(lens, kv, hq, hkv, page, dtype, topk):
    c = ref.Case(lens, kv, hq, hkv, page, dtype, seed=topk, extra_rows=1)
    g = torch.Generator().manual_seed(5)
    idx = torch.full((c.total, hkv, topk), -1, dtype=torch.int32)
    cnt = torch.zeros(c.total, hkv, dtype=torch.int32)
    for s, r, pos in c.rows():
        for h in range(hkv):
            n = max(0, pos // page + 1) if pos >= 0 else 0
            k = int(torch.randint(0, min(n, topk) + 1, (1,), generator=g)) if r % 3 == 0 else min(n, topk)
            idx[r, h, :k] = torch.randperm(max(n, 1), generator=g)[:k].sort().values.int()
            cnt[r, h] = k
    pages = [[set(idx[r, h, :cnt[r, h]].tolist()) for h in range(hkv)] for r in range(c.total)]

    def pick(s, r, h, pos):
        return torch.tensor([(i // page) in pages[r][h] for i in range(pos + 1)], dtype=torch.bool, device="cuda")

    out = torch.full((c.total, hq, 128), 9.0, dtype=dtype, device="cuda")
    ws = minf.workspace(minf.paged_workspace_bytes(minf.OP_PAGED_BLOCK_ATTENTION, hq, hkv, c.total, len(lens),
                                                   c.max_q, c.width, topk), c.dev)
    got = minf.minf_paged_block_attention(c.q, c.k_cache, c.v_cache, *c.meta(), idx.cuda(), cnt.cuda(), scale=SCALE,
                                          out=out, ws=ws)
    assert minf.minf_status(ws) == 0
    ref.check(c, got, ref.attention(c, SCALE, pick))
    assert (out[sum(lens):] == 9.0).all()


def test_block_attention_leaves_out_bad_entries():
    """Negative entries, pages past the token's own and entries not above the one before."""
    c = ref.Case([1], [70], 4, 1, 16, BF, seed=8)
    lists = {(-1, 0, 2, 2, 1, 4, 9): {0, 2, 4}, (3, 3, 3, 3, 3, 3, 3): {3}, (-5, -1, 5, 6, 7, 8, 9): set()}
    for entries, pages in lists.items():
        idx = torch.tensor(entries, dtype=torch.int32, device="cuda").view(1, 1, 7)
        cnt = torch.full((1, 1), 7, dtype=torch.int32, device="cuda")

        def pick(s, r, h, pos):
            return torch.tensor([(i // 16) in pages for i in range(pos + 1)], dtype=torch.bool, device="cuda")

        got = minf.minf_paged_block_attention(c.q, c.k_cache, c.v_cache, *c.meta(), idx, cnt, scale=SCALE)
        ref.check(c, got, ref.attention(c, SCALE, pick))


# ------------------------------------------------------------------ page selection
@pytest.mark.parametrize("lens,kv,hq,hkv,page,dtype,topk", [
    ([1], [1], 4, 1, 64, BF, 4),
    ([1, 1, 1], [640, 5000, 64 * 37], 8, 2, 64, BF, 10),
    ([70, 0, 3], [1500, 16, 900], 6, 2, 16, BF, 12),
    ([37], [2000], 4, 4, 16, HF, 30),
    ([2, 3], [1, 800], 8, 1, 32, HF, 1),
    ([1], [16 * 1200 + 5], 4, 2, 16, BF, 100),
])
@pytest.mark.parametrize("bias", [0.0, 2.0])
def test_block_estimate(lens, kv, hq, hkv, page, dtype, topk, bias):
    c = ref.Case(lens, kv, hq, hkv, page, dtype, seed=topk, extra_rows=1, bias=bias)
    kb = ref.bounds(c)
    ws = minf.workspace(minf.paged_workspace_bytes(minf.OP_PAGED_BLOCK_ESTIMATE, hq, hkv, c.total, len(lens),
                                                   c.max_q, c.width, topk), c.dev)
    idx, cnt = minf.minf_paged_block_estimate(c.q, kb, *c.meta(), page_size=page, topk=topk, ws=ws)
    assert minf.minf_status(ws) == 0
    wi, wc = ref.estimate(c, kb, topk)
    n = sum(lens)
    assert torch.equal(cnt[:n], wc[:n])
    assert torch.equal(idx[:n], wi[:n])


@pytest.mark.parametrize("n_proto,pages", [(1, 60), (3, 300), (2, 1500)])
def test_block_estimate_ties_go_to_the_lower_page(n_proto, pages):
    """Pages copied from a few prototypes score alike to the last bit: from a few in doubt
    to more than a row ranks in shared memory."""
    c = ref.Case([2], [pages * 16 + 7], 4, 2, 16, BF, seed=n_proto)
    g = torch.Generator().manual_seed(1)
    proto = torch.sort(torch.randn(n_proto, 2, 2, 128, generator=g), dim=2).values.to(BF).cuda()
    kb = torch.zeros(c.num_pages, 2, 2, 128, dtype=BF, device="cuda")
    kb[c.tables[0, :pages].long()] = proto[torch.randint(0, n_proto, (pages,), generator=g)]
    idx, cnt = minf.minf_paged_block_estimate(c.q, kb, *c.meta(), page_size=16, topk=25)
    wi, wc = ref.estimate(c, kb, 25)
    assert torch.equal(cnt, wc) and torch.equal(idx, wi)


# ------------------------------------------------------------------ attention, chunks
CHUNK = [
    ([17], [17], 4, 1, 64, BF),
    ([64], [64], 8, 2, 64, BF),
    ([65, 1, 130], [65, 129, 1000], 8, 2, 64, BF),
    ([200], [2000], 4, 4, 16, HF),
    ([33, 0, 7, 64], [333, 50, 9, 64], 12, 4, 32, HF),
    ([50], [700], 6, 2, 128, BF),
    ([40, 30], [10, 0], 8, 2, 64, BF),           # rows that see no key
    ([3], [3000], 64, 1, 64, BF),
    ([2, 2], [257, 255], 128, 1, 64, BF),
    ([300], [300], 5, 1, 16, BF),                # 25 tokens to a tile, rows left over
]


@pytest.mark.parametrize("lens,kv,hq,hkv,page,dtype", CHUNK)
def test_chunk(lens, kv, hq, hkv, page, dtype):
    c = ref.Case(lens, kv, hq, hkv, page, dtype, seed=sum(kv), extra_rows=1, gap=1)
    out = torch.full((c.total, hq, 128), 9.0, dtype=dtype, device="cuda")
    ws = minf.workspace(minf.paged_workspace_bytes(minf.OP_PAGED_ATTENTION, hq, hkv, c.total, len(lens), c.max_q),
                        c.dev)
    got = minf.minf_paged_attention(c.q, c.k_cache, c.v_cache, *c.meta(), scale=SCALE, out=out, ws=ws)
    assert minf.minf_status(ws) == 0
    ref.check(c, got, ref.attention(c, SCALE))
    assert (out[sum(lens):] == 9.0).all()


def test_chunk_many_units_of_one_and_two_row_tiles():
    """Several units to a CTA, pairs of row tiles and single ones in every order."""
    g = torch.Generator().manual_seed(7)
    lens = torch.randint(1, 90, (70,), generator=g).tolist()
    lens = [1 if i % 3 == 1 else n for i, n in enumerate(lens)]
    kv = [n + int(x) for n, x in zip(lens, torch.randint(0, 400, (70,), generator=g))]
    c = ref.Case(lens, kv, 16, 8, 16, HF, seed=11)
    ws = minf.workspace(minf.paged_workspace_bytes(minf.OP_PAGED_ATTENTION, 16, 8, c.total, 70, c.max_q), c.dev)
    got = minf.minf_paged_attention(c.q, c.k_cache, c.v_cache, *c.meta(), scale=SCALE, ws=ws)
    assert minf.minf_status(ws) == 0
    ref.check(c, got, ref.attention(c, SCALE))


def test_block_estimate_tiles_of_a_chunk_agree_on_the_largest_bound():
    """Tiles of one sequence end at different pages of a 16-page step; the last page of the
    step holds by far the largest bounds, which the later tiles' error bound must cover."""
    c = ref.Case([200], [200 + 16 * 20], 4, 2, 16, BF, seed=2)
    kb = ref.bounds(c)
    pages = c.tables[0, :32].long()
    kb[pages[27], :, 1] *= 50
    kb = torch.nan_to_num(kb)
    idx, cnt = minf.minf_paged_block_estimate(c.q, kb, *c.meta(), page_size=16, topk=9)
    wi, wc = ref.estimate(c, kb, 9)
    assert torch.equal(cnt, wc) and torch.equal(idx, wi)


def test_block_estimate_many_rows_and_long_rows():
    """A warp per row (many rows of at most 2,048 pages), and a CTA per row beyond."""
    for lens, kv, page in (([350, 250], [9000, 5000], 16), ([140], [16 * 2500], 16)):
        c = ref.Case(lens, kv, 4, 2, page, BF, seed=5)
        kb = torch.nan_to_num(ref.bounds(c))
        idx, cnt = minf.minf_paged_block_estimate(c.q, kb, *c.meta(), page_size=page, topk=33)
        wi, wc = ref.estimate(c, kb, 33)
        assert torch.equal(cnt, wc) and torch.equal(idx, wi)


def test_append_and_estimate_of_a_chunk_beside_many_single_tokens():
    """The longest sequence far above the others: pages and tiles are found by what all tokens touch."""
    lens = [1] * 40 + [0, 500] + [1] * 30 + [3, 700, 0]
    kv = [1 + (i * 37) % 200 for i in range(len(lens))]
    kv = [max(n, x) + (i % 5) for i, (n, x) in enumerate(zip(lens, kv))]
    c = ref.Case(lens, kv, 4, 2, 16, BF, seed=21, extra_rows=3)
    kb0 = torch.nan_to_num(ref.bounds(c))
    idx, cnt = minf.minf_paged_block_estimate(c.q, kb0, *c.meta(), page_size=16, topk=6)
    wi, wc = ref.estimate(c, kb0, 6)
    n = sum(lens)
    assert torch.equal(cnt[:n], wc[:n]) and torch.equal(idx[:n], wi[:n])
    tab = rope_table(max(kv), 128)
    kc, vc = torch.zeros_like(c.k_cache), torch.zeros_like(c.v_cache)
    kb = torch.zeros(c.num_pages, 2, 2, 128, dtype=BF, device="cuda")
    ws = minf.workspace(256, c.dev)
    q = minf.minf_paged_append(c.k_new, c.v_new, kc, vc, *c.meta(), rope=tab, q=c.q, k_bounds=kb, ws=ws)
    assert minf.minf_status(ws) == 0
    rows = list(c.rows())
    pos = torch.tensor([p for _, _, p in rows], device="cuda")
    yk, tk = ref.rotate(c.k_new[:n], tab, pos, 128, False)
    yq, tq = ref.rotate(c.q[:n], tab, pos, 128, False)
    assert ((q[:n].double() - yq).abs() <= tq).all()
    seq = torch.tensor([s for s, _, _ in rows], device="cuda")
    page = c.tables[seq, pos // 16].long()
    assert ((kc[page, :, pos % 16].double() - yk).abs() <= tk).all()
    assert torch.equal(vc[page, :, pos % 16], c.v_new[:n])
    written = torch.zeros(c.num_pages, 16, dtype=torch.bool, device="cuda")
    written[page, pos % 16] = True
    assert not kc.transpose(1, 2)[~written].any() and not vc.transpose(1, 2)[~written].any()
    for s, (m, x) in enumerate(zip(lens, kv)):
        for b in range((x - m) // 16, (x - 1) // 16 + 1 if m else 0):
            pg, a = int(c.tables[s, b]), max(0, x - m - 16 * b)
            keys = kc[pg, :, a:min(16, x - 16 * b)]
            lo, hi = keys.amin(1), keys.amax(1)
            if a:  # joined with what stood there: zeros
                lo, hi = lo.clamp(max=0), hi.clamp(min=0)
            assert torch.equal(kb[pg, :, 0], lo) and torch.equal(kb[pg, :, 1], hi)


def test_chunk_with_whole_rounds_uncut():
    """One sequence whose row-tile pairs fill the SMs once and a third: the first round's pairs stay
    whole, the rest are cut and joined."""
    n, kv, hq, hkv = 1275, 3300, 40, 10
    c = ref.Case([n, 0], [kv, 9], hq, hkv, 64, BF, seed=31)
    out, lse = minf.minf_paged_attention(c.q, c.k_cache, c.v_cache, *c.meta(), scale=SCALE)
    hide = torch.arange(kv, device="cuda") > torch.arange(kv - n, kv, device="cuda")[:, None]
    for h in range(hq):
        k, v = c.stored(0, h // 4, kv)
        x = (c.q[:, h].double() @ k.T) * SCALE
        d = 2 ** -19 * float((c.q[:, h].double().abs() @ k.abs().T).max()) * SCALE + 2 ** -19  # error of a logit
        x.masked_fill_(hide, -math.inf)
        z = torch.logsumexp(x, 1)
        p = (x - z[:, None]).exp()
        tol = ref.u(BF) * (p @ v).abs() + (ref.u(BF) + 2 * d) * (p @ v.abs()) + 1e-7
        assert ((out[:, h].double() - p @ v).abs() <= tol).all(), h
        assert ((lse[:, h].double() - z).abs() <= d + kv * 2 ** -24 + 1e-5).all(), h
