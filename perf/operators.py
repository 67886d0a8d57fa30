"""Cases of the paged key/value cache operators, with their plain and exact forms.

The operators carry a sequence on after its prompt: `minf_paged_append` rotates
new keys (and queries) and stores keys and values in a paged cache,
`minf_paged_attention` attends a chunk of new tokens (one token in decoding)
to everything stored, `minf_paged_block_estimate` picks, for each new token and
kv-head, the pages whose key bounds promise the largest logits, and
`minf_paged_block_attention` attends to the picked pages only.

Layouts (d = 128, G = hq / hkv, P = page size, everything on one device):

    q [tokens][hq][d]; k, v [tokens][hkv][d]      any token and head stride
    k_cache, v_cache [pages][hkv][P][d]           bf16 or fp16
    k_bounds [pages][hkv][2][d]                   smallest and largest stored key, per channel
    block_tables [seqs][width] int32              page of each P tokens of a sequence
    cu_q [seqs + 1] int32, kv_lens [seqs] int32   new tokens of sequence s: rows cu_q[s] .. cu_q[s + 1) - 1,
                                                  at positions kv_lens[s] - n .. kv_lens[s] - 1
    rope [positions][rot] fp32                    cosines in the first half of a row, sines in the second
"""
import math

import torch

own = False

D = 128
SCALE = 1.0 / math.sqrt(D)
THETA = 500000.0

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step of a small batch: the latency of a launch
        {"name": "append-decode-8", "op": "append", "lens": "1x8", "ctx": "uniform:900:9000", "hq": 32, "hkv": 8,
         "page": 64, "type": "bf16", "rot": 128, "interleaved": False},
        # a chunk of a long prompt, strided out of one fused projection
        {"name": "append-chunk-8192", "op": "append", "lens": "8192x1", "ctx": "fixed:24611", "hq": 32, "hkv": 8,
         "page": 64, "type": "bf16", "rot": 128, "interleaved": False},
        # chunks and single tokens of many sequences in one step, pages that begin half full
        {"name": "append-ragged-fp16", "op": "append", "lens": "ragged:37:1:700", "ctx": "uniform:0:3000", "hq": 12,
         "hkv": 4, "page": 16, "type": "fp16", "rot": 64, "interleaved": True},
        # one decoding step of a small batch at short contexts
        {"name": "attend-decode-4x4k", "op": "attend", "lens": "1x4", "ctx": "uniform:1000:4095", "hq": 32, "hkv": 8,
         "page": 64, "type": "bf16"},
        # one decoding step of a serving batch with mixed context lengths
        {"name": "attend-decode-64x32k", "op": "attend", "lens": "1x64", "ctx": "uniform:257:32767", "hq": 32,
         "hkv": 8, "page": 64, "type": "bf16"},
        # a chunk of a long prompt over what is stored of it (the flagship's lengths)
        {"name": "attend-chunk-2048x128k", "op": "attend", "lens": "2048x1", "ctx": "fixed:129024", "hq": 32,
         "hkv": 8, "page": 64, "type": "bf16"},
        # prompt chunks and decoding sequences in one step, small pages, three q-heads to a kv-head
        {"name": "attend-mixed-fp16", "op": "attend", "lens": "ragged:21:1:900", "ctx": "uniform:0:12000", "hq": 24,
         "hkv": 8, "page": 16, "type": "fp16"},
        # a decoding step's page selection at 128K tokens
        {"name": "estimate-decode-16x128k", "op": "estimate", "lens": "1x16", "ctx": "uniform:100000:131071",
         "hq": 32, "hkv": 8, "page": 64, "type": "bf16", "topk": 100},
        # page selection of every token of a chunk
        {"name": "estimate-chunk-512x64k", "op": "estimate", "lens": "512x1", "ctx": "fixed:65003", "hq": 32,
         "hkv": 8, "page": 64, "type": "bf16", "topk": 100},
        # one sequence's decoding step over its selected pages: latency
        {"name": "sparse-decode-1x128k", "op": "sparse", "lens": "1x1", "ctx": "fixed:131001", "hq": 32, "hkv": 8,
         "page": 64, "type": "bf16", "topk": 100},
        # a serving batch's decoding step over selected pages
        {"name": "sparse-decode-16x128k", "op": "sparse", "lens": "1x16", "ctx": "uniform:100000:131071", "hq": 32,
         "hkv": 8, "page": 64, "type": "bf16", "topk": 100},
        # a chunk, each token over its own pages
        {"name": "sparse-chunk-320-fp16", "op": "sparse", "lens": "313x1", "ctx": "fixed:40009", "hq": 16, "hkv": 2,
         "page": 32, "type": "fp16", "topk": 64},
    ]


_HEADS = [(32, 8), (24, 8), (16, 2), (12, 4), (8, 8), (8, 1), (28, 4), (40, 8)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "estimate", "sparse"])
    hq, hkv = rng.choice(_HEADS)
    c = {"op": op, "hq": hq, "hkv": hkv, "page": rng.choice([16, 32, 64, 128]), "type": rng.choice(["bf16", "fp16"])}
    kind = rng.choice(["decode", "chunk", "ragged"])
    if op == "append":
        c["rot"] = rng.choice([32, 64, 96, 128])
        c["interleaved"] = rng.random() < 0.5
        if kind == "decode":
            c["lens"], c["ctx"] = f"1x{_log(rng, 1, 200)}", f"uniform:0:{_log(rng, 16, 4000)}"
        elif kind == "chunk":
            c["lens"], c["ctx"] = f"{_log(rng, 2, 8000)}x1", f"fixed:{_log(rng, 1, 24000)}"
        else:
            c["lens"], c["ctx"] = f"ragged:{_log(rng, 2, 40)}:1:{_log(rng, 2, 600)}", f"uniform:0:{_log(rng, 16, 3000)}"
        return c
    if op == "attend":
        if kind == "decode":
            n = _log(rng, 1, 64)
            hi = _log(rng, 64, min(131072, 2000000 // n))
            c["lens"], c["ctx"] = f"1x{n}", f"uniform:{hi // 20}:{hi}"
        elif kind == "chunk":
            c["lens"], c["ctx"] = f"{_log(rng, 2, 1800)}x1", f"fixed:{_log(rng, 1, 60000)}"
        else:
            c["lens"] = f"ragged:{_log(rng, 2, 30)}:1:{_log(rng, 2, 600)}"
            c["ctx"] = f"uniform:0:{_log(rng, 64, 12000)}"
        return c
    # a context of 64 pages at least, of which the lists take a quarter at most
    page = c["page"]
    top = 131072 if page >= 64 else 1024 * page
    if kind == "decode":
        n = _log(rng, 1, 16)
        hi = _log(rng, 64 * page, top)
        c["lens"], c["ctx"] = f"1x{n}", f"uniform:{hi // 2}:{hi}"
    elif kind == "chunk":
        hi = _log(rng, 64 * page, min(top, 60000))
        c["lens"], c["ctx"] = f"{_log(rng, 2, 300)}x1", f"fixed:{hi}"
    else:
        hi = _log(rng, 64 * page, min(top, 30000))
        c["lens"], c["ctx"] = f"ragged:{_log(rng, 2, 12)}:1:{_log(rng, 2, 40)}", f"uniform:{hi // 8}:{hi}"
    c["topk"] = _log(rng, 4, min(128, hi // page // 4))
    return c


def _ints(seed, n, lo, hi):
    """n reproducible integers of [lo, hi]."""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(lo, hi + 1, (n,), generator=g).tolist()


def _shape(case):
    """New tokens and lengths (after the new tokens) of each sequence: part of the case, not of the seed."""
    t = case["lens"]
    if t.startswith("ragged:"):
        n, lo, hi = (int(x) for x in t.split(":")[1:])
        lens = _ints(n * 7919 + hi, n, lo, hi)
        lens = [1 if i % 3 == 1 else x for i, x in enumerate(lens)]  # a third of the sequences decode
    else:
        x, n = (int(v) for v in t.split("x"))
        lens = [x] * n
    c = case["ctx"].split(":")
    if c[0] == "fixed":
        ctx = [int(c[1])] * len(lens)
    else:
        ctx = _ints(len(lens) * 104729 + int(c[2]), len(lens), int(c[1]), int(c[2]))
    return lens, [a + b for a, b in zip(lens, ctx)]


# ------------------------------------------------------------------ inputs
def _rope_table(n, rot, device):
    inv = THETA ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    ang = torch.arange(n, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed * 1000003 + 17)
    dt = _TYPES[case["type"]]
    hq, hkv, page = case["hq"], case["hkv"], case["page"]
    lens, kv = _shape(case)
    total, n_seqs = sum(lens), len(lens)
    width = max(-(-x // page) for x in kv) + 1
    used = [-(-x // page) for x in kv]
    n_pages = sum(used) + 3
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    tables = torch.full((n_seqs, width), -1, dtype=torch.int32, device=dev)
    at = 0
    for s, n in enumerate(used):
        tables[s, :n] = perm[at:at + n]
        at += n
    cu = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(dev)
    st = {"case": case, "tables": tables, "cu": cu, "kv_lens": torch.tensor(kv, dtype=torch.int32, device=dev),
          "lens": lens, "kv": kv, "max_q": max(lens), "page": page, "hq": hq, "hkv": hkv}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=dt)

    # one direction per kv-head that some keys carry and every query asks for: heavy keys
    u = torch.randn(hkv, D, generator=g, device=dev)
    u = u / u.norm(dim=1, keepdim=True)
    if case["op"] == "append":
        # the projection's output: queries, keys and values of a token side by side
        x = normal(total, hq + 2 * hkv, D)
        st["q"], st["k"], st["v"] = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        st["rope"] = _rope_table(max(kv), case["rot"], dev)
        st["q_out"] = torch.empty(total, hq, D, dtype=dt, device=dev)
        st["k_cache"], st["v_cache"] = normal(n_pages, hkv, page, D), normal(n_pages, hkv, page, D)
        st["k_bounds"] = torch.stack(st["k_cache"].aminmax(dim=2), 2)
    else:
        q = torch.randn(total, hq, D, generator=g, device=dev) + 1.5 * u.repeat_interleave(hq // hkv, 0)
        st["q"] = q.to(dt)
        if case["op"] == "estimate":
            lo = -1.5 - torch.rand(n_pages, hkv, D, generator=g, device=dev) * 1.5
            hi = 1.5 + torch.rand(n_pages, hkv, D, generator=g, device=dev) * 1.5
            heavy = torch.rand(n_pages, hkv, 1, generator=g, device=dev) < 0.05
            shift = torch.where(heavy, 4.0, 0.0) * u
            st["k_bounds"] = torch.stack([lo + shift.clamp(max=0), hi + shift.clamp(min=0)], 2).to(dt)
        else:
            st["k_cache"], st["v_cache"] = normal(n_pages, hkv, page, D), normal(n_pages, hkv, page, D)
            n_heavy = max(1, n_pages * page // 200)
            at = torch.randint(0, n_pages * page, (n_heavy,), generator=g, device=dev)
            st["k_cache"][at // page, :, at % page] += (4 * u).to(dt)
        if case["op"] == "sparse":
            st["blk_idx"], st["blk_cnt"] = _some_pages(case, st, g)
    if own:
        from dynamic_sparse_attention_est_b200 import minf

        op = {"append": minf.OP_PAGED_APPEND, "attend": minf.OP_PAGED_ATTENTION,
              "estimate": minf.OP_PAGED_BLOCK_ESTIMATE, "sparse": minf.OP_PAGED_BLOCK_ATTENTION}[case["op"]]
        need = minf.paged_workspace_bytes(op, hq, hkv, total, n_seqs, max(lens), width, case.get("topk", 0))
        st["ws"] = minf.workspace(need, dev)
    return st


def _some_pages(case, st, g):
    """Selected pages as an estimate leaves them: the query's own page, and earlier ones that
    neighbouring queries of a sequence mostly share; ascending, -1 behind the last."""
    dev, topk, page, hkv = st["q"].device, case["topk"], st["page"], st["hkv"]
    idx, cnt = [], []
    for n, kv in zip(st["lens"], st["kv"]):
        own_page = torch.arange(kv - n, kv, device=dev) // page
        width = (kv - 1) // page + 1
        base = torch.rand(1, hkv, width, generator=g, device=dev)
        sc = base + 0.2 * torch.rand(n, hkv, width, generator=g, device=dev)
        j = torch.arange(width, device=dev)
        sc = torch.where(j == own_page[:, None, None], 9.0, sc)
        sc = torch.where(j > own_page[:, None, None], -1.0, sc)
        k = min(topk, width)
        val, sel = sc.topk(k, dim=-1)
        sel = torch.where(val >= 0, sel, width + 1).sort(-1).values
        c = (sel <= width).sum(-1)
        sel = torch.where(sel <= width, sel, -1)
        idx.append(torch.nn.functional.pad(sel, (0, topk - k), value=-1))
        cnt.append(c)
    return torch.cat(idx).to(torch.int32).contiguous(), torch.cat(cnt).to(torch.int32).contiguous()


# ------------------------------------------------------------------ plain forms
def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_append(st):
    from dynamic_sparse_attention_est_b200 import minf

    minf.minf_paged_append(st["k"], st["v"], st["k_cache"], st["v_cache"], st["tables"], st["cu"], st["kv_lens"],
                           st["max_q"], rope=st["rope"], interleaved=st["case"]["interleaved"], q=st["q"],
                           q_out=st["q_out"], k_bounds=st["k_bounds"], ws=st["ws"])
    return st["q_out"], st["k_cache"], st["v_cache"], st["k_bounds"]


def _own_attend(st):
    from dynamic_sparse_attention_est_b200 import minf

    return minf.minf_paged_attention(st["q"], st["k_cache"], st["v_cache"], st["tables"], st["cu"], st["kv_lens"],
                                     st["max_q"], scale=SCALE, ws=st["ws"])


def _own_estimate(st):
    from dynamic_sparse_attention_est_b200 import minf

    return minf.minf_paged_block_estimate(st["q"], st["k_bounds"], st["tables"], st["cu"], st["kv_lens"],
                                          st["max_q"], page_size=st["page"], topk=st["case"]["topk"], ws=st["ws"])


def _own_sparse(st):
    from dynamic_sparse_attention_est_b200 import minf

    return minf.minf_paged_block_attention(st["q"], st["k_cache"], st["v_cache"], st["tables"], st["cu"],
                                           st["kv_lens"], st["max_q"], st["blk_idx"], st["blk_cnt"], scale=SCALE,
                                           ws=st["ws"])


def _rotate(x, table, rot, interleaved):
    """x [tokens][heads][d] in fp32; table [tokens][rot]: cosines, sines."""
    c, s = table[:, None, :rot // 2], table[:, None, rot // 2:]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return y


def _positions(st):
    return torch.cat([torch.arange(kv - n, kv, device=st["q"].device) for n, kv in zip(st["lens"], st["kv"])])


def _plain_append(st):
    case, page = st["case"], st["page"]
    pos = _positions(st)
    tab = st["rope"][pos]
    st["q_out"].copy_(_rotate(st["q"].float(), tab, case["rot"], case["interleaved"]))
    k = _rotate(st["k"].float(), tab, case["rot"], case["interleaved"]).to(st["k"].dtype)
    seq = torch.repeat_interleave(torch.arange(len(st["lens"]), device=pos.device),
                                  torch.tensor(st["lens"], device=pos.device))
    where = st["tables"][seq, pos // page].long()
    st["k_cache"][where, :, pos % page] = k
    st["v_cache"][where, :, pos % page] = st["v"]
    for s, (n, kv) in enumerate(zip(st["lens"], st["kv"])):
        first, last = (kv - n) // page, (kv - 1) // page
        pg = st["tables"][s, first:last + 1].long()
        keys = st["k_cache"][pg]  # [pages][hkv][P][d]
        slot = torch.arange(first * page, (last + 1) * page, device=pos.device).view(-1, 1, page, 1)
        new = (slot >= kv - n) & (slot < kv)
        lo = torch.where(new, keys, torch.inf).amin(2)
        hi = torch.where(new, keys, -torch.inf).amax(2)
        if (kv - n) % page:  # the first page held keys before: its bounds cover them
            old = st["k_bounds"][pg[0]]
            lo[0], hi[0] = torch.minimum(lo[0], old[:, 0]), torch.maximum(hi[0], old[:, 1])
        st["k_bounds"][pg] = torch.stack([lo, hi], 2)
    return st["q_out"], st["k_cache"], st["v_cache"], st["k_bounds"]


def _plain_attend(st):
    q, hq, hkv, page = st["q"], st["hq"], st["hkv"], st["page"]
    grp = hq // hkv
    out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    row = 0
    for s, (n, kv) in enumerate(zip(st["lens"], st["kv"])):
        pg = st["tables"][s, :-(-kv // page)].long()
        pos = torch.arange(kv - n, kv, device=q.device)
        hide = torch.arange(kv, device=q.device) > pos[:, None]
        for h in range(hkv):
            k = st["k_cache"][pg, h].reshape(-1, D)[:kv].float()
            v = st["v_cache"][pg, h].reshape(-1, D)[:kv].float()
            for h2 in range(h * grp, (h + 1) * grp):
                x = (q[row:row + n, h2].float() @ k.T) * SCALE
                x.masked_fill_(hide, -torch.inf)
                top = x.amax(1, keepdim=True)
                x.sub_(top).exp_()
                tot = x.sum(1, keepdim=True)
                out[row:row + n, h2] = ((x @ v) / tot).to(out.dtype)
                lse[row:row + n, h2] = (top + tot.log())[:, 0]
        row += n
    return out, lse


def _plain_estimate(st):
    # In 64 bits throughout: scores next to the last selected one decide which page is taken.
    q, hq, hkv, page, topk = st["q"], st["hq"], st["hkv"], st["page"], st["case"]["topk"]
    idx = torch.full((q.shape[0], hkv, topk), -1, dtype=torch.int32, device=q.device)
    cnt = torch.empty(q.shape[0], hkv, dtype=torch.int32, device=q.device)
    row = 0
    for s, (n, kv) in enumerate(zip(st["lens"], st["kv"])):
        own_page = torch.arange(kv - n, kv, device=q.device) // page
        width = (kv - 1) // page + 1
        pg = st["tables"][s, :width].long()
        x = q[row:row + n].double().view(n, hkv, hq // hkv, D)
        up, down = x.clamp(min=0).sum(2), x.clamp(max=0).sum(2)  # [n][hkv][d]
        b = st["k_bounds"][pg].double()  # [width][hkv][2][d]
        j = torch.arange(width, device=q.device)
        for h in range(hkv):
            sc = up[:, h] @ b[:, h, 1].T + down[:, h] @ b[:, h, 0].T
            sc = torch.where(j == own_page[:, None], torch.inf, sc)
            sc = torch.where(j > own_page[:, None], -torch.inf, sc)
            order = sc.sort(dim=1, descending=True, stable=True).indices[:, :topk]
            take = torch.clamp(own_page + 1, max=topk)
            kept = torch.arange(order.shape[1], device=q.device) < take[:, None]
            sel = torch.where(kept, order, width).sort(1).values
            idx[row:row + n, h, :sel.shape[1]] = torch.where(sel < width, sel, -1).to(torch.int32)
            cnt[row:row + n, h] = take.to(torch.int32)
        row += n
    return idx, cnt


def _plain_sparse(st):
    q, hq, hkv, page = st["q"], st["hq"], st["hkv"], st["page"]
    grp, topk = hq // hkv, st["case"]["topk"]
    out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    seq = torch.repeat_interleave(torch.arange(len(st["lens"]), device=q.device),
                                  torch.tensor(st["lens"], device=q.device))
    pos = _positions(st)
    heads = torch.arange(hkv, device=q.device)
    slot = torch.arange(page, device=q.device)
    step = max(1, (1 << 28) // (hkv * topk * page * D))
    for a in range(0, q.shape[0], step):
        b = min(a + step, q.shape[0])
        sel = st["blk_idx"][a:b].long()  # [t][hkv][topk]
        live = torch.arange(topk, device=q.device) < st["blk_cnt"][a:b, :, None]
        pg = st["tables"][seq[a:b, None, None], sel.clamp(min=0)].long().clamp(min=0)
        k = st["k_cache"][pg, heads[:, None]].float().flatten(2, 3)  # [t][hkv][topk * P][d]
        v = st["v_cache"][pg, heads[:, None]].float().flatten(2, 3)
        see = live[..., None] & (sel[..., None] * page + slot <= pos[a:b, None, None, None])
        x = (q[a:b].float().view(b - a, hkv, grp, D) @ k.transpose(2, 3)) * SCALE
        x.masked_fill_(~see.flatten(2)[:, :, None], -torch.inf)
        top = x.amax(-1, keepdim=True)
        x = (x - top).exp()
        tot = x.sum(-1, keepdim=True)
        out[a:b] = ((x @ v) / tot).to(out.dtype).view(b - a, hq, D)
        lse[a:b] = (top + tot.log()).view(b - a, hq)
    return out, lse


_OWN = {"append": _own_append, "attend": _own_attend, "estimate": _own_estimate, "sparse": _own_sparse}
_PLAIN = {"append": _plain_append, "attend": _plain_attend, "estimate": _plain_estimate, "sparse": _plain_sparse}


# ------------------------------------------------------------------ exact forms
def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "estimate": _exact_estimate,
            "sparse": _exact_sparse}[case["op"]](st)


def _exact_append(st):
    """The rotation as a complex product by cos + i sin of the position's row."""
    case, rot, page = st["case"], st["case"]["rot"], st["page"]

    def turned(x):
        x = x.double()
        t = st["rope"].double()[_positions(st)]
        w = torch.complex(t[:, :rot // 2], t[:, rot // 2:])[:, None]
        lead = x[..., :rot]
        pairs = lead.unflatten(-1, (rot // 2, 2)) if case["interleaved"] else \
            lead.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * w)
        z = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return torch.cat([z, x[..., rot:]], -1)

    q, k, v = turned(st["q"]), turned(st["k"]), st["v"].double()
    kc, vc, kb = st["k_cache"].double(), st["v_cache"].double(), st["k_bounds"].double()
    tables = st["tables"].tolist()
    row = 0
    for s, (n, kv) in enumerate(zip(st["lens"], st["kv"])):
        p = kv - n
        while p < kv:  # page by page
            e = min(kv, (p // page + 1) * page)
            pg, o = tables[s][p // page], p % page
            new_k = k[row + p - (kv - n):row + e - (kv - n)].transpose(0, 1)  # [hkv][tokens][d]
            kc[pg, :, o:o + e - p] = new_k
            vc[pg, :, o:o + e - p] = v[row + p - (kv - n):row + e - (kv - n)].transpose(0, 1)
            lo, hi = new_k.amin(1), new_k.amax(1)
            if o:
                lo, hi = torch.minimum(lo, kb[pg, :, 0]), torch.maximum(hi, kb[pg, :, 1])
            kb[pg, :, 0], kb[pg, :, 1] = lo, hi
            p = e
        row += n
    return q, kc, vc, kb


def _exact_attend(st):
    """Rows of the stored tokens fetched one position at a time, softmax by log-sum-exp."""
    q, hq, hkv, page = st["q"], st["hq"], st["hkv"], st["page"]
    grp, dev = hq // hkv, q.device
    out = torch.empty(q.shape, dtype=torch.float64, device=dev)
    lse = torch.empty(q.shape[:2], dtype=torch.float64, device=dev)
    row = 0
    for s, (n, kv) in enumerate(zip(st["lens"], st["kv"])):
        at = torch.arange(kv, device=dev)
        line = st["tables"][s].long()[at // page]
        for h in range(hkv):
            k, v = st["k_cache"][line, h, at % page].double(), st["v_cache"][line, h, at % page].double()
            step = max(1, (1 << 28) // (kv * grp))
            for a in range(0, n, step):
                b = min(n, a + step)
                x = torch.einsum("tgd,kd->tgk", q[row + a:row + b, h * grp:(h + 1) * grp].double(), k) / math.sqrt(D)
                x[(at > kv - n + torch.arange(a, b, device=dev)[:, None])[:, None].expand_as(x)] = -torch.inf
                z = torch.logsumexp(x, -1)
                out[row + a:row + b, h * grp:(h + 1) * grp] = torch.einsum("tgk,kd->tgd", (x - z[..., None]).exp(), v)
                lse[row + a:row + b, h * grp:(h + 1) * grp] = z
        row += n
    return out, lse


def _exact_estimate(st):
    """The bound of a page head by head: sum over channels of max(q min, q max)."""
    q, hq, hkv, page, topk = st["q"], st["hq"], st["hkv"], st["page"], st["case"]["topk"]
    grp, dev = hq // hkv, q.device
    idx = torch.full((q.shape[0], hkv, topk), -1, dtype=torch.int32, device=dev)
    cnt = torch.zeros(q.shape[0], hkv, dtype=torch.int32, device=dev)
    row = 0
    for s, (n, kv) in enumerate(zip(st["lens"], st["kv"])):
        b = st["k_bounds"][st["tables"][s, :(kv - 1) // page + 1].long()].double()
        for t in range(n):
            mine = (kv - n + t) // page
            sc = torch.zeros(hkv, mine, dtype=torch.float64, device=dev)
            for g in range(grp):
                x = q[row + t, g::grp].double()  # q-head g of every kv-head
                sc += torch.maximum(x * b[:mine, :, 0], x * b[:mine, :, 1]).sum(-1).T
            k = min(topk - 1, mine)
            best = torch.argsort(-sc, dim=1, stable=True)[:, :k]
            idx[row + t, :, :k] = best.sort(1).values.to(torch.int32)
            idx[row + t, :, k] = mine
            cnt[row + t] = k + 1
        row += n
    return idx, cnt


def _exact_sparse(st):
    """Token by token: the keys of its pages up to its own position, in one list per kv-head."""
    q, hq, hkv, page = st["q"], st["hq"], st["hkv"], st["page"]
    grp, dev = hq // hkv, q.device
    out = torch.empty(q.shape, dtype=torch.float64, device=dev)
    lse = torch.empty(q.shape[:2], dtype=torch.float64, device=dev)
    row = 0
    for s, (n, kv) in enumerate(zip(st["lens"], st["kv"])):
        for t in range(n):
            for h in range(hkv):
                sel = st["blk_idx"][row + t, h][:int(st["blk_cnt"][row + t, h])].long()
                at = (sel[:, None] * page + torch.arange(page, device=dev)).flatten()
                at = at[at <= kv - n + t]
                line = st["tables"][s].long()[at // page]
                k, v = st["k_cache"][line, h, at % page].double(), st["v_cache"][line, h, at % page].double()
                x = (q[row + t, h * grp:(h + 1) * grp].double() @ k.T) / math.sqrt(D)
                z = torch.logsumexp(x, -1)
                out[row + t, h * grp:(h + 1) * grp] = (x - z[:, None]).exp() @ v
                lse[row + t, h * grp:(h + 1) * grp] = z
        row += n
    return out, lse


# ------------------------------------------------------------------ work
def work(case):
    lens, kv = _shape(case)
    hq, hkv, page = case["hq"], case["hkv"], case["page"]
    total = sum(lens)
    pages = sum(-(-x // page) for x in kv)
    meta = 4 * (pages + 2 * len(lens))
    if case["op"] == "append":
        touched = sum((x - 1) // page - (x - n) // page + 1 for n, x in zip(lens, kv))
        old = sum(1 for n, x in zip(lens, kv) if (x - n) % page)
        rows = 2 * 2 * total * (hq + 2 * hkv) * D  # read and written, 2 bytes each
        bounds = 2 * (touched + old) * hkv * 2 * D
        return {"bytes": rows + bounds + 4 * total * case["rot"] + meta,
                "flops": 3 * total * (hq + hkv) * case["rot"] + 2 * total * hkv * D}
    if case["op"] == "attend":
        pairs = sum(n * (x - n) + n * (n + 1) // 2 for n, x in zip(lens, kv))
        return {"bytes": 2 * total * hq * D * 2 + 4 * total * hq + 2 * 2 * sum(kv) * hkv * D + meta,
                "flops": 4 * D * hq * pairs}
    if case["op"] == "estimate":
        cand = sum((x - n + t) // page for n, x in zip(lens, kv) for t in range(n))
        return {"bytes": 2 * total * hq * D + 2 * pages * hkv * 2 * D + 4 * total * hkv * (case["topk"] + 1) + meta,
                "flops": 2 * 2 * D * hkv * cand + total * hq * D * 2}
    topk = case["topk"]
    keys = reads = 0
    for n, x in zip(lens, kv):
        mine = 0
        for t in range(n):
            p = x - n + t
            mine += (min(topk, p // page + 1) - 1) * page + p % page + 1
        keys += mine
        reads += min(mine, x)
    return {"bytes": 2 * total * hq * D * 2 + 4 * total * hq + 2 * 2 * reads * hkv * D
            + 4 * total * hkv * (topk + 1) + meta, "flops": 4 * D * hq * keys}
