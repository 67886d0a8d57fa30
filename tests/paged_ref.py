"""Plain 64-bit forms of the paged key/value cache operators, and error bounds for their 16-bit results."""
import math

import torch

D = 128


def u(dtype):
    """Half a step of a rounding to `dtype`, relative to the value."""
    return torch.finfo(dtype).eps / 2


class Case:
    """Sequences over a paged cache with shuffled pages; unused page slots hold NaN."""

    def __init__(self, lens, kv, hq, hkv, page, dtype, seed=0, dev="cuda", extra_rows=0, gap=0, cache_gap=False,
                 bias=0.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.kv, self.hq, self.hkv, self.page, self.dtype, self.dev = lens, kv, hq, hkv, page, dtype, dev
        self.total = sum(lens) + extra_rows
        self.max_q = max(max(lens), 1)
        used = [-(-x // page) for x in kv]
        self.width = max(max(used), 1) + gap
        self.num_pages = sum(used) + 2
        perm = torch.randperm(self.num_pages, generator=g, dtype=torch.int32)
        self.tables = torch.full((len(lens), self.width), -1, dtype=torch.int32)
        at = 0
        for s, n in enumerate(used):
            self.tables[s, :n] = perm[at:at + n]
            at += n
        self.cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
        self.kv_lens = torch.tensor(kv, dtype=torch.int32)

        def rnd(*shape):
            return torch.randn(*shape, generator=g)

        self.q = (rnd(self.total, hq, D) + bias).to(dtype)
        self.k_new, self.v_new = (rnd(self.total, hkv, D) + bias).to(dtype), rnd(self.total, hkv, D).to(dtype)
        shape = (self.num_pages, hkv, page, D)
        kc, vc = torch.full(shape, math.nan), torch.full(shape, math.nan)
        for s, x in enumerate(kv):
            for b in range(used[s]):
                n = min(page, x - b * page)
                kc[self.tables[s, b], :, :n] = rnd(hkv, n, D) + bias
                vc[self.tables[s, b], :, :n] = rnd(hkv, n, D)
        if cache_gap:  # keys and values of a page side by side: page strides of two pages
            both = torch.stack([kc, vc], 1).to(dtype).to(dev)
            self.k_cache, self.v_cache = both[:, 0], both[:, 1]
        else:
            self.k_cache, self.v_cache = kc.to(dtype).to(dev), vc.to(dtype).to(dev)
        for name in ("tables", "cu", "kv_lens", "q", "k_new", "v_new"):
            setattr(self, name, getattr(self, name).to(dev))

    def meta(self):
        return self.tables, self.cu, self.kv_lens, self.max_q

    def rows(self):
        """(sequence, token row, position) of every token."""
        r = 0
        for s, (n, x) in enumerate(zip(self.lens, self.kv)):
            for i in range(n):
                yield s, r, x - n + i
                r += 1

    def stored(self, s, h, n):
        """The first n keys and values of sequence s, kv-head h, in 64 bits."""
        pg = self.tables[s, :-(-n // self.page)].long()
        k = self.k_cache[pg, h].reshape(-1, D)[:n].double()
        v = self.v_cache[pg, h].reshape(-1, D)[:n].double()
        return k, v


def attention(c, scale, pick=None):
    """Exact out and lse, and the tolerances of a 16-bit kernel's.

    The kernel's result differs by the rounding of the output (u |o|), of the
    weights before the product with V (u each: at most u sum p |v|), and by the
    error d of a logit: 128 products summed in fp32, eight tensor-core steps
    within 2^-22 of their magnitudes each (2^-19 sum |q| |k|), the scaling and
    the exponential (2^-20 together with |logit| 2^-23); a logit error d moves
    the result by at most 2 d sum p |v|.  fp16 weights end at 2^-25 of a scale
    that lies 2^6 below the row's largest at the least: n 2^-31 max |v|."""
    out = torch.zeros(c.total, c.hq, D, dtype=torch.float64, device=c.dev)
    lse = torch.full((c.total, c.hq), -math.inf, dtype=torch.float64, device=c.dev)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    grp = c.hq // c.hkv
    for s, r, pos in c.rows():
        if pos < 0:
            continue
        for h in range(c.hkv):
            k, v = c.stored(s, h, pos + 1)
            if pick is not None:
                keep = pick(s, r, h, pos)
                k, v = k[keep], v[keep]
            if len(k) == 0:
                continue
            q = c.q[r, h * grp:(h + 1) * grp].double()
            x = q @ k.T * scale
            z = torch.logsumexp(x, 1)
            p = (x - z[:, None]).exp()
            out[r, h * grp:(h + 1) * grp], lse[r, h * grp:(h + 1) * grp] = p @ v, z
            mag = (q.abs() @ k.abs().T).amax(1) * scale
            d = mag * 2 ** -19 + x.abs().amax(1) * 2 ** -23 + 2 ** -20
            a = p @ v.abs()
            t = u(c.dtype) * (p @ v).abs() + (u(c.dtype) + 2 * d[:, None]) * a + 1e-7
            if c.dtype == torch.float16:
                t += len(k) * 2 ** -31 * v.abs().max() + 2 ** -25  # and the output's own smallest step
            tol_o[r, h * grp:(h + 1) * grp] = t
            tol_l[r, h * grp:(h + 1) * grp] = d + len(k) * 2 ** -24 + z.abs() * 2 ** -22 + 2 ** -20
    return out, lse, tol_o, tol_l


def check(c, got, want, rows=None):
    out, lse = got
    ref, rl, to, tl = want
    n = sum(c.lens)
    err = (out[:n].double() - ref[:n]).abs()
    bad = ~(err <= to[:n])
    assert not bad.any(), f"{int(bad.sum())} values off, worst {float((err / to[:n].clamp(min=1e-30)).max()):.2f} x tol"
    if lse is not None:
        inf = rl[:n] == -math.inf
        assert torch.equal(lse[:n] == -math.inf, inf)
        el = (lse[:n].double() - rl[:n])[~inf].abs()
        assert (el <= tl[:n][~inf]).all(), float((el / tl[:n][~inf]).max())


def bounds(c):
    """Channels' smallest and largest stored key of every page in use."""
    kb = torch.full((c.num_pages, c.hkv, 2, D), math.nan, dtype=c.dtype, device=c.dev)
    for s, x in enumerate(c.kv):
        for b in range(-(-x // c.page)):
            n = min(c.page, x - b * c.page)
            pg = int(c.tables[s, b])
            kb[pg, :, 0], kb[pg, :, 1] = c.k_cache[pg, :, :n].amin(1), c.k_cache[pg, :, :n].amax(1)
    return kb


def estimate(c, kb, topk):
    idx = torch.full((c.total, c.hkv, topk), -1, dtype=torch.int32, device=c.dev)
    cnt = torch.zeros(c.total, c.hkv, dtype=torch.int32, device=c.dev)
    grp = c.hq // c.hkv
    for s, r, pos in c.rows():
        if pos < 0:
            continue
        own = pos // c.page
        b = kb[c.tables[s, :own].long()].double()
        for h in range(c.hkv):
            x = c.q[r, h * grp:(h + 1) * grp].double()
            sc = x.clamp(min=0).sum(0) @ b[:, h, 1].T + x.clamp(max=0).sum(0) @ b[:, h, 0].T
            k = min(topk - 1, own)
            best = torch.sort(sc, descending=True, stable=True).indices[:k].sort().values
            idx[r, h, :k], idx[r, h, k] = best.to(torch.int32), own
            cnt[r, h] = k + 1
    return idx, cnt


def rotate(x, table, pos, rot, interleaved):
    """64-bit rotation of [tokens, heads, 128], and the error of an fp32 one rounded to x's type."""
    t = table[pos].double()[:, None]
    c, s = t[..., :rot // 2], t[..., rot // 2:]
    y, mag = x.double(), x.double().abs()
    if interleaved:
        i, j = slice(0, rot, 2), slice(1, rot, 2)
    else:
        i, j = slice(0, rot // 2), slice(rot // 2, rot)
    a, b = y[..., i].clone(), y[..., j].clone()
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    mag[..., i], mag[..., j] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    # two products and a sum in fp32, then half a step of the result (fp16: or of its smallest)
    return y, u(x.dtype) * y.abs() + 3 * 2 ** -24 * mag * (1 + u(x.dtype)) + 2 ** -25


def rope_table(n, rot, dev="cuda"):
    inv = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    ang = torch.arange(n, dtype=torch.float64)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float().to(dev)
