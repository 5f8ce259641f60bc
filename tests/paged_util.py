"""64-bit results of the query/key transform and the paged-cache operators, and
the pools the tests run them on.

Tolerances (u = 2^-24, half a step of fp32; half a step of the output type is
finfo.eps / 2 relative):
* transform: fp32 arithmetic, one rounding at the end.  A norm's sum of n <= 2048
  squares runs in chains of at most 64 terms and a tree of 5, and the reciprocal
  root is off by 2 ulp, so r is off by at most (64 + 5 + 2) / 2 + 4 u; with the
  weight, the rotation's two products and their sum 48 u of |a cos| + |b sin|.
* its gradient: the mean of g w x^ adds a chain of 64 + 5 terms of 4 roundings
  each: 160 u of r (|g w| + |x^| mean|g w x^|); d_weight: 48 u and one u per row of
  a lane's chain (at most 16 in these tests), 8 warps, 4 rows a warp: 80 u of
  sum |g x^|.
* attention: a score z = scale * q.k is off by ez = (dk + 8) u scale sum|q k|,
  its probability by 2 ez relative (its own and the sum's); bf16 probabilities
  and outputs add half a step each, exp2/log2 and the joining of parts 2^-18.
"""
import numpy as np
import torch

U = 2.0 ** -24
NOT_SET = 77.0  # outputs before a call; rows a call leaves alone keep it


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ----------------------------------------------------------------------------- transform
def _pairs(ra):
    b, d, il = ra["rope_begin"], ra["rope_dim"], ra["interleaved"]
    c = torch.arange(d)
    return (b + c[0::2], b + c[1::2]) if il else (b + c[:d // 2], b + c[d // 2:])


def row_spec(norm_dim=0, weight=None, eps=1e-6, rope_begin=0, rope_dim=0, cos_sin=None, interleaved=True):
    return dict(norm_dim=norm_dim, weight=weight, eps=eps, rope_begin=rope_begin, rope_dim=rope_dim, cos_sin=cos_sin,
                interleaved=interleaved)


def transform(x, pos, ra):
    """(y, magnitude) in 64 bits of x [T, H, D] at positions pos [T]."""
    y = x.double().clone()
    n = ra["norm_dim"]
    if n:
        r = (y[..., :n].square().mean(-1, keepdim=True) + ra["eps"]).rsqrt()
        y[..., :n] = y[..., :n] * r * (ra["weight"].double() if ra["weight"] is not None else 1.0)
    mag = y.abs()
    d = ra["rope_dim"]
    if d:
        i, j = (t.to(x.device) for t in _pairs(ra))
        cs = ra["cos_sin"][pos].double()[:, None]
        c, s = cs[..., :d // 2], cs[..., d // 2:]
        a, b, ma, mb = y[..., i].clone(), y[..., j].clone(), mag[..., i].clone(), mag[..., j].clone()
        y[..., i], y[..., j] = a * c - b * s, b * c + a * s
        mag[..., i], mag[..., j] = ma * c.abs() + mb * s.abs(), mb * c.abs() + ma * s.abs()
    return y, mag


def transform_bwd(x, dy, pos, ra):
    """dx, dw and their magnitudes, from the formula in 64 bits."""
    def back(v, magnitude):  # the transposed rotation, or its terms' magnitudes
        v = v.clone()
        d = ra["rope_dim"]
        if d:
            i, j = (t.to(x.device) for t in _pairs(ra))
            cs = ra["cos_sin"][pos].double()[:, None]
            c, s = cs[..., :d // 2], cs[..., d // 2:]
            a, b = v[..., i].clone(), v[..., j].clone()
            if magnitude:
                v[..., i], v[..., j] = a * c.abs() + b * s.abs(), b * c.abs() + a * s.abs()
            else:
                v[..., i], v[..., j] = a * c + b * s, b * c - a * s
        return v

    g, mg = back(dy.double(), False), back(dy.double().abs(), True)
    n = ra["norm_dim"]
    dx, mag = g.clone(), mg.clone()
    if not n:
        return dx, mag, None, None
    w = ra["weight"].double() if ra["weight"] is not None else torch.ones(n, dtype=torch.float64, device=x.device)
    xn = x.double()[..., :n]
    r = (xn.square().mean(-1, keepdim=True) + ra["eps"]).rsqrt()
    xh = xn * r
    gn, mgn = g[..., :n], mg[..., :n]
    dx[..., :n] = r * (gn * w - xh * (gn * w * xh).mean(-1, keepdim=True))
    mag[..., :n] = r * (mgn * w.abs() + xh.abs() * (mgn * w.abs() * xh.abs()).mean(-1, keepdim=True))
    return dx, mag, (gn * xh).sum((0, 1)), (mgn * xh.abs()).sum((0, 1))


def e4m3_rows(k):
    """(codes as values, scale) of 64-bit rows [T, 128]: scale = fp32(amax / 448),
    values nearest to k / scale, ties to the even code."""
    sc = (k.abs().amax(1) / 448.0).float()
    sc = torch.where(sc > 0, sc, torch.ones_like(sc))
    grid = torch.arange(0, 127, dtype=torch.uint8, device=k.device).view(torch.float8_e4m3fn).double()
    mid = (grid[1:] + grid[:-1]) / 2
    v = (k / sc.double()[:, None]).abs()
    at = torch.bucketize(v, mid)
    on = (at < 126) & (v == mid[at.clamp(max=125)])
    at = at + (on & (at % 2 == 1)).long()
    return grid[at] * torch.where(k < 0, -1.0, 1.0), sc


# ----------------------------------------------------------------------------- pools
class Cache:
    """Lengths [(queries, keys)], a shuffled page table and pools whose unused
    rows are poisoned (NaN; every byte 0xFF for codes)."""

    def __init__(self, lens, page, seed=0, spare=3, extra_cols=0, table_pad=2):
        from sparse_attention_11_b200 import dsa

        self.dsa, self.lens, self.page = dsa, lens, page
        self.rng = np.random.default_rng(seed)
        cq = np.concatenate([[0], np.cumsum([q for q, _ in lens])])
        ck = np.concatenate([[0], np.cumsum([k for _, k in lens])])
        self.seqs = dsa.Seqs(cq, ck)
        self.cq, self.T = cq, int(cq[-1])
        per = [-(-k // page) for _, k in lens]
        self.pages = sum(per) + spare
        perm = self.rng.permutation(self.pages).astype(np.int32)
        table = np.full((len(lens), max(per) + table_pad), -1, np.int32)
        at = 0
        for b, n in enumerate(per):
            table[b, :n] = perm[at:at + n]
            at += n
        self.table = torch.from_numpy(table).cuda()
        self.extra = extra_cols
        self.b = np.concatenate([np.full(q, b) for b, (q, _) in enumerate(lens)]) if self.T else np.zeros(0, int)
        self.pos = np.concatenate([np.arange(k - q, k) for q, k in lens]) if self.T else np.zeros(0, int)
        self.tpos = torch.from_numpy(self.pos.astype(np.int64)).cuda()

    def rows(self, b):
        """(page, slot) index tensors of sequence b's positions."""
        j = torch.arange(self.lens[b][1], device="cuda")
        return self.table[b].long()[j // self.page], j % self.page

    def pool(self, cols, dtype, spread=1.0):
        """[pages, page, cols + extra] viewed to cols; rows of no position NaN."""
        p = torch.full((self.pages, self.page, cols + self.extra), float("nan"), dtype=dtype, device="cuda")[..., :cols]
        for b, (_, k) in enumerate(self.lens):
            if k:
                pg, sl = self.rows(b)
                p[pg, sl] = torch.from_numpy(self.rng.standard_normal((k, cols)).astype(np.float32) * spread).cuda().to(dtype)
        return p

    def key_pool(self, fp8=True):
        """Indexer keys of every position (codes and scales, or fp32)."""
        if not fp8:
            return self.pool_plain(128), None
        p = torch.full((self.pages, self.page, 128), 0xFF, dtype=torch.uint8, device="cuda")
        s = torch.full((self.pages, self.page), float("nan"), device="cuda")
        for b, (_, k) in enumerate(self.lens):
            if k:
                pg, sl = self.rows(b)
                v, sc = e4m3_rows(torch.from_numpy(self.rng.standard_normal((k, 128))).cuda())
                p[pg, sl] = v.float().to(torch.float8_e4m3fn).view(torch.uint8)
                s[pg, sl] = sc
        return p, s

    def pool_plain(self, cols):
        extra, self.extra = self.extra, 0
        try:
            return self.pool(cols, torch.float32)
        finally:
            self.extra = extra

    def randn(self, *shape, dtype=torch.float32):
        return torch.from_numpy(self.rng.standard_normal(shape).astype(np.float32)).cuda().to(dtype)


# ----------------------------------------------------------------------------- attention
def attention(c, q, kv, v, scale, sel=None):
    """out, lse and their error bounds' parts in 64 bits: out [T,H,dv], lse,
    sum p|v|, ez [T,H].  sel: int [T, k] positions or None (dense causal).  Slots
    past the sequence are skipped; a position listed twice counts twice."""
    T, H, dk = q.shape
    dv = v.shape[2]
    out = torch.zeros((T, H, dv), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    lse = torch.full((T, H), -float("inf"), dtype=torch.float64, device="cuda")
    ez = torch.zeros_like(lse)
    for t in range(T):
        b, pos = int(c.b[t]), int(c.pos[t])
        j = torch.arange(pos + 1, device="cuda") if sel is None else sel[t].long()
        j = j[(j >= 0) & (j < c.lens[b][1])]
        if pos < 0 or not len(j):
            continue
        pg = c.table[b].long()[j // c.page]
        j, pg = j[pg >= 0], pg[pg >= 0]
        if not len(j):
            continue
        K, V = kv[pg, j % c.page, :dk].double(), v[pg, j % c.page, :dv].double()
        z = q[t].double() @ K.T * scale
        p = torch.softmax(z, -1)
        out[t], mag[t], lse[t] = p @ V, p @ V.abs(), torch.logsumexp(z, -1)
        ez[t] = (dk + 8) * U * scale * (q[t].double().abs() @ K.abs().T).amax(-1)
    return out, lse, mag, ez


def assert_attention(c, got, got_lse, want, dtype):
    out, lse, mag, ez = want
    extra = half_step(torch.bfloat16) if dtype == torch.bfloat16 else (max(c.lens, key=lambda x: x[1])[1] + 40) * U
    tol = (extra + 2 * ez[..., None] + 2.0 ** -18) * mag + half_step(dtype) * out.abs()
    err = (got.double() - out).abs()
    assert bool((err <= tol).all()), f"out: {float((err - tol).max())} above its bound, {float(err.max())}"
    none = torch.isinf(lse)
    assert torch.equal(torch.isneginf(got_lse), none)
    assert bool((got[none] == 0).all())
    err = (got_lse.double() - lse).abs()[~none]
    tol = (ez + 2.0 ** -16 + 4 * U * lse.abs())[~none]
    assert bool((err <= tol).all()), f"lse: {float((err - tol).max())} above its bound"
