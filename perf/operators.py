"""The paged-cache operators: cases, plain forms and 64-bit results.

A serving step of the framework's sparse attention over a paged cache, and
the training step of its query/key transform:

  norm_rope      RMS norm of every head's row and the position rotation in one
                 pass (forward)
  norm_rope_bwd  its gradients
  append         the new tokens' KV rows (latent normed, rope part rotated) and
                 indexer keys (rotated, quantised to e4m3 with one scale per
                 token) into their pages
  scores         lightning-indexer scores of folded queries over the paged
                 indexer keys
  attn           MQA attention of a chunk of new tokens over the paged KV rows:
                 dense causal, or over each query's selected positions

`run` computes the plain form in elementary torch operations, or makes the
framework's calls where `own` is true.  `exact` gives the 64-bit result.
Sequences follow the framework's rule: the queries of a sequence are its last
positions, pos = seqlen_k - seqlen_q + i.
"""
import math
import random

import torch

own = False

IDX_DIM = 128
E4M3_MAX = 448.0
EPS = 1e-6


# ----------------------------------------------------------------------------- cases
def _case(c):
    """A case as plain values: a range is kept as its two ends."""
    d = dict(c)
    for k in ("lq", "lk"):
        d[k + "_lo"], d[k + "_hi"] = d.pop(k)
    return d


# The attention's own query transform: latent columns as they are, 64 rotated.
MLA_Q = dict(dim=576, norm_dim=0, rope_begin=512, rope_dim=64, interleaved=True)


def listed():
    """Sizes: 128 heads, KV rows of 512 latent + 64 rope columns, k = 2048,
    decode batches of 64 sequences with 16K to 64K tokens, 8K prefill and the
    4-head fp32 configuration are the framework's own workloads; the rest are
    generic."""
    return [_case(c) for c in (
        # one decode step's queries: 64 sequences, a single token each, far positions
        dict(name="norm_rope_decode", op="norm_rope", dtype="bf16", batch=64, lq=[1, 1], lk=[16384, 65536], heads=128,
             lens=1, **MLA_Q),
        # an 8K prefill's queries
        dict(name="norm_rope_prefill", op="norm_rope", dtype="bf16", batch=1, lq=[8192, 8192], lk=[8192, 8192],
             heads=128, lens=2, **MLA_Q),
        # training: per-head norm and rotation of 32 heads, packed ragged sequences
        dict(name="norm_rope_bwd_train", op="norm_rope_bwd", dtype="bf16", batch=7, lq=[100, 2000], lk=[0, 0], heads=32,
             dim=128, norm_dim=128, rope_begin=0, rope_dim=128, interleaved=False, lens=3),
        # training of the latent row (512 normed, 64 rotated), fp32
        dict(name="norm_rope_bwd_latent", op="norm_rope_bwd", dtype="f32", batch=5, lq=[500, 4000], lk=[0, 0], heads=1,
             dim=576, norm_dim=512, rope_begin=512, rope_dim=64, interleaved=True, lens=4),
        # one decode step's new rows into 64 caches
        dict(name="append_decode", op="append", dtype="bf16", batch=64, lq=[1, 1], lk=[16384, 65536], page=64, lens=5),
        # a prefill's new rows: ragged chunks behind ragged prefixes, pages of 48
        dict(name="append_prefill", op="append", dtype="bf16", batch=9, lq=[500, 1500], lk=[2000, 9000], page=48,
             lens=6),
        # decode selection: one folded query per sequence over its whole cache
        dict(name="scores_decode", op="scores", batch=64, lq=[1, 1], lk=[16384, 65536], page=64, lens=7),
        # chunked prefill: 1000 new tokens behind 31K
        dict(name="scores_chunk", op="scores", batch=1, lq=[1000, 1000], lk=[32000, 32000], page=64, lens=8),
        # decode attention over the 2048 selected rows of each cache
        dict(name="attn_selected_decode", op="attn", dtype="bf16", selected=2048, batch=64, lq=[1, 1],
             lk=[16384, 65536], heads=128, dk=576, dv=512, page=64, lens=9),
        # chunked prefill over the selected rows, ragged batch
        dict(name="attn_selected_chunk", op="attn", dtype="bf16", selected=2048, batch=3, lq=[200, 500],
             lk=[9000, 30000], heads=128, dk=576, dv=512, page=64, lens=10),
        # dense causal attention of new chunks behind short prefixes
        dict(name="attn_dense_chunk", op="attn", dtype="bf16", selected=0, batch=2, lq=[300, 700], lk=[3000, 5000],
             heads=128, dk=576, dv=512, page=64, lens=11),
        # the fp32 configuration: 4 heads of 64, short caches, pages of 20
        dict(name="attn_dense_f32", op="attn", dtype="f32", selected=0, batch=6, lq=[1, 9], lk=[100, 700], heads=4,
             dk=64, dv=64, page=20, lens=12),
    )]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "append", "scores", "attn", "attn"])
    lens = rng.randrange(1 << 30)
    c = dict(op=op, lens=lens)
    page = rng.choice([16, 20, 32, 48, 64, 64, 100, 128, 256])
    if op in ("norm_rope", "norm_rope_bwd"):
        kind = rng.choice(["latent_q", "head", "latent_k"])
        if kind == "latent_q":
            c.update(heads=rng.choice([16, 32, 64, 128]), **MLA_Q)
        elif kind == "latent_k":
            c.update(dim=576, norm_dim=512, rope_begin=512, rope_dim=64, interleaved=True, heads=1)
        else:
            dim = rng.choice([64, 96, 128, 192, 256])
            rope = rng.choice([dim, dim // 2])
            c.update(dim=dim, norm_dim=dim, rope_begin=rng.choice([0, dim - rope]), rope_dim=rope,
                     interleaved=rng.random() < 0.5, heads=rng.choice([1, 3, 8, 32]))
        c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
        most = 300_000_000 if op == "norm_rope" else 15_000_000  # elements
        tokens = _log(rng, 1, min(8192, most // (c["heads"] * c["dim"])))
        batch = rng.choice([1, 2, 5])
        hi = max(1, tokens // batch)
        c.update(batch=batch, lq=[max(1, hi // 2), hi], lk=[hi, rng.choice([hi, hi + 1000, 60000])])
    elif op == "append":
        batch, dtype = _log(rng, 1, 64), rng.choice(["bf16", "bf16", "f32"])
        hi = _log(rng, 1, (8192 if dtype == "bf16" else 4096) // batch)
        c.update(dtype=dtype, batch=batch, lq=[max(1, hi // 3), hi],
                 lk=[hi, _log(rng, hi + 1, 16000)], page=page)
    elif op == "scores":
        batch = _log(rng, 1, 64)
        lq = rng.choice([1, 1, _log(rng, 2, max(2, 1000 // batch))])
        lk = _log(rng, max(256, lq), min(65536, max(lq + 256, 32_000_000 // (batch * lq))))
        c.update(batch=batch, lq=[max(1, lq // 2), lq], lk=[max(lq, lk // 3), lk], page=page)
    else:
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        selected = rng.choice([0, 0, 64, 500, 1000, 2048]) if dtype == "bf16" else rng.choice([0, 64])
        c.update(dtype=dtype, selected=selected, page=page)
        if dtype == "f32":
            c.update(heads=rng.choice([1, 4, 8]), dk=rng.choice([32, 64, 128]), dv=rng.choice([32, 64, 96]))
            batch, lq, lk = rng.randint(1, 8), _log(rng, 1, 40), _log(rng, 64, 3000)
        else:
            c.update(heads=rng.choice([16, 64, 128, 128]), dk=576, dv=512)
            batch = _log(rng, 1, 32)
            lq = _log(rng, 1, max(1, 600 // batch))
            lk = _log(rng, 200, 20000 if selected else max(300, min(30000, 4_000_000 // (batch * lq))))
        c.update(batch=batch, lq=[max(1, lq // 2), lq], lk=[max(lq, lk // 2), max(lq, lk)])
    return _case(c)


def _lengths(case):
    """(queries, keys) per sequence, from the case alone."""
    r = random.Random(case["lens"])
    got = []
    for _ in range(case["batch"]):
        q = r.randint(case["lq_lo"], case["lq_hi"])
        got.append((q, max(q, r.randint(case["lk_lo"], max(case["lk_lo"], case["lk_hi"])))))
    return got


def _dt(case):
    return torch.bfloat16 if case.get("dtype", "bf16") == "bf16" else torch.float32


def _rope_table(n, dim):
    """cos | sin of pos / 10000^(2i/dim), angles in 64 bits."""
    f = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64, device="cuda") / dim)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


# ----------------------------------------------------------------------------- inputs
def prepare(case, seed):
    lens = _lengths(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    cu_q, cu_k = [0], [0]
    for q, k in lens:
        cu_q.append(cu_q[-1] + q)
        cu_k.append(cu_k[-1] + k)
    T, B = cu_q[-1], len(lens)
    mq, mk = max(q for q, _ in lens), max(k for _, k in lens)
    s = dict(case=case, T=T, B=B, max_q=mq, max_k=mk, cu_q=torch.tensor(cu_q, device="cuda"),
             cu_k=torch.tensor(cu_k, device="cuda"))
    dt = _dt(case)
    op = case["op"]

    def randn(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype)

    if op in ("norm_rope", "norm_rope_bwd"):
        shape = (T, case["heads"], case["dim"])
        s["x"] = randn(*shape, dtype=dt)
        s["weight"] = 1 + 0.2 * randn(case["norm_dim"]) if case["norm_dim"] else None
        s["cos_sin"] = _rope_table(mk, case["rope_dim"])
        if op == "norm_rope":
            s["y"] = torch.empty_like(s["x"])
        else:
            s["dy"] = randn(*shape, dtype=dt)
            s["dx"] = torch.empty_like(s["x"])
            s["dw"] = torch.empty(case["norm_dim"], device="cuda") if case["norm_dim"] else None
    else:
        # every sequence's pages at shuffled places of the pool, a few pages spare
        P = case["page"]
        per = [-(-k // P) for _, k in lens]
        pages = sum(per) + 5
        perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((B, max(per)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(per):
            table[b, :n] = perm[at:at + n]
            at += n
        s["table"] = table
        s["pages"] = pages
        if op in ("append", "scores"):
            s["idx"] = torch.randint(0, 256, (pages, P, IDX_DIM), generator=g, device="cuda", dtype=torch.uint8)
            if op == "scores":  # key codes as quantisation gives them: normal values over the row's scale
                k = randn(pages * P, IDX_DIM)
                sc = k.abs().amax(1) / E4M3_MAX
                s["idx"] = (k / sc[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(pages, P, IDX_DIM)
                s["idx_scale"] = sc.view(pages, P)
                del k
                u = randn(T, IDX_DIM)
                su = u.abs().amax(1) / E4M3_MAX
                s["u"] = (u / su[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
                s["s_row"] = su
                s["scores"] = torch.empty((T, mk), device="cuda")
            else:
                s["idx"] = (s["idx"] & 0x7F).clamp_(max=0x7E)  # finite codes
                s["idx_scale"] = torch.rand((pages, P), generator=g, device="cuda")
        if op == "append":
            s["kv"] = randn(pages, P, 576, dtype=dt)
            s["kv_new"] = randn(T, 576, dtype=dt)
            s["idx_new"] = randn(T, IDX_DIM, dtype=dt)
            s["weight"] = 1 + 0.2 * randn(512)
            s["cos_sin"] = _rope_table(mk, 64)
        if op == "attn":
            H, dk, dv = case["heads"], case["dk"], case["dv"]
            s["kv"] = randn(pages, P, dk, dtype=dt)
            s["v"] = None if dt == torch.bfloat16 else randn(pages, P, dv, dtype=dt)
            s["q"] = randn(T, H, dk, dtype=dt)
            s["scale"] = 1.0 / math.sqrt(dk)
            s["out"] = torch.empty((T, H, dv), dtype=dt, device="cuda")
            s["lse"] = torch.empty((T, H), device="cuda")
            s["sel"] = None
            if case["selected"]:
                # each query's selection: distinct earlier positions, ascending, then -1;
                # about one query in 50 has selected nothing
                _, pos = _where(s)
                r = torch.rand((T, mk), generator=g, device="cuda")
                r.masked_fill_(torch.arange(mk, device="cuda")[None] > pos[:, None], -1.0)
                n = min(case["selected"], mk)
                val, ix = r.topk(n, dim=1)
                ix = torch.where(val >= 0, ix, torch.full_like(ix, mk)).sort(1).values
                ix = torch.where(ix < mk, ix, torch.full_like(ix, -1)).to(torch.int32)
                ix[torch.rand(T, generator=g, device="cuda") < 0.02] = -1
                s["sel"] = torch.full((T, case["selected"]), -1, dtype=torch.int32, device="cuda")
                s["sel"][:, :n] = ix
    if own:
        _plan(s, cu_q, cu_k)
    return s


def _plan(s, cu_q, cu_k):
    """What a program using the framework keeps between calls: the batch's
    description, the page pool's, the argument structs and a workspace."""
    from sparse_attention_11_b200 import dsa

    c, op = s["case"], s["case"]["op"]
    s["dsa"], s["seqs"] = dsa, dsa.Seqs(cu_q, cu_k)
    n = 256
    if op in ("norm_rope", "norm_rope_bwd"):
        s["ra"] = dsa.row_args(norm_dim=c["norm_dim"], weight=s["weight"], eps=EPS, rope_begin=c["rope_begin"],
                               rope_dim=c["rope_dim"], cos_sin=s["cos_sin"], interleaved=c["interleaved"])
        if op == "norm_rope_bwd":
            n = dsa.dsa_workspace_size(dsa.DSA_OP_NORM_ROPE_BWD, s["seqs"], c["norm_dim"])
    elif op == "append":
        s["pg"] = dsa.Pages(s["table"], kv=s["kv"], idx=s["idx"], idx_scale=s["idx_scale"])
        kv_row = dsa.row_args(norm_dim=512, weight=s["weight"], eps=EPS, rope_begin=512, rope_dim=64,
                              cos_sin=s["cos_sin"])
        idx_row = dsa.row_args(rope_begin=0, rope_dim=64, cos_sin=s["cos_sin"], interleaved=False)
        s["ap"] = dsa.append_args(s["pg"], kv_new=s["kv_new"], kv_row=kv_row, idx_new=s["idx_new"], idx_row=idx_row)
    elif op == "scores":
        s["pg"] = dsa.Pages(s["table"], idx=s["idx"], idx_scale=s["idx_scale"])
    else:
        s["pg"] = dsa.Pages(s["table"], kv=s["kv"], v=s["v"])
        s["aa"] = dsa.paged_attn_args(s["pg"], s["q"], s["scale"], s["out"], s["lse"])
        n = dsa.dsa_workspace_size(dsa.DSA_OP_PAGED_ATTN, s["seqs"], c["selected"], None, s["aa"])
    s["ws"] = dsa.workspace(n)


# ----------------------------------------------------------------------------- the calls
def run(s):
    op = s["case"]["op"]
    if own:
        return _OWN[op](s)
    return _PLAIN[op](s)


def _own_norm_rope(s):
    s["dsa"].dsa_norm_rope(s["seqs"], s["ra"], s["x"], s["y"], s["ws"])
    return s["y"]


def _own_norm_rope_bwd(s):
    s["dsa"].dsa_norm_rope_bwd(s["seqs"], s["ra"], s["x"], s["dy"], s["dx"], s["dw"], s["ws"])
    return {"dx": s["dx"], "dw": s["dw"]} if s["dw"] is not None else {"dx": s["dx"]}


def _own_append(s):
    s["dsa"].dsa_cache_append(s["seqs"], s["pg"], s["ap"], s["ws"])
    return {"kv": s["kv"], "idx": s["idx"].view(torch.float8_e4m3fn), "idx_scale": s["idx_scale"]}


def _own_scores(s):
    s["dsa"].dsa_paged_scores(s["seqs"], s["pg"], s["u"], s["s_row"], 0, s["T"], s["scores"], s["ws"])
    return s["scores"]


def _own_attn(s):
    s["dsa"].dsa_paged_attn(s["seqs"], s["pg"], s["aa"], s["sel"], s["case"]["selected"], s["ws"])
    return {"out": s["out"], "lse": s["lse"]}


_OWN = dict(norm_rope=_own_norm_rope, norm_rope_bwd=_own_norm_rope_bwd, append=_own_append, scores=_own_scores,
            attn=_own_attn)


# ----------------------------------------------------------------------------- plain forms
def _where(s):
    """Sequence and position of every packed query."""
    t = torch.arange(s["T"], device="cuda")
    b = torch.searchsorted(s["cu_q"][1:].contiguous(), t, right=True)
    cq, ck = s["cu_q"], s["cu_k"]
    return b, (ck[b + 1] - ck[b]) - (cq[b + 1] - cq[b]) + (t - cq[b])


def _pair(x, interleaved):
    """The two halves of every rotated pair."""
    if interleaved:
        return x[..., 0::2], x[..., 1::2]
    h = x.shape[-1] // 2
    return x[..., :h], x[..., h:]


def _unpair(a, b, interleaved):
    return torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)


def _rotate(x, cos, sin, interleaved):
    a, b = _pair(x, interleaved)
    return _unpair(a * cos - b * sin, b * cos + a * sin, interleaved)


def _transform(x, cos_sin, weight, norm_dim, begin, rope_dim, interleaved):
    """norm, then rotation, of x [T, H, D] (32 or 64 bits); cos_sin [T, 1, rope_dim]."""
    if norm_dim:
        n = x[..., :norm_dim]
        n = n * torch.rsqrt(n.square().mean(-1, keepdim=True) + EPS) * weight
        x = torch.cat([n, x[..., norm_dim:]], -1)
    if rope_dim:
        h = rope_dim // 2
        r = _rotate(x[..., begin:begin + rope_dim], cos_sin[..., :h], cos_sin[..., h:], interleaved)
        x = torch.cat([x[..., :begin], r, x[..., begin + rope_dim:]], -1)
    return x


def _plain_norm_rope(s):
    c = s["case"]
    _, pos = _where(s)
    y = _transform(s["x"].float(), s["cos_sin"][pos][:, None], s["weight"], c["norm_dim"], c["rope_begin"],
                   c["rope_dim"], c["interleaved"])
    return y.to(s["x"].dtype)


def _plain_norm_rope_bwd(s):
    c = s["case"]
    _, pos = _where(s)
    cs = s["cos_sin"][pos][:, None]
    h, b0, n = c["rope_dim"] // 2, c["rope_begin"], c["norm_dim"]
    g = s["dy"].float()
    r = _rotate(g[..., b0:b0 + 2 * h], cs[..., :h], -cs[..., h:], c["interleaved"])  # the transposed rotation
    g = torch.cat([g[..., :b0], r, g[..., b0 + 2 * h:]], -1)
    if not n:
        return {"dx": g.to(s["x"].dtype)}
    x = s["x"].float()[..., :n]
    rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xh = x * rstd
    gn = g[..., :n]
    gw = gn * s["weight"]
    dn = rstd * (gw - xh * (gw * xh).mean(-1, keepdim=True))
    dw = (gn * xh).sum((0, 1), dtype=torch.float64).float()
    return {"dx": torch.cat([dn, g[..., n:]], -1).to(s["x"].dtype), "dw": dw}


def _e4m3(v):
    """64-bit values rounded to the nearest e4m3 value (ties to even, saturating)."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -9))).clamp(min=-6.0)
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _plain_append(s):
    b, pos = _where(s)
    P = s["case"]["page"]
    row = s["table"][b, pos // P].long() * P + pos % P
    cs = s["cos_sin"][pos][:, None]
    kv = _transform(s["kv_new"].float()[:, None], cs, s["weight"], 512, 512, 64, True)[:, 0]
    s["kv"].view(-1, 576)[row] = kv.to(s["kv"].dtype)
    # in 64 bits: a value next to a rounding border of e4m3 must fall on its side
    k = _transform(s["idx_new"].double()[:, None], cs.double(), None, 0, 0, 64, False)[:, 0]
    amax = k.abs().amax(1)
    scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax)).float()
    codes = _e4m3(k / scale.double()[:, None]).float().to(torch.float8_e4m3fn)
    s["idx"].view(-1, IDX_DIM)[row] = codes.view(torch.uint8)
    s["idx_scale"].view(-1)[row] = scale
    return {"kv": s["kv"], "idx": s["idx"].view(torch.float8_e4m3fn), "idx_scale": s["idx_scale"]}


def _padded(s):
    """Rows of every sequence's positions in the flattened pool [B, max_k], and
    the place of every packed query in a [B, max_q] grid."""
    P = s["case"]["page"]
    j = torch.arange(s["max_k"], device="cuda")
    row = s["table"].long().clamp(min=0)[:, j // P] * P + j % P
    b, pos = _where(s)
    at = b * s["max_q"] + torch.arange(s["T"], device="cuda") - s["cu_q"][b]
    return row, at, pos


def _plain_scores(s):
    row, at, pos = _padded(s)
    B, mq, mk = s["B"], s["max_q"], s["max_k"]
    k = s["idx"].view(torch.float8_e4m3fn).view(-1, IDX_DIM)[row].float()
    u = torch.zeros((B * mq, IDX_DIM), device="cuda")
    u[at] = s["u"].view(torch.float8_e4m3fn).float()
    x = torch.matmul(u.view(B, mq, IDX_DIM), k.transpose(1, 2))
    x = (x * s["idx_scale"].view(-1)[row][:, None]).view(B * mq, mk)[at] * s["s_row"][:, None]
    x = x.clamp(min=0)
    return x.masked_fill(torch.arange(mk, device="cuda")[None] > pos[:, None], -math.inf)


def _softmax_v(z, mask, v):
    """Masked softmax of z [N, R, K] times v [N, K, D], and log-sum-exp."""
    z = z.masked_fill(~mask, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - m.clamp(min=-3e38))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / l.clamp(min=1e-38)
    return o, (m + torch.log(l))[..., 0]


def _plain_attn(s):
    c = s["case"]
    H, dk, dv, T, B, mq = c["heads"], c["dk"], c["dv"], s["T"], s["B"], s["max_q"]
    kv = s["kv"].view(-1, dk)
    vv = kv[:, :dv] if s["v"] is None else s["v"].view(-1, dv)
    if c["selected"]:
        P = c["page"]
        b, _ = _where(s)
        j = s["sel"].long()
        row = s["table"][b[:, None], j.clamp(min=0) // P].long() * P + j.clamp(min=0) % P
        k = kv[row].float()
        z = torch.matmul(s["q"].float(), k.transpose(1, 2)) * s["scale"]
        o, lse = _softmax_v(z, (j >= 0)[:, None], k[..., :dv] if s["v"] is None else vv[row].float())
        return {"out": o.to(s["q"].dtype), "lse": lse}
    row, at, pos = _padded(s)
    q = torch.zeros((B * mq, H, dk), device="cuda")
    q[at] = s["q"].float()
    k = kv[row].float()
    z = torch.matmul(q.view(B, mq * H, dk), k.transpose(1, 2)) * s["scale"]
    lim = torch.full((B * mq,), -1, device="cuda")
    lim[at] = pos
    mask = torch.arange(s["max_k"], device="cuda")[None, None] <= lim.view(B, mq, 1)
    mask = mask[:, :, None].expand(B, mq, H, s["max_k"]).reshape(B, mq * H, s["max_k"])
    o, lse = _softmax_v(z, mask, k[..., :dv] if s["v"] is None else vv[row].float())
    return {"out": o.view(B * mq, H, dv)[at].to(s["q"].dtype), "lse": lse.view(B * mq, H)[at]}


_PLAIN = dict(norm_rope=_plain_norm_rope, norm_rope_bwd=_plain_norm_rope_bwd, append=_plain_append,
              scores=_plain_scores, attn=_plain_attn)


# ----------------------------------------------------------------------------- least work
def work(case):
    """Bytes: every input row read once, every output written once.  A cache
    row counts once per sequence (selected rows: once per query that selected
    them, or the whole cache where that is less)."""
    lens = _lengths(case)
    T = sum(q for q, _ in lens)
    e = 2 if case.get("dtype", "bf16") == "bf16" else 4
    op = case["op"]
    if op in ("norm_rope", "norm_rope_bwd"):
        n = T * case["heads"] * case["dim"]
        tab = T * case["rope_dim"] * 4
        if op == "norm_rope":
            return {"bytes": 2 * n * e + tab, "flops": 8 * n}
        moved = 3 if case["norm_dim"] == case["dim"] else 2 + case["norm_dim"] / case["dim"]
        return {"bytes": moved * n * e + tab, "flops": 14 * n}
    if op == "append":
        return {"bytes": T * (2 * 576 * e + IDX_DIM * e + IDX_DIM + 4 + 64 * 4), "flops": T * (576 + IDX_DIM) * 8}
    causal = sum(q * k - q * (q - 1) // 2 for q, k in lens)
    keys = sum(k for _, k in lens)
    if op == "scores":
        # what lies past a row's position is written too (-inf)
        return {"bytes": keys * (IDX_DIM + 4) + T * (IDX_DIM + 4) + T * max(k for _, k in lens) * 4,
                "flops": causal * IDX_DIM * 2}
    H, dk, dv = case["heads"], case["dk"], case["dv"]
    row = dk * e + (dv * e if e == 4 else 0)
    if case["selected"]:
        n = [sum(min(case["selected"], k - q + i + 1) for i in range(q)) for q, k in lens]
        pairs, rows = sum(n), sum(min(m, k) for m, (_, k) in zip(n, lens))
        extra = T * case["selected"] * 4
    else:
        pairs, rows, extra = causal, keys, 0
    return {"bytes": rows * row + T * H * (dk + dv) * e + T * H * 4 + extra, "flops": 2 * pairs * H * (dk + dv)}


# ----------------------------------------------------------------------------- 64-bit results
def exact(case, seed):
    """From the definitions, sequence by sequence, in 64 bits."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    lens, op = _lengths(case), case["op"]
    spans, t = [], 0
    for b, (q, k) in enumerate(lens):
        spans.append((b, t, t + q, q, k))
        t += q
    if op in ("norm_rope", "norm_rope_bwd", "append"):
        pos = torch.cat([torch.arange(k - q, k, device="cuda") for _, _, _, q, k in spans])
    if op == "norm_rope":
        w = s["weight"].double() if case["norm_dim"] else None
        # in pieces of tokens: 64-bit copies of the largest case are large
        return torch.cat([_exact_rows(s["x"][i:i + 1024].double(), s["cos_sin"][pos[i:i + 1024]].double(), w, case)
                          for i in range(0, s["T"], 1024)])
    if op == "norm_rope_bwd":
        dx, dw = [], 0
        for i in range(0, s["T"], 1024):
            a, w = _exact_rows_bwd(s["x"][i:i + 1024].double(), s["dy"][i:i + 1024].double(),
                                   s["cos_sin"][pos[i:i + 1024]].double(), s["weight"], case)
            dx.append(a)
            dw = dw + w
        return {"dx": torch.cat(dx), "dw": dw} if case["norm_dim"] else {"dx": torch.cat(dx)}
    P = case["page"]
    if op == "append":
        kv, codes, scale = s["kv"].double(), s["idx"].view(torch.float8_e4m3fn).double(), s["idx_scale"].double()
        cs = s["cos_sin"][pos].double()
        rows = _exact_rows(s["kv_new"].double()[:, None], cs, s["weight"].double(),
                           dict(norm_dim=512, rope_begin=512, rope_dim=64, interleaved=True))[:, 0]
        keys = _exact_rows(s["idx_new"].double()[:, None], cs, None,
                           dict(norm_dim=0, rope_begin=0, rope_dim=64, interleaved=False))[:, 0]
        sc = (keys.abs().max(1).values / E4M3_MAX).float().double()
        grid = torch.arange(0, 127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
        mid = (grid[1:] + grid[:-1]) / 2
        v = (keys / sc[:, None]).abs()
        near = torch.bucketize(v, mid)                # values on a border go down ...
        on = (near < 126) & (v == mid[near.clamp(max=125)])
        near = near + (on & (near % 2 == 1)).long()   # ... or up, to the even code
        val = grid[near] * keys.sign()
        for b, t0, t1, q, k in spans:
            p = torch.arange(k - q, k, device="cuda")
            pg = s["table"][b].long()[p // P]
            kv[pg, p % P], codes[pg, p % P], scale[pg, p % P] = rows[t0:t1], val[t0:t1], sc[t0:t1]
        return {"kv": kv, "idx": codes, "idx_scale": scale}
    if op == "scores":
        out = torch.full((s["T"], s["max_k"]), -math.inf, dtype=torch.float64, device="cuda")
        for b, t0, t1, q, k in spans:
            p = torch.arange(k, device="cuda")
            pg = s["table"][b].long()[p // P]
            key = s["idx"][pg, p % P].view(torch.float8_e4m3fn).double() * s["idx_scale"][pg, p % P].double()[:, None]
            qr = s["u"][t0:t1].view(torch.float8_e4m3fn).double() * s["s_row"][t0:t1].double()[:, None]
            x = torch.relu(qr @ key.T)
            late = p[None] > torch.arange(k - q, k, device="cuda")[:, None]
            out[t0:t1, :k] = torch.where(late, torch.full_like(x, -math.inf), x)
        return out
    H, dk, dv = case["heads"], case["dk"], case["dv"]
    out = torch.zeros((s["T"], H, dv), dtype=torch.float64, device="cuda")
    lse = torch.full((s["T"], H), -math.inf, dtype=torch.float64, device="cuda")
    for b, t0, t1, q, k in spans:
        p = torch.arange(k, device="cuda")
        pg = s["table"][b].long()[p // P]
        K = s["kv"][pg, p % P].double()
        V = K[:, :dv] if s["v"] is None else s["v"][pg, p % P].double()
        for i in range(t0, t1, 64):
            n = min(i + 64, t1) - i
            if case["selected"]:
                sel = s["sel"][i:i + n].long()
                may = torch.zeros((n, k + 1), dtype=torch.bool, device="cuda")
                may.scatter_(1, torch.where(sel >= 0, sel, torch.full_like(sel, k)), True)
                may = may[:, :k]
            else:
                may = p[None] <= torch.arange(k - q + i - t0, k - q + i - t0 + n, device="cuda")[:, None]
            z = (s["q"][i:i + n].double().reshape(n * H, dk) @ K.T).view(n, H, k) * s["scale"]
            z = torch.where(may[:, None], z, torch.full_like(z, -math.inf))
            some = may.any(1)
            w = torch.softmax(z[some], -1)
            o, r = out[i:i + n], lse[i:i + n]
            o[some] = (w.reshape(-1, k) @ V).view(-1, H, dv)
            r[some] = torch.logsumexp(z[some], -1)
    return {"out": out, "lse": lse}


def _exact_rows(x, cs, w, c):
    n, b0, d = c["norm_dim"], c["rope_begin"], c["rope_dim"]
    y = x.clone()
    if n:
        y[..., :n] = x[..., :n] / ((x[..., :n] ** 2).sum(-1, keepdim=True) / n + EPS) ** 0.5 * w
    cols = torch.arange(d, device="cuda")
    first, second = (cols[0::2], cols[1::2]) if c["interleaved"] else (cols[:d // 2], cols[d // 2:])
    z = torch.complex(y[..., b0 + first], y[..., b0 + second]) * torch.complex(cs[:, :d // 2], cs[:, d // 2:])[:, None]
    y[..., b0 + first], y[..., b0 + second] = z.real, z.imag
    return y


def _exact_rows_bwd(x, dy, cs, w, c):
    """By differentiation of the 64-bit forward."""
    x = x.requires_grad_(True)
    w = w.double().requires_grad_(True) if c["norm_dim"] else None
    with torch.enable_grad():
        y = _exact_rows(x, cs, w, c)
        got = torch.autograd.grad(y, [x] + ([w] if w is not None else []), dy)
    return got[0], got[1] if w is not None else 0
