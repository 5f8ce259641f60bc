"""The paged cache: append, indexer scores, selection and attention, each
against its formula in 64 bits, on pools whose unused rows hold NaN; then a run
of them together.  Bounds as derived in paged_util; scores by the rule of
gpu_util."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import SCORE_FLOOR, SCORE_REL
from paged_util import (NOT_SET, U, Cache, assert_attention, attention, e4m3_rows, half_step, row_spec, transform)

pytestmark = pytest.mark.gpu

RAGGED = [(3, 3), (1, 200), (0, 64), (70, 333), (1, 1), (20, 1025)]
BF, F32 = torch.bfloat16, torch.float32


# ----------------------------------------------------------------------------- append
@pytest.mark.parametrize("page", [1, 7, 64])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim,rope,interleaved,pad", [(576, 64, True, 0), (576, 64, True, 8), (128, 128, False, 0),
                                                      (75, 26, True, 1), (1500, 512, False, 4)])
def test_append(page, dtype, dim, rope, interleaved, pad):
    c = Cache(RAGGED, page, seed=dim + page, extra_cols=pad)
    dsa = c.dsa
    kv = c.pool(dim, dtype)
    idx, scale = c.key_pool()
    kv_new, idx_new = c.randn(c.T, dim + pad, dtype=dtype)[:, :dim], c.randn(c.T, 128 + pad, dtype=dtype)[:, :128]
    idx_new[0] = 0  # an all-zero key
    n = dim - rope
    kr = row_spec(n, 1 + c.randn(n) * 0.2 if n else None, 1e-6, n, rope, dsa.rope_table(1025, rope), interleaved)
    ir = row_spec(128, 1 + c.randn(128) * 0.2, 1e-6, 0, 64, dsa.rope_table(1025, 64), not interleaved)
    want_kv, mag = kv.double(), torch.zeros_like(kv, dtype=torch.float64)
    want_idx, want_scale = idx.clone(), scale.clone()
    y, m = transform(kv_new[:, None], c.tpos, kr)
    v, sc = e4m3_rows(transform(idx_new[:, None], c.tpos, ir)[0][:, 0])
    codes = v.float().to(torch.float8_e4m3fn).view(torch.uint8)
    for b, (q, k) in enumerate(c.lens):
        pg, sl = (t[k - q:] for t in c.rows(b))
        t = slice(int(c.cq[b]), int(c.cq[b]) + q)
        want_kv[pg, sl], mag[pg, sl] = y[t, 0], m[t, 0]
        want_idx[pg, sl], want_scale[pg, sl] = codes[t], sc[t]
    pages = dsa.Pages(c.table, kv=kv, idx=idx, idx_scale=scale)
    ap = dsa.append_args(pages, kv_new, dsa.row_args(**kr), idx_new, dsa.row_args(**ir))
    ws = dsa.workspace(256)
    dsa.dsa_cache_append(c.seqs, pages, ap, ws)
    dsa.check_device_status(ws)
    err, tol = (kv.double() - want_kv).abs(), half_step(dtype) * want_kv.abs() + 48 * U * mag
    same = torch.isnan(kv) & torch.isnan(want_kv)
    assert bool((same | (err <= tol)).all())
    untouched = mag == 0  # every other row keeps its bits
    assert bool((same | (kv.double() == want_kv) | ~untouched).all())
    # equal values: the sign of a zero code is the key's
    assert torch.equal(idx.view(torch.float8_e4m3fn).float().nan_to_num(-9), want_idx.view(torch.float8_e4m3fn).float()
                       .nan_to_num(-9))
    assert torch.equal(scale.nan_to_num(-9), want_scale.nan_to_num(-9))


@pytest.mark.parametrize("part", ["kv", "idx", "idx_f32"])
def test_append_one_part(part):
    c = Cache(RAGGED, 48)
    dsa = c.dsa
    kv, (idx, scale) = c.pool(64, F32), c.key_pool(part != "idx_f32")
    new = c.randn(c.T, 64 if part == "kv" else 128)
    pages = dsa.Pages(c.table, kv=kv) if part == "kv" else dsa.Pages(c.table, idx=idx, idx_scale=scale)
    ap = dsa.append_args(pages, kv_new=new) if part == "kv" else dsa.append_args(pages, idx_new=new)
    ws = dsa.workspace(256)
    dsa.dsa_cache_append(c.seqs, pages, ap, ws)
    dsa.check_device_status(ws)
    v, sc = e4m3_rows(new.double()) if part == "idx" else (new.double(), None)
    pool = {"kv": kv, "idx": idx.view(torch.float8_e4m3fn) if part == "idx" else None, "idx_f32": idx}[part]
    for b, (q, k) in enumerate(c.lens):
        pg, sl = (t[k - q:] for t in c.rows(b))
        t = slice(int(c.cq[b]), int(c.cq[b]) + q)
        assert torch.equal(pool[pg, sl].double(), v[t])
        if sc is not None:
            assert torch.equal(scale[pg, sl], sc[t])


def test_append_bad_pages():
    """Positions whose table entry is no page, and positions past the cos | sin
    table: recorded, nothing written; the other tokens arrive."""
    c = Cache([(4, 40), (5, 9), (3, 64)], 8)
    dsa = c.dsa
    kv = c.pool(64, F32)
    c.table[0, 4] = -1          # positions 32..39 of sequence 0
    c.table[1, 1] = c.pages     # position 8 of sequence 1
    before = kv.clone()
    new = c.randn(c.T, 64)
    pages = dsa.Pages(c.table, kv=kv)
    ra = dsa.row_args(rope_begin=0, rope_dim=64, cos_sin=dsa.rope_table(63, 64))  # position 63 is past it
    ws = dsa.workspace(256)
    dsa.dsa_cache_append(c.seqs, pages, dsa.append_args(pages, kv_new=new, kv_row=ra), ws)
    assert dsa.dsa_sync_status(ws)[0] == dsa.DSA_ERR_INDEX
    assert dsa.dsa_sync_status(ws)[0] == dsa.DSA_OK
    want, mag = transform(new[:, None], c.tpos.clamp(max=62), row_spec(rope_dim=64, cos_sin=dsa.rope_table(63, 64)))
    for t, (b, p) in enumerate(zip(c.b, c.pos)):
        pg, sl = int(c.table[b, p // 8]), int(p % 8)
        if 0 <= pg < c.pages and p < 63:
            assert bool(((kv[pg, sl].double() - want[t, 0]).abs() <= U * want[t, 0].abs() + 48 * U * mag[t, 0]).all())
            before[pg, sl] = kv[pg, sl]
    assert torch.equal(kv.nan_to_num(-9), before.nan_to_num(-9))


# ----------------------------------------------------------------------------- scores
def _score_inputs(c, fp8):
    k, sc = c.key_pool(fp8)
    if not fp8:
        u = c.randn(c.T, 128)
        return u, None, k, None, u.double()
    v, su = e4m3_rows(c.randn(c.T, 128).double())
    return v.float().to(torch.float8_e4m3fn).view(torch.uint8), su, k, sc, v * su.double()[:, None]


def _score_want(c, uv, k, sc, cols):
    want = torch.full((c.T, cols), -float("inf"), dtype=torch.float64, device="cuda")
    for t in range(c.T):
        b, pos = int(c.b[t]), int(c.pos[t])
        pg, sl = (x[:pos + 1] for x in c.rows(b))
        ok = (pg >= 0) & (pg < c.pages)
        key = k[pg.clamp(0, c.pages - 1), sl]
        key = key.double() if sc is None else key.view(torch.float8_e4m3fn).double() * sc[pg.clamp(0, c.pages - 1), sl,
                                                                                         None].double()
        want[t, :pos + 1] = torch.where(ok, torch.relu(key @ uv[t]), -float("inf"))
    return want


def _assert_scores(got, want):
    inf = torch.isneginf(want)
    assert torch.equal(torch.isneginf(got), inf)
    w = want.masked_fill(inf, 0.0)
    tol = SCORE_REL * w + SCORE_FLOOR * w.amax(1, keepdim=True)
    assert bool(((got.double() - want).abs()[~inf] <= tol[~inf]).all())
    assert not bool(torch.signbit(got[~inf]).any())


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("lens,page", [(RAGGED, 7), (RAGGED, 1), ([(1, 1000), (1, 1), (2, 130), (16, 128)], 64),
                                       ([(300, 300), (1, 129)], 100), ([(129, 2000)], 256), ([(17, 17)], 16)])
def test_scores(fp8, lens, page):
    c = Cache(lens, page, seed=page)
    dsa = c.dsa
    u, su, k, sc, uv = _score_inputs(c, fp8)
    pages = dsa.Pages(c.table, idx=k, idx_scale=sc)
    ws = dsa.workspace(256)
    ld = c.seqs.max_seqlen_k + 5
    got = torch.full((c.T, ld), NOT_SET, device="cuda")
    dsa.dsa_paged_scores(c.seqs, pages, u, su, 0, c.T, got, ws)
    dsa.check_device_status(ws)
    _assert_scores(got, _score_want(c, uv, k, sc, ld))
    # a range of rows: the same bits, and no others written
    r0, n = c.T // 3, c.T - c.T // 3 - c.T // 4
    part = torch.full((n + 2, ld), NOT_SET, device="cuda")
    dsa.dsa_paged_scores(c.seqs, pages, u, su, r0, n, part, ws)
    assert torch.equal(part[:n], got[r0:r0 + n]) and bool((part[n:] == NOT_SET).all())


@pytest.mark.parametrize("fp8", [True, False])
def test_scores_bad_pages(fp8):
    c = Cache([(20, 200), (1, 300)], 32)
    dsa = c.dsa
    u, su, k, sc, uv = _score_inputs(c, fp8)
    c.table[0, 2], c.table[1, 8] = -1, c.pages + 7
    pages = dsa.Pages(c.table, idx=k, idx_scale=sc)
    ws = dsa.workspace(256)
    got = torch.full((c.T, 300), NOT_SET, device="cuda")
    dsa.dsa_paged_scores(c.seqs, pages, u, su, 0, c.T, got, ws)
    assert dsa.dsa_sync_status(ws)[0] == dsa.DSA_ERR_INDEX
    _assert_scores(got, _score_want(c, uv, k, sc, 300))


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("lens,k", [([(1, 3000), (1, 100), (1, 2100), (0, 9)], 2048), ([(90, 700), (3, 3)], 64),
                                    ([(1, 1)], 1)])
def test_select(fp8, lens, k):
    """The oracle's top-k of the scores of dsa_paged_scores, on folded queries."""
    c = Cache(lens, 48, seed=k)
    dsa = c.dsa
    keys, sc = c.key_pool(fp8)
    q = c.randn(c.T, 128)
    w = c.randn(128, 128) / 11
    if fp8:
        v, qs = e4m3_rows(q.double())
        q, w = v.float().to(torch.float8_e4m3fn).view(torch.uint8), w.to(BF)
    else:
        qs = None
    k_rows = torch.from_numpy(c.rng.integers(0, k + 50, c.T).astype(np.int32)).cuda() if c.T > 10 else None
    pages = dsa.Pages(c.table, idx=keys, idx_scale=sc)
    ia = dsa.paged_indexer_args(pages, q, qs, w, k_rows)
    ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_PAGED_SELECT, c.seqs, k, ia))
    idx = torch.full((c.T, k + 3), -7, dtype=torch.int32, device="cuda")
    dsa.dsa_paged_select(c.seqs, pages, ia, k, idx, ws)
    dsa.check_device_status(ws)
    u = torch.empty((c.T, 128), dtype=q.dtype, device="cuda")
    su = torch.empty(c.T, device="cuda")
    dsa.dsa_fold(c.seqs, ia, u, su, ws)
    got = torch.empty((c.T, c.seqs.max_seqlen_k), device="cuda")
    dsa.dsa_paged_scores(c.seqs, pages, u, su if fp8 else None, 0, c.T, got, ws)
    dsa.check_device_status(ws)
    scn, idx = got.cpu().numpy(), idx.cpu().numpy()
    assert np.all(idx[:, k:] == -7)
    for t in range(c.T):
        n = int(c.pos[t]) + 1
        m = min(k if k_rows is None else min(int(k_rows[t]), k), n)
        assert np.all(idx[t, m:k] == -1)
        if m:
            want = oracle.topk(scn[t:t + 1], np.array([n]), m)[0, :m]
            assert np.array_equal(idx[t, :m], np.sort(want))


# ----------------------------------------------------------------------------- attention
def _attn(c, H, dk, dv, dtype, sel=None, scale=None, q=None, kv=None, v=None, lse=True, status=0, qpad=0):
    dsa = c.dsa
    kv = c.pool(dk, dtype) if kv is None else kv
    if q is None:
        q = c.randn(c.T + 1, H + 1, dk + qpad, dtype=dtype)[:, :H, :dk]
    scale = dk ** -0.5 if scale is None else scale
    out = torch.full((c.T + 2, H + (1 if qpad else 0), dv + qpad), NOT_SET, dtype=dtype, device="cuda")[:, :H, :dv]
    ls = torch.full((c.T + 2, H), NOT_SET, device="cuda")
    pages = dsa.Pages(c.table, kv=kv, v=v)
    full = torch.empty((c.T + 2, H, dk), dtype=dtype, device="cuda")
    if qpad == 0:  # as many rows as out
        full[:c.T] = q[:c.T]
        q = full
    else:
        q = torch.cat([q, q[:1]])
        buf = torch.empty((c.T + 2, H, dk + qpad), dtype=dtype, device="cuda")
        buf[..., :dk] = q
        q = buf[..., :dk]
    aa = dsa.paged_attn_args(pages, q, scale, out, ls if lse else None)
    k_sel = 0 if sel is None else sel.shape[1]
    ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_PAGED_ATTN, c.seqs, k_sel, None, aa))
    dsa.dsa_paged_attn(c.seqs, pages, aa, sel, k_sel, ws)
    assert dsa.dsa_sync_status(ws)[0] == status
    assert bool((out[c.T:] == NOT_SET).all()) and bool((ls[c.T:] == NOT_SET).all())
    want = attention(c, q[:c.T], kv, kv[..., :dv] if v is None else v, scale, sel)
    assert_attention(c, out[:c.T], ls[:c.T] if lse else want[1].float(), want, dtype)
    return out[:c.T], ls[:c.T]


def _selection(c, k, seed=0, order="ascending"):
    """Distinct earlier positions a query, -1 after (or between) them; some rows empty."""
    rng = np.random.default_rng(seed)
    sel = np.full((c.T, k), -1, np.int32)
    for t in range(c.T):
        if c.T > 8 and t % 11 == 3:
            continue
        n = int(c.pos[t]) + 1
        p = rng.permutation(n)[:k].astype(np.int32)
        if order == "ascending":
            p = np.sort(p)
            sel[t, :len(p)] = p
        else:
            at = np.sort(rng.permutation(k)[:len(p)])
            sel[t, at] = p
    return torch.from_numpy(sel).cuda()


@pytest.mark.parametrize("heads", [128, 64, 48, 16, 5, 1])
@pytest.mark.parametrize("lens,page", [(RAGGED, 7), ([(1, 1000), (1, 1), (1, 64), (1, 65)], 64), ([(130, 130)], 48)])
def test_attention_dense_bf16(heads, lens, page):
    _attn(Cache(lens, page, seed=heads), heads, 576, 512, BF)


@pytest.mark.parametrize("page", [1, 256])
def test_attention_dense_bf16_pages_and_strides(page):
    c = Cache([(9, 300), (2, 77)], page, extra_cols=24)
    _attn(c, 32, 576, 512, BF, qpad=8)


def test_attention_dense_bf16_many_sequences():
    """More work items than CTA pairs: the pipeline crosses item boundaries."""
    rng = np.random.default_rng(5)
    lens = [(int(rng.integers(0, 4)), int(rng.integers(4, 300))) for _ in range(150)]
    _attn(Cache(lens, 32), 128, 576, 512, BF)


def test_attention_dense_bf16_long():
    """Parts of a long cache, joined."""
    _attn(Cache([(1, 20000), (2, 9000)], 64), 128, 576, 512, BF)


@pytest.mark.parametrize("heads", [128, 40, 3])
@pytest.mark.parametrize("k,order", [(1, "ascending"), (63, "ascending"), (64, "mixed"), (500, "mixed"), (2048, "ascending")])
def test_attention_selected_bf16(heads, k, order):
    c = Cache([(30, 700), (1, 2500), (0, 3), (1, 1)], 20, seed=k)
    _attn(c, heads, 576, 512, BF, sel=_selection(c, k, k, order))


def test_attention_selected_bf16_many_queries():
    c = Cache([(200, 900), (60, 70)], 64)
    _attn(c, 128, 576, 512, BF, sel=_selection(c, 150, 1))


@pytest.mark.parametrize("heads,dk,dv,own_v", [(4, 64, 64, False), (1, 32, 32, True), (32, 128, 128, True),
                                                (9, 96, 32, True), (6, 32, 128, True), (7, 128, 96, False)])
def test_attention_f32(heads, dk, dv, own_v):
    c = Cache(RAGGED, 20, seed=dk)
    kv = c.pool(dk, F32)
    v = c.pool(dv, F32) if own_v else None
    if not own_v and dv > dk:
        pytest.skip("V within K")
    _attn(c, heads, dk, dv, F32, kv=kv, v=v)
    _attn(c, heads, dk, dv, F32, kv=kv, v=v, sel=_selection(c, 40, 3, "mixed"))


@pytest.mark.parametrize("lens", [[(1, 5000)], [(2, 12000), (1, 300)], [(1, 130), (1, 1)], [(300, 300)]])
@pytest.mark.parametrize("heads", [1, 4, 32])
def test_attention_f32_parts(lens, heads):
    """One block a token, clusters of 2 to 8 parts, and more parts than a cluster."""
    c = Cache(lens, 16)
    _attn(c, heads, 64, 96, F32, v=c.pool(96, F32))
    _attn(c, heads, 64, 96, F32, v=c.pool(96, F32), sel=_selection(c, 1000, 1))


def test_attention_f32_unaligned_rows():
    c = Cache([(5, 100), (1, 33)], 7, extra_cols=3)
    _attn(c, 4, 64, 64, F32, v=c.pool(64, F32), qpad=1)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_large_scores(dtype):
    """Scores of some hundred, of both signs, rising and falling along the keys:
    the running maximum moves often, and the two halves of the contraction
    nearly cancel."""
    c = Cache([(3, 500), (1, 900)], 32)
    H, dk, dv = (128, 576, 512) if dtype == BF else (4, 64, 64)
    kv = c.pool(dk, dtype)
    half = dk // 2
    for b, (_, n) in enumerate(c.lens):
        pg, sl = c.rows(b)
        ramp = torch.sin(torch.arange(n, device="cuda") * 0.05) * 3
        rows = torch.randn(n, dk, device="cuda") * 0.05
        rows[:, :half] += ramp[:, None]
        rows[:, half:] -= ramp[:, None] * 0.98
        kv[pg, sl] = rows.to(dtype)
    q = torch.ones(c.T + 1, H + 1, dk, device="cuda", dtype=dtype)[:, :H]
    q = q * torch.linspace(-1, 1, H, device="cuda", dtype=dtype)[None, :, None]
    _attn(c, H, dk, dv, dtype, q=q, kv=kv, scale=0.5)
    _attn(c, H, dk, dv, dtype, q=q, kv=kv, scale=0.0)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_bad_slots(dtype):
    """Slots past the sequence or without a page are skipped and recorded."""
    c = Cache([(3, 100), (2, 60)], 16)
    H, dk, dv = (128, 576, 512) if dtype == BF else (4, 64, 64)
    kv = c.pool(dk, dtype)
    sel = _selection(c, 50)
    sel[1, 4] = 100
    c.table[1, 1] = -1
    _attn(c, H, dk, dv, dtype, kv=kv, sel=sel, status=c.dsa.DSA_ERR_INDEX)


@pytest.mark.parametrize("selected", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_nan_query(dtype, selected):
    """A query row of NaN gives a row of NaN and a NaN lse, its neighbours what
    they give without it; a row of a selection with no valid slot gives zeros."""
    c = Cache([(3, 200), (2, 60)], 16)
    dsa = c.dsa
    H, dk, dv = (128, 576, 512) if dtype == BF else (4, 64, 64)
    kv, q = c.pool(dk, dtype), c.randn(c.T, H, dk, dtype=dtype)
    sel = torch.arange(40, dtype=torch.int32, device="cuda").repeat(c.T, 1) if selected else None
    if selected:
        sel[3] = -1
    pages = dsa.Pages(c.table, kv=kv)
    got = []
    for bad in (False, True):
        if bad:
            q[1, 2], q[3, 0] = float("nan"), float("nan")
        out, lse = torch.empty(c.T, H, dv, dtype=dtype, device="cuda"), torch.empty(c.T, H, device="cuda")
        aa = dsa.paged_attn_args(pages, q, 0.1, out, lse)
        k = sel.shape[1] if selected else 0
        ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_PAGED_ATTN, c.seqs, k, None, aa))
        dsa.dsa_paged_attn(c.seqs, pages, aa, sel, k, ws)
        dsa.check_device_status(ws)
        got.append((out, lse))
    (o0, l0), (o1, l1) = got
    nan = torch.zeros(c.T, H, dtype=torch.bool, device="cuda")
    nan[1, 2], nan[3, 0] = True, not selected
    assert torch.equal(torch.isnan(l1), nan) and torch.equal(torch.isnan(o1).all(-1), nan)
    assert torch.equal(o1[~nan], o0[~nan]) and torch.equal(l1[~nan], l0[~nan])
    if selected:
        assert bool((o1[3] == 0).all()) and bool((l1[3] == -float("inf")).all())


def test_attention_without_lse():
    c = Cache([(3, 100)], 16)
    _attn(c, 128, 576, 512, BF, lse=False)


def test_rows_without_a_position():
    """A sequence of more queries than positions, and rows behind the last
    sequence: recorded, left as they were."""
    for dtype, H, dk, dv in ((BF, 128, 576, 512), (F32, 4, 64, 64)):
        for k_sel in (0, 8):
            c = Cache([(2, 50)], 16)
            dsa = c.dsa
            c.seqs.c.total_q, c.T = 4, 4
            kv = c.pool(dk, dtype)
            q = c.randn(4, H, dk, dtype=dtype)
            out, lse = torch.full((4, H, dv), NOT_SET, dtype=dtype, device="cuda"), torch.full((4, H), NOT_SET, device="cuda")
            pages = dsa.Pages(c.table, kv=kv)
            aa = dsa.paged_attn_args(pages, q, 0.1, out, lse)
            sel = torch.arange(8, dtype=torch.int32, device="cuda").repeat(4, 1) if k_sel else None
            ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_PAGED_ATTN, c.seqs, k_sel, None, aa))
            dsa.dsa_paged_attn(c.seqs, pages, aa, sel, k_sel, ws)
            assert dsa.dsa_sync_status(ws)[0] == dsa.DSA_ERR_INDEX
            assert bool((out[2:] == NOT_SET).all()) and bool((lse[2:] == NOT_SET).all())
            want = attention(c, q[:2], kv, kv[..., :dv], 0.1, None if sel is None else sel[:2])
            assert_attention(c, out[:2], lse[:2], want, dtype)


def test_offsets_past_32_bits():
    """Pages whose rows start past 2^31 elements (and 2^32 bytes) of the pool."""
    c = Cache([(2, 150)], 64)
    dsa = c.dsa
    stride = 1 << 29  # elements between pages
    n = c.pages
    flat = torch.empty((n - 1) * stride + 64 * 576, dtype=BF, device="cuda")
    kv = flat.as_strided((n, 64, 576), (stride, 576, 1))
    assert (n - 1) * stride > 1 << 31
    c.table[0, :3] = torch.tensor([n - 1, 0, n - 2], dtype=torch.int32)
    new = c.randn(150, 576, dtype=BF)
    pages = dsa.Pages(c.table, kv=kv)
    fill = dsa.Seqs([0, 150], [0, 150])
    ws = dsa.workspace(256)
    dsa.dsa_cache_append(fill, pages, dsa.append_args(pages, kv_new=new), ws)
    dsa.check_device_status(ws)
    pg, sl = c.rows(0)
    assert torch.equal(kv[pg, sl], new)
    _attn(c, 128, 576, 512, BF, kv=kv)
    _attn(c, 128, 576, 512, BF, kv=kv, sel=_selection(c, 64))


# ----------------------------------------------------------------------------- together
class Layer:
    """One layer's attention step on a paged cache: rotate the queries, append the
    new tokens, select, attend."""

    def __init__(self, c, k, H=128):
        self.c, self.k, self.H, self.dsa = c, k, H, c.dsa
        dsa = self.dsa
        self.kv = torch.full((c.pages, c.page, 576), float("nan"), dtype=BF, device="cuda")
        self.idx = torch.full((c.pages, c.page, 128), 0x7F, dtype=torch.uint8, device="cuda")
        self.scale = torch.full((c.pages, c.page), float("nan"), device="cuda")
        self.pages = dsa.Pages(c.table, kv=self.kv, idx=self.idx, idx_scale=self.scale)
        tab = dsa.rope_table(2048, 64)
        self.q_row = dsa.row_args(rope_begin=512, rope_dim=64, cos_sin=tab)
        self.w = 1 + 0.2 * c.randn(512)
        self.kv_row = dsa.row_args(norm_dim=512, weight=self.w, rope_begin=512, rope_dim=64, cos_sin=tab)
        self.idx_row = dsa.row_args(rope_begin=0, rope_dim=64, cos_sin=tab, interleaved=False)
        self.tab, self.w_index = tab, (c.randn(128, 128) / 11).to(BF)

    def inputs(self, T):
        c = self.c
        v, s = e4m3_rows(c.randn(T, 128).double())
        return dict(q=c.randn(T, self.H, 576, dtype=BF), kv=c.randn(T, 576, dtype=BF), key=c.randn(T, 128, dtype=BF),
                    q_idx=v.float().to(torch.float8_e4m3fn).view(torch.uint8), q_s=s,
                    idx=torch.empty((T, self.k), dtype=torch.int32, device="cuda"),
                    qr=torch.empty((T, self.H, 576), dtype=BF, device="cuda"),
                    out=torch.empty((T, self.H, 512), dtype=BF, device="cuda"), lse=torch.empty((T, self.H), device="cuda"))

    def plan(self, seqs, x):
        dsa = self.dsa
        p = dict(seqs=seqs, x=x, ap=dsa.append_args(self.pages, x["kv"], self.kv_row, x["key"], self.idx_row),
                 ia=dsa.paged_indexer_args(self.pages, x["q_idx"], x["q_s"], self.w_index),
                 aa=dsa.paged_attn_args(self.pages, x["qr"], 576 ** -0.5, x["out"], x["lse"]))
        p["ws"] = dsa.workspace(max(dsa.dsa_workspace_size(dsa.DSA_OP_PAGED_SELECT, seqs, self.k, p["ia"]),
                                    dsa.dsa_workspace_size(dsa.DSA_OP_PAGED_ATTN, seqs, self.k, None, p["aa"])))
        return p

    def step(self, p):
        dsa, s, x, ws = self.dsa, p["seqs"], p["x"], p["ws"]
        dsa.dsa_norm_rope(s, self.q_row, x["q"], x["qr"], ws)
        dsa.dsa_cache_append(s, self.pages, p["ap"], ws)
        dsa.dsa_paged_select(s, self.pages, p["ia"], self.k, x["idx"], ws)
        dsa.dsa_paged_attn(s, self.pages, p["aa"], x["idx"], self.k, ws)


def test_binding_refusals():
    """What the binding can see of a call that would read or write out of range."""
    c = Cache([(2, 100), (1, 40)], 16)
    dsa = c.dsa
    kv = c.pool(576, BF)
    q, out = c.randn(3, 128, 576, dtype=BF), torch.empty(3, 128, 512, dtype=BF, device="cuda")
    ws = dsa.workspace(1 << 26)

    def attn(table=c.table, q=q, idx=None, k=0, ws=ws):
        pages = dsa.Pages(table, kv=kv)
        dsa.dsa_paged_attn(c.seqs, pages, dsa.paged_attn_args(pages, q, 0.1, out[:len(q)]), idx, k, ws)

    attn()
    sel = torch.zeros(3, 8, dtype=torch.int32, device="cuda")
    bad = [lambda: attn(table=c.table[:, :6]), lambda: attn(table=c.table[:1]), lambda: attn(q=q[:2]),
           lambda: attn(idx=sel, k=9), lambda: attn(idx=sel[:2], k=8), lambda: attn(idx=sel.long(), k=8),
           lambda: attn(idx=sel.cpu(), k=8), lambda: attn(ws=ws.cpu()),
           lambda: dsa.paged_attn_args(dsa.Pages(c.table, kv=kv), q.cpu(), 0.1, out),
           lambda: dsa.append_args(dsa.Pages(c.table, kv=kv), kv_new=torch.zeros(3, 576, dtype=BF)),
           lambda: dsa.append_args(dsa.Pages(c.table, kv=kv), kv_new=q[:, 0],
                                   kv_row=dsa.row_args(norm_dim=8, weight=torch.ones(8))),
           lambda: dsa.dsa_norm_rope(c.seqs, dsa.row_args(norm_dim=8, weight=torch.ones(8)), q, torch.empty_like(q), ws),
           lambda: dsa.dsa_norm_rope(c.seqs, None, q, torch.empty_like(q)[:2], ws)]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, dsa.DsaError)):
            f()
            pytest.fail(f"accepted: {i}")
    with pytest.raises(dsa.DsaError):
        attn(ws=ws[:128])
    dsa.check_device_status(ws)


@pytest.mark.parametrize("fp8", [True, False])
def test_select_binding_refusals(fp8):
    """Arguments made over other pools, fewer queries than the batch, another device."""
    c = Cache([(2, 100), (1, 40)], 16)
    dsa = c.dsa
    idx, sc = c.key_pool(fp8)
    pages, other = dsa.Pages(c.table, idx=idx, idx_scale=sc), None
    if fp8:
        q, qs = torch.zeros(3, 128, dtype=torch.uint8, device="cuda"), torch.ones(3, device="cuda")
        w = torch.ones(128, 128, dtype=BF, device="cuda")
        other = dsa.Pages(c.table, idx=idx, idx_scale=sc.clone())
    else:
        q, qs, w = torch.zeros(3, 128, device="cuda"), None, torch.ones(128, 128, device="cuda")
    short = dsa.Pages(c.table, idx=idx[:4].clone(), idx_scale=None if sc is None else sc[:4].clone())
    out = torch.empty(3, 8, dtype=torch.int32, device="cuda")
    ia = dsa.paged_indexer_args(pages, q, qs, w)
    ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_PAGED_SELECT, c.seqs, 8, ia))
    bad = [lambda: dsa.dsa_paged_select(c.seqs, pages, dsa.paged_indexer_args(short, q, qs, w), 8, out, ws),
           lambda: dsa.dsa_paged_select(c.seqs, pages, dsa.paged_indexer_args(pages, q[:2], qs, w), 8, out, ws),
           lambda: dsa.paged_indexer_args(pages, q.cpu(), qs, w), lambda: dsa.paged_indexer_args(pages, q, qs, w.cpu())]
    if other is not None:
        bad.append(lambda: dsa.dsa_paged_select(c.seqs, other, ia, 8, out, ws))
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"accepted: {i}")


def _prefix(lens):
    return np.concatenate([[0], np.cumsum(lens)])


def test_prefill_then_decode():
    """A prefill of three sequences in two chunks, then decode steps, against the
    framework's packed path on the whole sequences: the same selections, the
    same rows within the attention's bound."""
    total = [300, 130, 411]
    c = Cache([(n, n) for n in total], 48)
    L = Layer(c, 64)
    dsa = L.dsa
    T = c.T
    full = L.inputs(T)

    def piece(lo, hi):  # positions [lo, hi) of every sequence, clipped to its length
        rows = np.concatenate([c.cq[b] + np.arange(min(lo[b], n), min(hi[b], n)) for b, n in enumerate(total)])
        r = torch.from_numpy(rows).cuda()
        x = L.inputs(len(rows))
        for k in ("q", "kv", "key", "q_idx", "q_s"):
            x[k].copy_(full[k][r])
        q = [min(hi[b], n) - min(lo[b], n) for b, n in enumerate(total)]
        seqs = dsa.Seqs(_prefix(q), _prefix([min(hi[b], n) for b, n in enumerate(total)]))
        p = L.plan(seqs, x)
        L.step(p)
        dsa.check_device_status(p["ws"])
        for k in ("idx", "out", "lse", "qr"):
            full[k][r] = x[k]

    piece([0, 0, 0], [100, 57, 200])
    piece([100, 57, 200], [296, 126, 407])
    for i in range(4):
        piece([296 + i, 126 + i, 407 + i], [297 + i, 127 + i, 408 + i])
    # the packed path on all tokens at once
    kv = torch.cat([L.kv[c.rows(b)] for b in range(3)])
    codes, sc = torch.cat([L.idx[c.rows(b)] for b in range(3)]), torch.cat([L.scale[c.rows(b)] for b in range(3)])
    y, mag = transform(full["kv"][:, None], c.tpos, row_spec(512, L.w, 1e-6, 512, 64, L.tab, True))
    assert bool(((kv.double() - y[:, 0]).abs() <= half_step(BF) * y[:, 0].abs() + 48 * U * mag[:, 0]).all())
    seqs = dsa.Seqs(c.cq, c.cq)
    ia = dsa.indexer_args(full["q_idx"], full["q_s"], L.w_index, codes, sc)
    out, lse = torch.empty_like(full["out"]), torch.empty_like(full["lse"])
    aa = dsa.attn_args(full["qr"], kv, kv[:, :512], 576 ** -0.5, out, lse)
    idx = torch.empty_like(full["idx"])
    ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_FORWARD, seqs, 64, ia, aa))
    dsa.dsa_forward(seqs, ia, aa, 64, idx, ws)
    dsa.check_device_status(ws)
    a, b = full["idx"].cpu().numpy(), idx.cpu().numpy()
    same = np.array([len(np.intersect1d(x[x >= 0], y[y >= 0])) / max((y >= 0).sum(), 1) for x, y in zip(a, b)])
    assert same.mean() >= 0.999
    want = attention(c, full["qr"], L.kv, L.kv[..., :512], 576 ** -0.5, full["idx"])
    assert_attention(c, full["out"], full["lse"], want, BF)
    agree = torch.from_numpy((a == b).all(1)).cuda()
    assert_attention(c, out[agree], lse[agree], [x[agree] for x in want], BF)


def test_captured_decode_step():
    """A decode step captured once and replayed while the sequences grow: lengths,
    table and inputs are read when it runs.  Two graphs with workspaces of their
    own run at once on two streams."""
    bound = 500  # the longest any sequence gets
    n = 5

    def make(seed):
        c = Cache([(1, bound)] * n, 32, seed=seed)
        L = Layer(c, 100)
        # a cache in use: rows of every position, so that any length is valid
        fill = c.dsa.Seqs(_prefix([bound] * n), _prefix([bound] * n))
        p = L.plan(fill, L.inputs(bound * n))
        c.dsa.dsa_cache_append(fill, L.pages, p["ap"], p["ws"])
        c.dsa.check_device_status(p["ws"])
        seqs = c.dsa.Seqs(np.arange(n + 1), _prefix([bound] * n))
        return c, L, L.plan(seqs, L.inputs(n))

    sides = [make(1), make(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs = []
    for (c, L, p), st in zip(sides, streams):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            L.step(p)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            L.step(p)
        graphs.append(g)
    for lens in ([1, 64, 65, 300, 500], [2, 65, 66, 301, 500], [33, 1, 499, 100, 7]):
        for (c, L, p), st in zip(sides, streams):
            x = L.inputs(n)
            for k in ("q", "kv", "key", "q_idx", "q_s"):
                p["x"][k].copy_(x[k])
            p["seqs"].cu_k.copy_(torch.from_numpy(_prefix(lens)))
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for c, L, p in sides:
            c.dsa.check_device_status(p["ws"])
            got = {k: p["x"][k].clone() for k in ("idx", "out", "lse")}
            live = Cache([(1, k) for k in lens], 32)
            live.table = c.table
            want = attention(live, p["x"]["qr"], L.kv, L.kv[..., :512], 576 ** -0.5, got["idx"])
            assert_attention(live, got["out"], got["lse"], want, BF)
            for t, k in enumerate(lens):
                assert int((got["idx"][t] >= 0).sum()) == min(k, 100) and int(got["idx"][t].max()) < k
            L.step(p)  # the same step without the graph: the same bits
            for k, v in got.items():
                assert torch.equal(p["x"][k], v), k
