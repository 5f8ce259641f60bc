"""Calls at the edges of the paged operators: short work items in a long queue,
tokens of no sequence, positions without a page, rows that hold NaN, workspaces
kept for smaller batches.  Formulas and bounds as in paged_util."""
import numpy as np
import pytest
import torch

from paged_util import NOT_SET, Cache, assert_attention, attention

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _plan(c, kv, H, dk, dv, dtype, q=None, k_sel=0, v=None, scale=None):
    """Arguments of an attention call over kv: (aa, q, out, lse, ws, pages, scale)."""
    dsa = c.dsa
    q = c.randn(c.T, H, dk, dtype=dtype) if q is None else q
    out = torch.full((c.T, H, dv), NOT_SET, dtype=dtype, device="cuda")
    lse = torch.full((c.T, H), NOT_SET, device="cuda")
    pages = dsa.Pages(c.table, kv=kv, v=v)
    scale = dk ** -0.5 if scale is None else scale
    aa = dsa.paged_attn_args(pages, q, scale, out, lse)
    ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_PAGED_ATTN, c.seqs, k_sel, None, aa))
    return aa, q, out, lse, ws, pages, scale


# ----------------------------------------------------------------------------- short items
@pytest.mark.parametrize("heads", [128, 16])
@pytest.mark.parametrize("selected", [False, True])
def test_attention_bf16_items_of_one_tile(heads, selected):
    """Many items of one tile each in a CTA's queue: nothing but the barriers of
    the items themselves keeps the softmax from running ahead of the epilogue."""
    rng = np.random.default_rng(3)
    c = Cache([(1, int(n)) for n in rng.integers(1, 65, 700)], 64)
    kv = c.pool(576, BF)
    sel = None
    if selected:
        sel = torch.full((c.T, 64), -1, dtype=torch.int32)
        for t, p in enumerate(c.pos):
            sel[t, :p + 1] = torch.arange(int(p) + 1, dtype=torch.int32)
        sel = sel.cuda()
    aa, q, out, lse, ws, pages, scale = _plan(c, kv, heads, 576, 512, BF, k_sel=64 if selected else 0)
    got = []
    for _ in range(20):
        out.fill_(NOT_SET)
        c.dsa.dsa_paged_attn(c.seqs, pages, aa, sel, 64 if selected else 0, ws)
        got.append((out.clone(), lse.clone()))
    c.dsa.check_device_status(ws)
    assert_attention(c, *got[0], attention(c, q, kv, kv[..., :512], scale, sel), BF)
    for o, l in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(l, got[0][1])


# ----------------------------------------------------------------------------- tokens of no sequence
@pytest.mark.parametrize("heads", [128, 64, 16, 1])
def test_attention_dense_token_behind_the_last_sequence(heads):
    """Recorded, its rows left as they were, where tokens are handled in groups too."""
    c = Cache([(2, 50), (3, 70)], 16)
    c.seqs.c.total_q, c.T = 7, 7
    aa, q, out, lse, ws, pages, scale = _plan(c, c.pool(576, BF), heads, 576, 512, BF)
    c.dsa.dsa_paged_attn(c.seqs, pages, aa, None, 0, ws)
    code, token = c.dsa.dsa_sync_status(ws)
    assert code == c.dsa.DSA_ERR_INDEX and token in (5, 6)
    assert bool((out[5:] == NOT_SET).all()) and bool((lse[5:] == NOT_SET).all())
    c.T = 5
    assert_attention(c, out[:5], lse[:5], attention(c, q[:5], pages.kv, pages.kv[..., :512], scale), BF)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("lens", [[(1, 300), (2, 40)], [(40, 300), (2, 40)]])
def test_scores_token_behind_the_last_sequence(fp8, lens):
    """At most 16 queries a sequence and more: recorded where its row is asked for."""
    c = Cache(lens, 32)
    dsa, n = c.dsa, c.T
    k, sc = c.key_pool(fp8)
    u = c.randn(n + 2, 128)
    if fp8:
        u = u.to(torch.float8_e4m3fn).view(torch.uint8)
    s_row = torch.ones(n + 2, device="cuda")
    c.seqs.c.total_q = n + 2
    pages = dsa.Pages(c.table, idx=k, idx_scale=sc)
    ws = dsa.workspace(256)
    got = torch.full((n + 2, 300), NOT_SET, device="cuda")
    dsa.dsa_paged_scores(c.seqs, pages, u, s_row, 0, n, got, ws)
    assert dsa.dsa_sync_status(ws)[0] == dsa.DSA_OK
    first = got.clone()
    dsa.dsa_paged_scores(c.seqs, pages, u, s_row, 1, n, got[1:], ws)
    code, token = dsa.dsa_sync_status(ws)
    assert code == dsa.DSA_ERR_INDEX and token == n
    assert torch.equal(got, first) and bool((got[n:] == NOT_SET).all())
    dsa.dsa_paged_scores(c.seqs, pages, u, s_row, 0, n + 2, got, ws)
    assert dsa.dsa_sync_status(ws)[0] == dsa.DSA_ERR_INDEX
    assert bool((got[n:] == NOT_SET).all())


# ----------------------------------------------------------------------------- positions without a page
@pytest.mark.parametrize("dtype,heads", [(BF, 128), (BF, 64), (BF, 5), (F32, 4)])
@pytest.mark.parametrize("lens,page", [([(3, 100), (2, 60), (1, 16)], 16), ([(1, 3000), (2, 700)], 48),
                                       ([(70, 260)], 1), ([(4, 4000)], 4096)])
def test_attention_dense_positions_without_a_page(dtype, heads, lens, page):
    """Skipped and recorded by the dense form of every type and head count, inside
    a tile, across tiles and parts, and where no position of a row has a page."""
    c = Cache(lens, page)
    dk, dv = (576, 512) if dtype == BF else (64, 64)
    kv = c.pool(dk, dtype)
    per = [-(-k // page) for _, k in lens]
    bad = [(b, p) for b, n in enumerate(per) for p in range(n) if p % 5 == 1 or n == 1]
    for i, (b, p) in enumerate(bad):
        c.table[b, p] = -1 if i % 2 else c.pages + i
    valid = c.table.clone()
    aa, q, out, lse, ws, pages, scale = _plan(c, kv, heads, dk, dv, dtype)
    c.dsa.dsa_paged_attn(c.seqs, pages, aa, None, 0, ws)
    assert c.dsa.dsa_sync_status(ws)[0] == c.dsa.DSA_ERR_INDEX
    valid[valid >= c.pages] = -1
    c.table = valid
    assert_attention(c, out, lse, attention(c, q, kv, kv[..., :dv], scale), dtype)


# ----------------------------------------------------------------------------- later tokens' rows
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("heads", [128, 64, 16, 5, 1])
@pytest.mark.parametrize("lens,splits", [([(20, 150), (7, 64)], False), ([(130, 130)], False), ([(3, 5000)], True)])
def test_attention_dense_later_rows_hold_anything(heads, bad, lens, splits):
    """A NaN or an infinity in a token's cache row (a latent column of either half, a
    rotated one, or all) reaches no earlier token, to the bit; with a NaN every
    token from its own on is NaN."""
    c = Cache(lens, 16)
    kv = c.pool(576, BF)
    aa, q, out, lse, ws, pages, scale = _plan(c, kv, heads, 576, 512, BF)
    c.dsa.dsa_paged_attn(c.seqs, pages, aa, None, 0, ws)
    c.dsa.check_device_status(ws)
    assert_attention(c, out, lse, attention(c, q, kv, kv[..., :512], scale), BF)
    o0, l0 = out.clone(), lse.clone()
    nq, n = lens[0]
    pg, sl = c.rows(0)
    for cols in (slice(3, 4), slice(300, 301), slice(570, 571), slice(0, 576)):
        for t in {nq - 1, nq // 2, 1}:  # the token of position n - nq + t of sequence 0
            at = n - nq + t
            keep = kv[pg[at], sl[at]].clone()
            kv[pg[at], sl[at], cols] = bad
            out.fill_(NOT_SET), lse.fill_(NOT_SET)
            c.dsa.dsa_paged_attn(c.seqs, pages, aa, None, 0, ws)
            kv[pg[at], sl[at]] = keep
            clean = torch.ones(c.T, dtype=torch.bool, device="cuda")
            clean[t:nq] = False
            assert torch.equal(out[clean], o0[clean]) and torch.equal(lse[clean], l0[clean]), (cols, t)
            if bad != bad:
                assert bool(torch.isnan(out[t:nq]).all()) and bool(torch.isnan(lse[t:nq]).all())
    c.dsa.check_device_status(ws)


# ----------------------------------------------------------------------------- a workspace kept while the batch shrinks
@pytest.mark.parametrize("dtype,heads,selected", [(BF, 128, True), (BF, 128, False), (BF, 16, False), (F32, 4, False),
                                                  (F32, 4, True)])
def test_attention_workspace_of_a_larger_batch(dtype, heads, selected):
    """Sized for 64 sequences, used for 20, 3 and 1: the call takes the parts that fit
    (in bf16 the larger batch has none)."""
    dk, dv = (576, 512) if dtype == BF else (64, 64)
    k_sel = 2048 if selected else 0
    ws = None
    for n in (64, 20, 3, 1):
        c = Cache([(1, 2500 + 7 * i) for i in range(n)], 64, seed=n)
        sel = None
        if selected:
            sel = np.full((n, k_sel), -1, np.int32)
            for t, p in enumerate(c.pos):
                sel[t, :2000] = np.sort(c.rng.permutation(int(p) + 1)[:2000])
            sel = torch.from_numpy(sel).cuda()
        aa, q, out, lse, own, pages, scale = _plan(c, c.pool(dk, dtype), heads, dk, dv, dtype, k_sel=k_sel)
        ws = own if ws is None else ws
        want = attention(c, q, pages.kv, pages.kv[..., :dv], scale, sel)
        for w in (ws, own):
            out.fill_(NOT_SET), lse.fill_(NOT_SET)
            c.dsa.dsa_paged_attn(c.seqs, pages, aa, sel, k_sel, w)
            c.dsa.check_device_status(w)
            assert_attention(c, out, lse, want, dtype)
    with pytest.raises(c.dsa.DsaError):
        c.dsa.dsa_paged_attn(c.seqs, pages, aa, sel, k_sel, own[:128])


def test_select_workspace_of_a_longer_cache():
    """Score rows are handled in whole blocks of queries, so a shorter cache may ask
    for more than a longer one; a workspace of the longer one does, with the same
    indices.  Several pieces of rows, with a k of each query's own."""
    T, longer, shorter, page, k = 300, 1052700, 1048576, 4096, 64
    c = Cache([(T, shorter)], page)
    dsa = c.dsa
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def codes(*shape):
        x = torch.randn(*shape, 128, generator=g, device="cuda")
        return x.to(torch.float8_e4m3fn).view(torch.uint8)

    pages = dsa.Pages(c.table, idx=codes(c.pages, page), idx_scale=torch.rand(c.pages, page, generator=g, device="cuda"))
    k_rows = torch.randint(0, k + 20, (T,), generator=g, device="cuda", dtype=torch.int32)
    ia = dsa.paged_indexer_args(pages, codes(T), torch.ones(T, device="cuda"), torch.randn(128, 128, generator=g,
                                                                                        device="cuda").to(BF), k_rows)
    need = [dsa.dsa_workspace_size(dsa.DSA_OP_PAGED_SELECT, dsa.Seqs([0, T], [0, n]), k, ia) for n in (longer, shorter)]
    assert need[0] < need[1]
    got = []
    for n in need:
        ws = dsa.workspace(n)
        idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
        dsa.dsa_paged_select(c.seqs, pages, ia, k, idx, ws)
        dsa.check_device_status(ws)
        got.append(idx)
    assert torch.equal(got[0], got[1])
    assert torch.equal((got[0] >= 0).sum(1).int(), k_rows.clamp(max=k))
    # a row of the last piece, from its own call
    one = dsa.Seqs([0, 1], [0, shorter])
    ia1 = dsa.paged_indexer_args(pages, ia._keep[0][T - 1:], ia._keep[1][T - 1:], ia._keep[2], k_rows[T - 1:])
    ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_PAGED_SELECT, one, k, ia1))
    idx = torch.empty((1, k), dtype=torch.int32, device="cuda")
    dsa.dsa_paged_select(one, pages, ia1, k, idx, ws)
    assert torch.equal(idx[0], got[0][T - 1])
    with pytest.raises(dsa.DsaError):
        dsa.dsa_paged_select(c.seqs, pages, ia, k, got[0], dsa.workspace(need[1] // 3))


# ----------------------------------------------------------------------------- the queries' scales
def test_scores_f32_scale_of_the_query():
    """s_row multiplies the fp32 scores too: one rounding more than without it."""
    c = Cache([(3, 200), (1, 65)], 16)
    dsa = c.dsa
    k, _ = c.key_pool(False)
    u, s_row = c.randn(c.T, 128), 0.5 + torch.rand(c.T, device="cuda")
    pages = dsa.Pages(c.table, idx=k)
    ws = dsa.workspace(256)
    plain, ones, got = (torch.empty((c.T, 200), device="cuda") for _ in range(3))
    dsa.dsa_paged_scores(c.seqs, pages, u, None, 0, c.T, plain, ws)
    dsa.dsa_paged_scores(c.seqs, pages, u, torch.ones(c.T, device="cuda"), 0, c.T, ones, ws)
    dsa.dsa_paged_scores(c.seqs, pages, u, s_row, 0, c.T, got, ws)
    dsa.check_device_status(ws)
    assert torch.equal(plain, ones)
    assert torch.equal(got, plain * s_row[:, None])


# ----------------------------------------------------------------------------- what the binding refuses
def test_scores_columns_beside_a_view():
    """The -inf of a row ends with the row: a view of a wider tensor keeps what lies
    beside it, so several of its rows are refused and one is served."""
    c = Cache([(3, 200), (1, 65)], 16)
    dsa = c.dsa
    k, _ = c.key_pool(False)
    pages, u, ws = dsa.Pages(c.table, idx=k), c.randn(c.T, 128), dsa.workspace(256)
    buf = torch.full((c.T, 350), NOT_SET, device="cuda")
    want = torch.empty((c.T, 220), device="cuda")
    dsa.dsa_paged_scores(c.seqs, pages, u, None, 0, c.T, want, ws)
    for view in (buf[:, :220], buf[:2, :220]):
        with pytest.raises(ValueError):
            dsa.dsa_paged_scores(c.seqs, pages, u, None, 0, len(view), view, ws)
    for t in range(c.T):
        dsa.dsa_paged_scores(c.seqs, pages, u, None, t, 1, buf[t:, 100:320], ws)
    dsa.check_device_status(ws)
    assert torch.equal(buf[:, 100:320], want)
    assert bool((buf[:, :100] == NOT_SET).all()) and bool((buf[:, 320:] == NOT_SET).all())


def test_lengths_on_another_device_are_refused():
    c = Cache([(2, 50), (1, 3)], 16)
    dsa = c.dsa
    idx, sc = c.key_pool()
    kv, new = c.pool(576, BF), c.randn(3, 576, dtype=BF)
    pages = dsa.Pages(c.table, kv=kv, idx=idx, idx_scale=sc)
    q, out = c.randn(3, 128, 576, dtype=BF), torch.empty(3, 128, 512, dtype=BF, device="cuda")
    u, s_row = torch.zeros(3, 128, dtype=torch.uint8, device="cuda"), torch.ones(3, device="cuda")
    sel = torch.zeros(3, 8, dtype=torch.int32, device="cuda")
    ia = dsa.paged_indexer_args(pages, u, s_row, torch.ones(128, 128, dtype=BF, device="cuda"))
    aa, ap = dsa.paged_attn_args(pages, q, 0.1, out), dsa.append_args(pages, kv_new=new)
    ws = dsa.workspace(1 << 26)

    def calls(s):
        return [lambda: dsa.dsa_norm_rope(s, None, q, q, ws),
                lambda: dsa.dsa_norm_rope_bwd(s, None, None, q, torch.empty_like(q), None, ws),
                lambda: dsa.dsa_cache_append(s, pages, ap, ws),
                lambda: dsa.dsa_paged_scores(s, pages, u, s_row, 0, 3, torch.empty(3, 50, device="cuda"), ws),
                lambda: dsa.dsa_paged_select(s, pages, ia, 8, sel, ws),
                lambda: dsa.dsa_paged_attn(s, pages, aa, None, 0, ws),
                lambda: dsa.dsa_paged_attn(s, pages, aa, sel, 8, ws)]

    for f in calls(dsa.Seqs([0, 2, 3], [0, 50, 53], device="cpu")):
        with pytest.raises(ValueError):
            f()
    for f in calls(c.seqs):
        f()
    dsa.check_device_status(ws)


# ----------------------------------------------------------------------------- parts and their join
@pytest.mark.parametrize("heads", [128, 16])
@pytest.mark.parametrize("n", [20000, 65536])
def test_attention_bf16_many_parts(heads, n):
    """One token over a long cache: more parts than lanes, up to the most there are."""
    c = Cache([(1, n)], 64)
    kv = torch.randn(c.pages, 64, 576, device="cuda").to(BF)
    aa, q, out, lse, ws, pages, scale = _plan(c, kv, heads, 576, 512, BF)
    assert ws.numel() > 256 + 32 * 128 * 513 * 4  # more than 32
    c.dsa.dsa_paged_attn(c.seqs, pages, aa, None, 0, ws)
    c.dsa.check_device_status(ws)
    assert_attention(c, out, lse, attention(c, q, kv, kv[..., :512], scale), BF)


@pytest.mark.parametrize("dtype,heads", [(BF, 128), (BF, 16), (F32, 4)])
@pytest.mark.parametrize("selected", [False, True])
def test_attention_parts_captured(dtype, heads, selected):
    """The kernel that joins parts starts before the parts are done: captured and
    replayed, with lengths that grow and shrink (parts at the end become empty), beside
    a second graph with a workspace of its own."""
    dk, dv = (576, 512) if dtype == BF else (64, 64)
    bound, k_sel = 9000, 1500 if selected else 0
    sides = []
    for seed in (1, 2):
        c = Cache([(1, bound), (2, bound)], 64, seed=seed)
        sel = torch.full((c.T, k_sel), -1, dtype=torch.int32, device="cuda") if selected else None
        plan = _plan(c, c.pool(dk, dtype), heads, dk, dv, dtype, k_sel=k_sel)
        assert plan[4].numel() > 256
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        aa, q, out, lse, ws, pages, scale = plan
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for _ in range(3):
                c.dsa.dsa_paged_attn(c.seqs, pages, aa, sel, k_sel, ws)
        sides.append((c, sel, plan, st, g))
    for lens in ((9000, 9000), (1, 2), (5000, 64), (130, 8999)):
        for c, sel, (aa, q, out, lse, ws, pages, scale), st, g in sides:
            q.copy_(c.randn(c.T, heads, dk, dtype=dtype))
            out.fill_(NOT_SET), lse.fill_(NOT_SET)
            c.seqs.cu_k.copy_(torch.tensor([0, lens[0], lens[0] + lens[1]]))
            live = Cache([(1, lens[0]), (2, lens[1])], 64)
            live.table = c.table
            if selected:
                s = np.full((c.T, k_sel), -1, np.int32)
                for t, p in enumerate(live.pos):
                    n = min(int(p) + 1, k_sel)
                    s[t, :n] = np.sort(c.rng.permutation(int(p) + 1)[:n])
                sel.copy_(torch.from_numpy(s))
        torch.cuda.synchronize()
        for *_, st, g in sides:
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for c, sel, (aa, q, out, lse, ws, pages, scale), st, g in sides:
            c.dsa.check_device_status(ws)
            live = Cache([(1, lens[0]), (2, lens[1])], 64)
            live.table = c.table
            assert_attention(live, out, lse, attention(live, q, pages.kv, pages.kv[..., :dv], scale, sel), dtype)


# ----------------------------------------------------------------------------- strides of dimensions of one
def _loose(t, dims):
    """The same tensor with other strides in its dimensions of one."""
    st = list(t.stride())
    for d in dims:
        assert t.shape[d] == 1
        st[d] = 3
    return t.as_strided(t.shape, st)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strides_of_dimensions_of_one(dtype):
    """One token, one head, pages of one row, a pool of one page: their strides mean
    nothing and refuse nothing, and keep no call from the aligned path."""
    dk, dv = (576, 512) if dtype == BF else (64, 64)
    for heads, page, n in ((1, 1, 9), (4, 1, 9), (4, 16, 9), (1, 16, 9)):
        c = Cache([(1, n)], page, spare=0)
        dsa = c.dsa
        kv = c.pool(dk, dtype)
        q, new = c.randn(1, heads, dk, dtype=dtype), c.randn(1, dk, dtype=dtype)
        out = torch.full((1, heads, dv), NOT_SET, dtype=dtype, device="cuda")
        one = [d for d in (0, 1) if q.shape[d] == 1]
        pools = [d for d in (0, 1) if kv.shape[d] == 1]
        pages = dsa.Pages(c.table, kv=_loose(kv, pools))
        ws = dsa.workspace(1 << 20)
        dsa.dsa_cache_append(c.seqs, pages, dsa.append_args(pages, kv_new=_loose(new, [0])), ws)
        pg, sl = c.rows(0)
        assert torch.equal(kv[pg[-1], sl[-1]], new[0])
        y = torch.empty_like(q)
        dsa.dsa_norm_rope(c.seqs, dsa.row_args(norm_dim=dk), _loose(q, one), _loose(y, one), ws)
        want = torch.empty_like(q)
        dsa.dsa_norm_rope(c.seqs, dsa.row_args(norm_dim=dk), q, want, ws)
        assert torch.equal(y, want)
        aa = dsa.paged_attn_args(pages, _loose(q, one), 0.1, _loose(out, one), lse := torch.empty(1, heads, device="cuda"))
        dsa.dsa_paged_attn(c.seqs, pages, aa, None, 0, ws)
        dsa.check_device_status(ws)
        assert_attention(c, out, lse, attention(c, q, kv, kv[..., :dv], 0.1), dtype)
    idx, sc = c.key_pool()
    pages = dsa.Pages(c.table, idx=_loose(idx, [0]), idx_scale=_loose(sc, [0]))
    key = c.randn(1, 128, dtype=dtype)
    dsa.dsa_cache_append(c.seqs, pages, dsa.append_args(pages, idx_new=_loose(key, [0])), ws)
    dsa.check_device_status(ws)
