"""Host-side checks of the query/key transform and the paged-cache entry points
(no GPU needed): bad arguments are refused before anything is launched, and the
workspace follows from the shapes."""
import ctypes

import pytest

P = ctypes.c_void_p
WS = (P(0x10000), 1 << 30, None)  # 256-aligned, never touched on rejection


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_11_b200 import build
    build.build()
    from sparse_attention_11_b200 import dsa
    return dsa


def _seqs(lib, batch=2, tq=64, tk=128, mq=40, mk=100):
    return lib.dsa_seqs(batch, tq, tk, mq, mk, 0x1000, 0x2000)


def _row(lib, **kw):
    a = dict(norm_dim=64, eps=1e-6, weight=0x3000, rope_begin=0, rope_dim=64, rope_interleaved=1, cos_sin=0x4000,
             rope_positions=100)
    a.update(kw)
    return lib.dsa_row_args(*a.values())


def _pages(lib, **kw):
    a = dict(page_size=16, num_pages=20, table=0x5000, ld_table=7, kv_page_stride=16 * 576, v_page_stride=16 * 576,
             idx_page_stride=16 * 128, scale_page_stride=16)
    a.update(kw)
    return lib.dsa_pages(*a.values())


def test_norm_rope_refusals(lib):
    I, U = lib.DSA_ERR_INVALID_ARG, lib.DSA_ERR_UNSUPPORTED

    def fwd(ra=None, dtype=lib.DSA_BF16, heads=2, dim=64, x=0x6000, xs=(128, 64), y=0x7000, ys=(128, 64), ws=WS, s=None):
        ra = ra if ra is not None else _row(lib)
        return lib.raw_call("dsa_norm_rope", ctypes.byref(s or _seqs(lib)), ctypes.byref(ra), dtype, heads, dim, P(x), *xs,
                            P(y), *ys, *ws)

    def bwd(ra=None, dtype=lib.DSA_BF16, x=0x6000, dy=0x7000, dx=0x8000, ws=WS, xs=(128, 64)):
        ra = ra if ra is not None else _row(lib)
        return lib.raw_call("dsa_norm_rope_bwd", ctypes.byref(_seqs(lib)), ctypes.byref(ra), dtype, 2, 64, P(x), *xs,
                            P(dy), 128, 64, P(dx), 128, 64, P(0x9000), *ws)

    for call in (fwd, bwd):
        assert call(_row(lib, norm_dim=65)) == I
        assert call(_row(lib, norm_dim=-1)) == I
        assert call(_row(lib, rope_dim=63)) == I
        assert call(_row(lib, rope_begin=2)) == I          # past the row's end
        assert call(_row(lib, rope_begin=-2, rope_dim=8)) == I
        assert call(_row(lib, cos_sin=None)) == I
        assert call(_row(lib, cos_sin=0x4002)) == I
        assert call(_row(lib, weight=0x3002)) == I
        assert call(_row(lib, eps=-1.0)) == I
        assert call(_row(lib, eps=float("nan"))) == I
        assert call(dtype=lib.DSA_E4M3) == U
        assert call(x=0) == I
        assert call(x=0x6001) == I
        assert call(ws=(P(0x10000), 255, None)) == lib.DSA_ERR_WORKSPACE
        assert call(xs=(127, 64)) == I
        assert call(xs=(128, 63)) == I
        assert call(ws=(P(0x10010), 1 << 20, None)) == I
        assert call(ws=(P(0), 1 << 20, None)) == I
        assert call(ws=(P(0x10000), 64, None)) == lib.DSA_ERR_WORKSPACE
    assert fwd(heads=0) == I
    assert fwd(dim=0) == I
    assert fwd(dim=2049, xs=(5000, 2049), ys=(5000, 2049)) == U
    assert fwd(y=0x6000, ys=(256, 64)) == I                # in place with other strides
    assert fwd(s=_seqs(lib, batch=0)) == I
    assert bwd(dx=0x6000) == I and bwd(dx=0x7000) == I
    assert bwd(ws=(P(0x10000), 4096, None)) == lib.DSA_ERR_WORKSPACE  # the partial sums of d_weight


def test_append_refusals(lib):
    I, U = lib.DSA_ERR_INVALID_ARG, lib.DSA_ERR_UNSUPPORTED

    def call(pg=None, ws=WS, **kw):
        row = _row(lib, norm_dim=512, rope_begin=512)
        key = _row(lib, norm_dim=0)
        a = dict(dtype=lib.DSA_BF16, dim=576, kv_new=0x6000, kv_new_stride=576, kv=0x7000, kv_stride=576,
                 kv_row=ctypes.pointer(row), idx_dtype=lib.DSA_E4M3, idx_new=0x8000, idx_new_stride=128, idx=0x9000,
                 idx_scale=0xA000, idx_row=ctypes.pointer(key))
        a.update(kw)
        ap = lib.dsa_append_args(*a.values())
        return lib.raw_call("dsa_cache_append", ctypes.byref(_seqs(lib)), ctypes.byref(pg or _pages(lib)), ctypes.byref(ap),
                            *ws)

    assert call(_pages(lib, page_size=0)) == I
    assert call(_pages(lib, page_size=65537, kv_page_stride=1 << 40, idx_page_stride=1 << 30, scale_page_stride=1 << 20)) == U
    assert call(_pages(lib, num_pages=-1)) == I
    assert call(_pages(lib, table=None)) == I
    assert call(_pages(lib, ld_table=6)) == I               # 100 positions need 7 pages of 16
    assert call(_pages(lib, kv_page_stride=16 * 576 - 1)) == I
    assert call(_pages(lib, idx_page_stride=15 * 128)) == I
    assert call(_pages(lib, idx_page_stride=16 * 128 + 8)) == I
    assert call(_pages(lib, scale_page_stride=15)) == I
    assert call(kv_new=None, idx_new=None) == I
    assert call(dtype=lib.DSA_E4M3) == U
    assert call(idx_dtype=lib.DSA_BF16) == U
    assert call(idx_dtype=lib.DSA_F32) == U                 # with scales
    assert call(idx_scale=None) == I
    assert call(idx=0x9008) == I
    assert call(kv=None) == I
    assert call(kv_stride=575) == I
    assert call(kv_new_stride=575) == I
    assert call(idx_new_stride=127) == I
    assert call(idx_new=0x8001) == I
    assert call(dim=2049, kv_new_stride=2049, kv_stride=2049, pg=_pages(lib, kv_page_stride=1 << 20)) == U
    assert call(idx_row=ctypes.pointer(_row(lib, norm_dim=129))) == I
    assert call(ws=(P(0x10000), 64, None)) == lib.DSA_ERR_WORKSPACE


def test_scores_and_select_refusals(lib):
    I, U = lib.DSA_ERR_INVALID_ARG, lib.DSA_ERR_UNSUPPORTED

    def scores(pg=None, dtype=lib.DSA_E4M3, u=0x6000, s_row=0x7000, k=0x8000, ks=0x9000, r0=0, n=64, sc=0xA000, ld=100,
               ws=WS):
        return lib.raw_call("dsa_paged_scores", ctypes.byref(_seqs(lib)), ctypes.byref(pg or _pages(lib)), dtype, P(u),
                            P(s_row), P(k), P(ks), r0, n, P(sc), ld, *ws)

    assert scores(dtype=lib.DSA_BF16) == U
    assert scores(dtype=lib.DSA_F32) == U                   # with scales
    assert scores(u=0) == I and scores(u=0x6008) == I and scores(s_row=0) == I
    assert scores(k=0) == I and scores(k=0x8004) == I and scores(ks=0) == I
    assert scores(r0=-1) == I and scores(r0=60, n=5) == I and scores(n=-1) == I
    assert scores(sc=0) == I and scores(ld=99) == I
    assert scores(sc=0xA002) == I and scores(s_row=0x7002) == I and scores(ks=0x9002) == I
    assert scores(_pages(lib, table=0x5002)) == I
    assert scores(_pages(lib, ld_table=6)) == I
    assert scores(ws=(P(0x10000), 64, None)) == lib.DSA_ERR_WORKSPACE

    def select(k=8, idx=0xB000, ld=8, ws=WS, dtype=lib.DSA_E4M3, scales=0x9000, w=0xD000):
        ia = lib.dsa_indexer_args(dtype, 0xC000, 0xC800, lib.DSA_BF16, w, 0x8000, scales, None)
        return lib.raw_call("dsa_paged_select", ctypes.byref(_seqs(lib)), ctypes.byref(_pages(lib)), ctypes.byref(ia), k,
                            P(idx), ld, *ws)

    assert select(k=0) == I and select(idx=0) == I and select(ld=7) == I and select(idx=0xB002) == I
    assert select(scales=None) == I and select(w=None) == I and select(dtype=lib.DSA_BF16) == U
    assert select(ws=(P(0x10000), 1024, None)) == lib.DSA_ERR_WORKSPACE


def test_attention_refusals(lib):
    I, U = lib.DSA_ERR_INVALID_ARG, lib.DSA_ERR_UNSUPPORTED

    def call(pg=None, idx=0, ld=0, k_sel=0, ws=WS, **kw):
        a = dict(dtype=lib.DSA_BF16, heads=128, dk=576, dv=512, q=0x6000, qt=128 * 576, qh=576, k=0x7000, ks=576, v=0x7000,
                 vs=576, scale=0.1, out=0x8000, ot=128 * 512, oh=512, lse=None)
        a.update(kw)
        aa = lib.dsa_attn_args(*a.values())
        return lib.raw_call("dsa_paged_attn", ctypes.byref(_seqs(lib)), ctypes.byref(pg or _pages(lib)), ctypes.byref(aa),
                            P(idx), ld, k_sel, *ws)

    f32 = dict(dtype=lib.DSA_F32, heads=4, dk=64, dv=64, qt=256, qh=64, ks=64, vs=64, ot=256, oh=64)
    assert call(heads=129, qt=129 * 576, ot=129 * 512) == U
    assert call(dk=512) == U and call(dv=576, oh=576, ot=128 * 576) == U
    assert call(v=0x9000) == U and call(vs=584) == U        # V apart from K
    assert call(dtype=lib.DSA_E4M3) == U
    assert call(idx=0xB000, ld=2049, k_sel=2049) == U
    assert call(q=0x6008) == I and call(k=0x7008, v=0x7008) == I and call(out=0x8008) == I
    assert call(q=None) == I and call(k=None, v=None) == I and call(out=None) == I
    assert call(ks=580, vs=580) == I and call(_pages(lib, kv_page_stride=16 * 576 + 4)) == I
    assert call(qt=128 * 576 - 8) == I and call(oh=504) == I
    assert call(scale=-0.1) == I and call(scale=float("nan")) == I
    assert call(heads=0) == I
    assert call(k_sel=8) == I and call(idx=0xB000, ld=8) == I and call(idx=0xB000, ld=7, k_sel=8) == I
    assert call(k_sel=-1) == I and call(idx=0xB002, ld=8, k_sel=8) == I and call(lse=0xE002) == I
    assert call(_pages(lib, kv_page_stride=15 * 576)) == I
    assert call(ws=(P(0x10000), 128, None)) == lib.DSA_ERR_WORKSPACE
    assert call(**dict(f32, heads=33, qt=33 * 64, ot=33 * 64)) == U
    assert call(**dict(f32, dk=48)) == U and call(**dict(f32, dv=160, oh=160, ot=640)) == U
    assert call(**dict(f32, v=0x7002)) == I and call(**dict(f32, vs=32)) == I
    assert call(_pages(lib, kv_page_stride=16 * 64, v_page_stride=15 * 64), **dict(f32, v=0x9000)) == I


def test_workspace_sizes(lib):
    n = ctypes.c_size_t(0)

    def size(op, s, k, ia=None, aa=None):
        r = lib.raw_call("dsa_workspace_size", op, ctypes.byref(s), k, ctypes.byref(ia) if ia else None,
                         ctypes.byref(aa) if aa else None, ctypes.byref(n))
        return n.value if r == 0 else -r

    s = _seqs(lib)
    assert size(lib.DSA_OP_NORM_ROPE_BWD, s, 0) == 256
    assert size(lib.DSA_OP_NORM_ROPE_BWD, s, 512) > 256
    assert size(lib.DSA_OP_NORM_ROPE_BWD, s, -1) < 0
    ia = lib.dsa_indexer_args(lib.DSA_E4M3, 0xC000, 0xC800, lib.DSA_BF16, 0xD000, 0x8000, 0x9000, None)
    assert size(lib.DSA_OP_PAGED_SELECT, s, 8, ia) >= 64 * 100 * 4
    assert size(lib.DSA_OP_PAGED_SELECT, s, 8) < 0
    # at most 1 GiB of scores at a time
    big = lib.dsa_seqs(1, 32768, 65536, 32768, 65536, 0x1000, 0x2000)
    assert size(lib.DSA_OP_PAGED_SELECT, big, 8, ia) < (1 << 30) + 32768 * 256
    aa = lib.dsa_attn_args(lib.DSA_BF16, 128, 576, 512, 0x6000, 128 * 576, 576, 0x7000, 576, 0x7000, 576, 0.1, 0x8000,
                           128 * 512, 512, None)
    # enough query rows for every CTA pair: no parts, a header alone
    many = lib.dsa_seqs(1, 4096, 4096, 4096, 4096, 0x1000, 0x2000)
    assert size(lib.DSA_OP_PAGED_ATTN, many, 2048, None, aa) == 256
    # one decode query over a long cache: its keys in parts
    one = lib.dsa_seqs(1, 1, 65536, 1, 65536, 0x1000, 0x2000)
    assert size(lib.DSA_OP_PAGED_ATTN, one, 0, None, aa) >= 8 * 128 * 512 * 4
    assert size(lib.DSA_OP_PAGED_ATTN, one, -1, None, aa) < 0
    assert size(lib.DSA_OP_PAGED_ATTN, one, 0) < 0


def test_binding_refusals(lib):
    """The binding's own checks, on CPU tensors (nothing is launched)."""
    import torch

    kv, table = torch.zeros(4, 16, 576, dtype=torch.bfloat16), torch.zeros(2, 2, dtype=torch.int32)
    idx, sc = torch.zeros(4, 16, 128, dtype=torch.uint8), torch.zeros(4, 16)
    pages = lib.Pages(table, kv=kv, idx=idx, idx_scale=sc)
    bad = [
        lambda: lib.Pages(table.long(), kv=kv),
        lambda: lib.Pages(table),
        lambda: lib.Pages(table, kv=kv, idx=idx[:3]),
        lambda: lib.Pages(table, kv=kv.half()),
        lambda: lib.Pages(table, kv=kv.transpose(1, 2)),
        lambda: lib.Pages(table, kv=kv, v=kv.float()),
        lambda: lib.Pages(table, idx=idx[..., :64]),
        lambda: lib.Pages(table, idx=idx, idx_scale=sc.double()),
        lambda: lib.row_args(norm_dim=8, weight=torch.ones(9)),
        lambda: lib.row_args(norm_dim=8, weight=torch.ones(8, dtype=torch.float64)),
        lambda: lib.row_args(rope_dim=8),
        lambda: lib.row_args(rope_dim=8, cos_sin=torch.ones(3, 4)),
        lambda: lib.append_args(pages),
        lambda: lib.append_args(pages, kv_new=torch.zeros(3, 576)),
        lambda: lib.append_args(pages, kv_new=torch.zeros(3, 577, dtype=torch.bfloat16)),
        lambda: lib.append_args(pages, idx_new=torch.zeros(3, 64, dtype=torch.bfloat16)),
        lambda: lib.append_args(lib.Pages(table, kv=kv), idx_new=torch.zeros(3, 128, dtype=torch.bfloat16)),
        lambda: lib.paged_attn_args(pages, torch.zeros(3, 2, 576), 1.0, torch.zeros(3, 2, 512)),
        lambda: lib.paged_attn_args(pages, torch.zeros(3, 2, 576).bfloat16(), 1.0, torch.zeros(3, 1, 512).bfloat16()),
        lambda: lib.paged_attn_args(pages, torch.zeros(3, 2, 600).bfloat16(), 1.0, torch.zeros(3, 2, 512).bfloat16()),
        lambda: lib.paged_attn_args(pages, torch.zeros(3, 2, 576).bfloat16(), 1.0, torch.zeros(3, 2, 512).bfloat16(),
                                    torch.zeros(3, 2).double()),
        lambda: lib.dsa_norm_rope(None, None, torch.zeros(3, 2, 8), torch.zeros(3, 2, 8), torch.zeros(256)),  # CPU tensors
        lambda: lib.dsa_cache_append(None, pages, None, torch.zeros(256)),
        lambda: lib.dsa_paged_attn(None, pages, None, None, 0, torch.zeros(256)),
        lambda: lib.paged_indexer_args(pages, torch.zeros(3, 128), None, torch.zeros(128, 128)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"accepted: {i}")


def test_rope_table(lib):
    import math

    import torch

    t = lib.rope_table(70000, 8, device="cpu")
    assert t.shape == (70000, 8) and t.dtype == torch.float32
    for pos in (0, 1, 69999):
        for i in range(4):
            a = pos * 10000.0 ** (-2 * i / 8)
            assert abs(float(t[pos, i]) - math.cos(a)) <= 2.0 ** -24
            assert abs(float(t[pos, 4 + i]) - math.sin(a)) <= 2.0 ** -24
