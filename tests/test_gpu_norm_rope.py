"""The query/key transform (RMS norm and position rotation) and its gradients
against the formulas in 64 bits and against differences; bounds as derived in
paged_util."""
import pytest
import torch

from paged_util import NOT_SET, U, half_step, row_spec, transform, transform_bwd

pytestmark = pytest.mark.gpu

LENS = [(1, 1), (0, 5), (37, 900), (1, 5000), (6, 6)]
# dim, norm_dim, rope_begin, rope_dim, interleaved, weight
ROWS = {
    "latent_q": (576, 0, 512, 64, True, False),
    "latent_k": (576, 512, 512, 64, True, True),
    "head": (128, 128, 0, 128, False, True),
    "head_part": (192, 192, 128, 64, False, True),
    "head_ones": (64, 64, 0, 32, True, False),
    "inside": (256, 192, 64, 96, False, True),
    "norm_only": (1024, 1024, 0, 0, True, True),
    "wide": (2048, 2000, 1024, 1024, False, True),
    "copy": (40, 0, 0, 0, True, False),
    "odd": (75, 70, 3, 26, True, True),      # not whole 16-byte pieces
    "odd_half": (130, 130, 1, 50, False, True),
    "one": (1, 1, 0, 0, True, True),
    "half8": (64, 64, 8, 24, False, True),   # half-split pairs 12 columns apart
}


def _setup(kind, dtype, heads, pad=0, seed=0):
    from sparse_attention_11_b200 import dsa

    dim, nd, rb, rd, il, weighted = ROWS[kind]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    cq, ck = [0], [0]
    for q, k in LENS:
        cq.append(cq[-1] + q)
        ck.append(ck[-1] + k)
    seqs = dsa.Seqs(cq, ck)
    pos = torch.cat([torch.arange(k - q, k, device="cuda") for q, k in LENS])
    T = cq[-1]

    def rows():
        full = torch.full((T + 2, heads + 1, dim + pad), NOT_SET, dtype=dtype, device="cuda")
        full[:T, :heads, :dim] = torch.randn((T, heads, dim), generator=g, device="cuda").to(dtype)
        return full[:, :heads, :dim]

    ra = row_spec(nd, 1 + 0.3 * torch.randn(nd, generator=g, device="cuda") if weighted else None, 1e-6, rb, rd,
                  dsa.rope_table(5000, rd) if rd else None, il)
    return dsa, seqs, T, pos, ra, rows


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", list(ROWS))
def test_forward(kind, dtype):
    for heads, pad in ((1, 0), (3, 8), (5, 1)):  # pad 1: rows on no 16-byte boundary
        dsa, seqs, T, pos, ra, rows = _setup(kind, dtype, heads, pad)
        x = rows()
        y = torch.full_like(x, NOT_SET)
        ws = dsa.workspace(256)
        dsa.dsa_norm_rope(seqs, dsa.row_args(**ra), x, y, ws)
        dsa.check_device_status(ws)
        want, mag = transform(x[:T], pos, ra)
        tol = half_step(dtype) * want.abs() + 48 * U * mag
        assert bool(((y[:T].double() - want).abs() <= tol).all()), (kind, heads, pad)
        assert bool((y[T:] == NOT_SET).all())
        y2 = torch.empty_strided(x.shape, x.stride(), dtype=dtype, device="cuda").copy_(x)
        dsa.dsa_norm_rope(seqs, dsa.row_args(**ra), y2, y2, ws)  # in place
        assert torch.equal(y2[:T], y[:T])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", list(ROWS))
def test_backward(kind, dtype):
    for heads, pad in ((1, 0), (3, 8), (5, 1)):
        dsa, seqs, T, pos, ra, rows = _setup(kind, dtype, heads, pad)
        x, dy = rows(), rows()
        dx = torch.full_like(x, NOT_SET)
        n = ra["norm_dim"]
        ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_NORM_ROPE_BWD, seqs, n))
        dw = torch.full((n,), NOT_SET, device="cuda") if n else None
        dsa.dsa_norm_rope_bwd(seqs, dsa.row_args(**ra), x, dy, dx, dw, ws)
        dsa.check_device_status(ws)
        want, mag, want_w, mag_w = transform_bwd(x[:T], dy[:T], pos, ra)
        tol = half_step(dtype) * want.abs() + 160 * U * mag
        assert bool(((dx[:T].double() - want).abs() <= tol).all()), (kind, heads, pad)
        assert bool((dx[T:] == NOT_SET).all())
        if n:
            assert bool(((dw.double() - want_w).abs() <= 80 * U * mag_w).all()), (kind, heads, pad)
            dx2, dw2 = torch.empty_like(dx), torch.empty_like(dw)
            dsa.dsa_norm_rope_bwd(seqs, dsa.row_args(**ra), x, dy, dx2, dw2, ws)
            assert torch.equal(dw, dw2) and torch.equal(dx[:T], dx2[:T])  # the same bits again
            dx3 = torch.empty_like(dx)
            dsa.dsa_norm_rope_bwd(seqs, dsa.row_args(**ra), x, dy, dx3, None, ws)  # without the weight's gradient
            assert torch.equal(dx[:T], dx3[:T])


@pytest.mark.parametrize("kind", ["latent_k", "head", "odd"])
def test_backward_against_differences(kind):
    """<dy, (f(x + h d) - f(x - h d)) / 2h> against <dx, d> with the forward in 64
    bits: the difference's own error is O(h^2) = 1e-8 relative, dx's bound 160 u of
    its magnitude, summed."""
    dsa, seqs, T, pos, ra, rows = _setup(kind, torch.float32, 2)
    x, dy, d = rows(), rows(), rows()
    n = ra["norm_dim"]
    dx, dw = torch.empty_like(x), torch.empty(n, device="cuda")
    ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_NORM_ROPE_BWD, seqs, n))
    dsa.dsa_norm_rope_bwd(seqs, dsa.row_args(**ra), x, dy, dx, dw, ws)
    h, x, dy, d = 1e-4, x[:T].double(), dy[:T].double(), d[:T].double()
    _, mag, _, mag_w = transform_bwd(x, dy, pos, ra)
    num = (dy * (transform(x + h * d, pos, ra)[0] - transform(x - h * d, pos, ra)[0])).sum() / (2 * h)
    bound = 160 * U * (mag * d.abs()).sum() + 1e-6 * (mag * d.abs()).sum()
    assert abs(float(num - (dx[:T].double() * d).sum())) <= float(bound)
    w, e = ra["weight"], torch.randn(n, device="cuda").double()
    up, dn = dict(ra, weight=w.double() + h * e), dict(ra, weight=w.double() - h * e)
    num = (dy * (transform(x, pos, up)[0] - transform(x, pos, dn)[0])).sum() / (2 * h)
    assert abs(float(num - (dw.double() * e).sum())) <= float((80 * U + 1e-9) * (mag_w * e.abs()).sum())


def test_many_rows_a_warp():
    """Enough rows that every lane sums several of them (a chain of 16 at most)."""
    from sparse_attention_11_b200 import dsa

    T, H, n = 3000, 16, 128
    seqs = dsa.Seqs([0, T], [0, T])
    ra = row_spec(n, torch.randn(n, device="cuda"), 1e-6, 0, n, dsa.rope_table(T, n), False)
    x, dy = torch.randn(T, H, n, device="cuda"), torch.randn(T, H, n, device="cuda")
    dx, dw, y = torch.empty_like(x), torch.empty(n, device="cuda"), torch.empty_like(x)
    ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_NORM_ROPE_BWD, seqs, n))
    dsa.dsa_norm_rope_bwd(seqs, dsa.row_args(**ra), x, dy, dx, dw, ws)
    dsa.dsa_norm_rope(seqs, dsa.row_args(**ra), x, y, ws)
    dsa.check_device_status(ws)
    pos = torch.arange(T, device="cuda")
    want, mag, want_w, mag_w = transform_bwd(x, dy, pos, ra)
    assert bool(((dx.double() - want).abs() <= half_step(x.dtype) * want.abs() + 160 * U * mag).all())
    assert bool(((dw.double() - want_w).abs() <= 80 * U * mag_w).all())
    want, mag = transform(x, pos, ra)
    assert bool(((y.double() - want).abs() <= half_step(x.dtype) * want.abs() + 48 * U * mag).all())


def test_rows_without_a_position():
    """Positions past the table and tokens of no sequence are recorded; their
    rows stay, and add nothing to the weight's gradient."""
    from sparse_attention_11_b200 import dsa

    seqs = dsa.Seqs([0, 3, 8], [0, 3, 15])  # positions 0..2 and 7..11
    seqs.c.total_q = 10                     # two rows behind the last sequence
    ra = row_spec(16, torch.randn(16, device="cuda"), 1e-6, 0, 16, dsa.rope_table(10, 16), True)
    x, dy = torch.randn(10, 2, 16, device="cuda"), torch.randn(10, 2, 16, device="cuda")
    x[6:], dy[6:] = float("nan"), float("inf")
    y, dx, dw = torch.full_like(x, NOT_SET), torch.full_like(x, NOT_SET), torch.empty(16, device="cuda")
    ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_NORM_ROPE_BWD, seqs, 16))
    live = [0, 1, 2, 3, 4, 5]
    pos = torch.tensor([0, 1, 2, 7, 8, 9], device="cuda")
    dsa.dsa_norm_rope(seqs, dsa.row_args(**ra), x, y, ws)
    assert dsa.dsa_sync_status(ws)[0] == dsa.DSA_ERR_INDEX
    want, mag = transform(x[live], pos, ra)
    assert bool(((y[live].double() - want).abs() <= U * want.abs() + 48 * U * mag).all())
    assert bool((y[6:] == NOT_SET).all())
    dsa.dsa_norm_rope_bwd(seqs, dsa.row_args(**ra), x, dy, dx, dw, ws)
    assert dsa.dsa_sync_status(ws)[0] == dsa.DSA_ERR_INDEX
    want, mag, want_w, mag_w = transform_bwd(x[live], dy[live], pos, ra)
    assert bool(((dx[live].double() - want).abs() <= U * want.abs() + 160 * U * mag).all())
    assert bool((dx[6:] == NOT_SET).all())
    assert bool(((dw.double() - want_w).abs() <= 80 * U * mag_w).all())


def test_no_rows():
    from sparse_attention_11_b200 import dsa

    seqs = dsa.Seqs([0, 0], [0, 5])
    ra = dsa.row_args(norm_dim=16)
    x, dw = torch.empty(0, 2, 16, device="cuda"), torch.full((16,), NOT_SET, device="cuda")
    ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_NORM_ROPE_BWD, seqs, 16))
    dsa.dsa_norm_rope(seqs, ra, x, torch.empty_like(x), ws)
    dsa.dsa_norm_rope_bwd(seqs, ra, x, torch.empty_like(x), torch.empty_like(x), dw, ws)
    assert bool((dw == 0).all())
