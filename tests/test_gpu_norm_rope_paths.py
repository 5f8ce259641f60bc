"""The query/key transform's paths for aligned and for other rows: the norm does
not depend on where a row lies."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _both(dim, n, fill):
    """fill(x) on a tensor of aligned rows and on one whose rows begin off 16 bytes."""
    for pad in (0, 1):
        t = torch.zeros(n, 1, dim + pad, device="cuda")[:, :, pad:]
        yield fill(t)


@pytest.mark.parametrize("dim", [8, 64, 128, 256, 576, 1024])
def test_norm_is_the_same_off_alignment(dim):
    """Rows with one value each: their sums have one term and so no order, and the
    reciprocal root shows in the output's last bits."""
    from sparse_attention_11_b200 import dsa

    n = 4096
    g = torch.Generator(device="cuda")
    g.manual_seed(dim)
    v = torch.randn(n, generator=g, device="cuda")
    at = torch.randint(0, dim, (n,), generator=g, device="cuda")
    t = torch.arange(n, device="cuda")
    seqs, ra = dsa.Seqs([0, n], [0, n]), dsa.row_args(norm_dim=dim, eps=1e-6)
    ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_NORM_ROPE_BWD, seqs, dim))

    def forward(x):
        x[t, 0, at] = v
        y = torch.empty_strided(x.shape, x.stride(), device="cuda")
        dsa.dsa_norm_rope(seqs, ra, x, y, ws)
        return y[t, 0, at]

    def backward(x):  # d_y beside x's value: d_x is r times it
        x[t, 0, at] = v
        dy, dx = torch.zeros_like(x), torch.empty_strided(x.shape, x.stride(), device="cuda")
        dy[t, 0, (at + 1) % dim] = 1.0
        dsa.dsa_norm_rope_bwd(seqs, ra, x, dy, dx, None, ws)
        return dx[t, 0, (at + 1) % dim]

    for f in (forward, backward):
        a, b = _both(dim, n, f)
        assert torch.equal(a, b), f.__name__
    dsa.check_device_status(ws)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim,heads", [(128, 32), (256, 4), (576, 1), (75, 3)])
def test_backward_captured(dim, heads, dtype):
    """The kernel that sums the weight's gradient starts before its terms are written:
    captured several times in a row, replayed with new inputs, the bits of the call."""
    from sparse_attention_11_b200 import dsa

    T = 700
    seqs = dsa.Seqs([0, T], [0, T])
    ra = dsa.row_args(norm_dim=dim, weight=torch.randn(dim, device="cuda"), rope_dim=24, rope_begin=8,
                      cos_sin=dsa.rope_table(T, 24))
    x, dy = (torch.empty(T, heads, dim, dtype=dtype, device="cuda") for _ in range(2))
    dx, dw = torch.empty_like(x), [torch.empty(dim, device="cuda") for _ in range(3)]
    ws = dsa.workspace(dsa.dsa_workspace_size(dsa.DSA_OP_NORM_ROPE_BWD, seqs, dim))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        for w in dw:
            dsa.dsa_norm_rope_bwd(seqs, ra, x, dy, dx, w, ws)
    for i in range(5):
        x.copy_(torch.randn(x.shape, device="cuda")), dy.copy_(torch.randn(x.shape, device="cuda"))
        g.replay()
        got = [t.clone() for t in (dx, *dw)]
        want = torch.empty_like(dw[0])
        dsa.dsa_norm_rope_bwd(seqs, ra, x, dy, dx, want, ws)
        assert torch.equal(got[0], dx) and all(torch.equal(t, want) for t in got[1:])
    dsa.check_device_status(ws)
