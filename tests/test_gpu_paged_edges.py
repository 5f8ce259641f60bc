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
